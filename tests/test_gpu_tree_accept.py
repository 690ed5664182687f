"""The accepted path of every tree of drafted tokens, on the GPU, against a plain
search through all rows."""
import numpy as np
import pytest
import torch

import paged_kv_cache_234_gb300 as pkv
import tree_reference as T
from gpu_common import dev, ensure_built

pytestmark = pytest.mark.gpu


def run(parents, tokens, targets, starts, n=None):
    ensure_built()
    n = len(starts) - 1 if n is None else n
    kept = torch.full((parents.size,), 77, dtype=torch.int32, device="cuda")
    lens = torch.full((n,), 77, dtype=torch.int32, device="cuda")
    last = torch.full((n,), 77, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.pkv_tree_accept(kept, lens, last, dev(tokens), dev(targets), dev(parents),
                        dev(np.asarray(starts, np.int32)), dev_status=status)
    torch.cuda.synchronize()
    return kept.cpu().numpy(), lens.cpu().numpy(), last.cpu().numpy(), int(status.item())


def drafts(seed, q_lens, shape, vocab, follow=0.8):
    rng = np.random.default_rng(seed)
    parents = T.trees(seed, q_lens, shape)
    starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    t = int(starts[-1])
    tokens = rng.integers(0, vocab, t).astype(np.int32)
    targets = rng.integers(0, vocab, t).astype(np.int32)
    up = np.repeat(starts[:-1], q_lens) + parents
    right = np.flatnonzero((parents >= 0) & (rng.random(t) < follow))
    targets[up[right]] = tokens[right]
    return parents, tokens, targets, starts


@pytest.mark.parametrize("shape", ["random", "chain", "star", "roots"])
@pytest.mark.parametrize("vocab", [2, 1000])
@pytest.mark.parametrize("q_lens", [[1], [8, 0, 1, 64, 31, 32, 33, 97, 2], [1500, 3], [5] * 600],
                         ids=["one", "ragged", "long", "many"])
def test_against_a_plain_search(shape, vocab, q_lens):
    # (2 tokens: many siblings that are alike, of which the first is taken)
    parents, tokens, targets, starts = drafts(len(q_lens) + vocab, q_lens, shape, vocab)
    kept, lens, last, status = run(parents, tokens, targets, starts)
    want = T.accept(parents, tokens, targets, starts)
    assert status == 0
    for got, ref in zip((kept, lens, last), want):
        assert np.array_equal(got, ref)


def test_whole_chain_and_nothing_but_the_root():
    n = 70
    parents = np.arange(-1, n - 1, dtype=np.int32)
    tokens = np.arange(n, dtype=np.int32)
    kept, lens, last, _ = run(parents, tokens, tokens + 1, [0, n])
    assert np.array_equal(kept, np.arange(n)) and lens[0] == n and last[0] == n
    kept, lens, last, _ = run(parents, tokens, tokens + 2, [0, n])
    assert lens[0] == 1 and last[0] == 2 and kept[0] == 0 and np.all(kept[1:] == -1)


def test_rows_behind_the_last_sequence_and_none_at_all():
    parents, tokens, targets, starts = drafts(4, [6, 0], "random", 3)
    pad = lambda x: np.concatenate([x, np.full(5, -9, np.int32)])  # noqa: E731
    kept, lens, last, status = run(pad(parents), pad(tokens), pad(targets), starts)
    want = T.accept(parents, tokens, targets, starts)
    assert status == 0 and np.array_equal(kept[:6], want[0]) and np.all(kept[6:] == 77)
    assert np.array_equal(lens, want[1]) and np.array_equal(last, want[2])
    # no tokens, three sequences
    kept, lens, last, status = run(*(np.zeros(0, np.int32),) * 3, [0, 0, 0, 0])
    assert status == 0 and np.all(lens == 0) and np.all(last == -1)


@pytest.mark.parametrize("value", [3, 9, 2 ** 31 - 1, -2, -2 ** 31])
@pytest.mark.parametrize("row", [0, 3, 40])
def test_bad_parents(value, row):
    if row == 40 and value in (3, 9):
        value += 40
    parents, tokens, targets, starts = drafts(5, [6, 50, 7], "random", 3)
    bad = parents.copy()
    bad[6 + row] = value
    kept, lens, last, status = run(bad, tokens, targets, starts)
    want = T.accept(parents, tokens, targets, starts)
    assert status == pkv.PKV_DEV_BAD_TREE
    assert lens[1] == 0 and last[1] == -1 and np.all(kept[6:56] == -1)
    for s, a, e in ((0, 0, 6), (2, 56, 63)):
        assert lens[s] == want[1][s] and last[s] == want[2][s]
        assert np.array_equal(kept[a:e], want[0][a:e])


@pytest.mark.parametrize("starts", [[0, 6, 100, 2 ** 31 - 1], [0, 6, 4, 4], [0, 6, 6, -5],
                                    [0, 6, 13, 13], [-1, 6, 6, 6]])
def test_sequences_outside_the_batch(starts):
    parents, tokens, targets, good = drafts(6, [6, 6], "random", 3)
    kept, lens, last, status = run(parents, tokens, targets, starts)
    want = T.accept(parents[:6], tokens[:6], targets[:6], [0, 6])
    assert status == pkv.PKV_DEV_BAD_CTX
    for s, (a, e) in enumerate(zip(starts[:-1], starts[1:])):
        if a == 0:
            assert lens[s] == want[1][0] and np.array_equal(kept[:6], want[0])
        else:
            assert lens[s] == 0 and last[s] == -1


def test_captured_and_on_another_stream():
    ensure_built()
    parents, tokens, targets, starts = drafts(7, [20, 9], "random", 2)
    want = T.accept(parents, tokens, targets, starts)
    out = [torch.full((x.size,), 77, dtype=torch.int32, device="cuda") for x in want]
    args = [dev(x) for x in (tokens, targets, parents, starts)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    call = pkv.prepare_tree_accept(*out, *args, stream=side)
    call()
    torch.cuda.synchronize()
    assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(out, want))
    for x in out:
        x.fill_(77)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.pkv_tree_accept(*out, *args)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(out, want))
