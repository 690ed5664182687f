"""The cached rows that stay, moved together in place, on the GPU: pools to the
bit, and for code caches the codes and scales that the quantizer gives the moved
tiles."""
import numpy as np
import pytest
import torch

import paged_kv_cache_234_gb300 as pkv
import serving_reference as R
import tree_reference as T
from gpu_common import dev, ensure_built

pytestmark = pytest.mark.gpu
KINDS = ["fp16", "int8", "fp8"]


class Run:
    def __init__(self, b, kind, kept, kept_lens, tables=None, lens=None, starts=None, codes=None,
                 stream=None):
        ensure_built()
        self.kind = kind
        self.pools = [dev(b.k), dev(b.v)]
        self.codes = []
        if kind != "fp16":
            t = torch.int8 if kind == "int8" else torch.uint8
            self.codes = [torch.full(b.k.shape, 5, dtype=t, device="cuda") for _ in "kv"]
            self.codes += [torch.full(b.k.shape[:2], -2.0, device="cuda") for _ in "kv"]
        self.new = torch.full((b.ctx.size,), 77, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.args = (*self.pools, *self.codes, dev(np.asarray(kept, np.int32)),
                     dev(np.asarray(kept_lens, np.int32)), self.new,
                     dev(b.starts if starts is None else np.asarray(starts, np.int32)),
                     dev(b.ctx if lens is None else np.asarray(lens, np.int32)),
                     dev(b.tables if tables is None else tables))
        self.kw = dict(dev_status=self.status, stream=stream)

    def __call__(self):
        getattr(pkv, "pkv_compact_" + self.kind)(*self.args, **self.kw)
        torch.cuda.synchronize()
        return self

    def check(self, b, lens, pools, written):
        assert np.array_equal(self.new.cpu().numpy(), lens)
        for got, want in zip(self.pools, pools):
            assert np.array_equal(got.cpu().numpy().view(np.uint16), want.view(np.uint16))
        if self.kind == "fp16":
            return
        for i in range(2):
            codes, scales = (self.codes[j].cpu().numpy() for j in (i, 2 + i))
            rest = np.setdiff1d(np.arange(codes.shape[0]), written)
            assert np.all(codes[rest] == 5) and np.all(scales[rest] == -2.0)
            if written.size:
                want_c, want_s = T.tiles(self.kind, pools[i], written)
                assert np.array_equal(codes[written].view(np.uint8), want_c.view(np.uint8))
                assert np.array_equal(scales[written].view(np.uint32), want_s.view(np.uint32))


def some(seed, q_lens, counts):
    """Rising rows, counts[s] of each sequence's q_lens[s]."""
    rng = np.random.default_rng(seed)
    kept = []
    for n, m in zip(q_lens, counts):
        k = np.full(n, -1, np.int32)
        k[:m] = np.sort(rng.permutation(n)[:m])
        kept.append(k)
    return np.concatenate(kept) if kept else np.zeros(0, np.int32)


def check(b, kind, kept, counts, **kw):
    r = Run(b, kind, kept, counts, **kw)()
    assert int(r.status.item()) == 0
    r.check(b, *T.compact(b, kept, counts, (b.k, b.v)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
def test_paths(kind, dim):
    q = [1, 7, 16, 0, 33, 17, 5, 40]
    ctx = [1, 30, 16, 9, 100, 64, 21, 40]
    counts = [1, 3, 4, 0, 9, 17, 0, 1]
    b = R.make(1, q, ctx, 4, 2, dim)
    check(b, kind, some(1, q, counts), counts)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("share", [0.02, 0.5, 0.97])
@pytest.mark.parametrize("n,seqs", [(90, 3), (700, 2), (5000, 1)])
def test_whole_contexts(kind, dim, share, n, seqs):
    # a warp, a CTA or a cluster to each sequence and head
    q = [n - 13 * s for s in range(seqs)]
    counts = [max(1, int(share * x)) for x in q]
    b = R.make(2, q, q, 2, 2, dim, nan_tail=False)
    check(b, kind, some(n, q, counts), counts)


@pytest.mark.parametrize("kind", KINDS)
def test_every_offset_in_a_page(kind):
    # the first row anywhere in its page, moved by every distance to another one
    q = [40] * 48
    ctx = [40 + i for i in range(48)]
    counts = [20] * 48
    kept = np.concatenate([np.concatenate([np.arange(20) + i % 21, np.full(20, -1)])
                           for i in range(48)]).astype(np.int32)
    check(R.make(3, q, ctx, 1, 1, 64), kind, kept, counts)


@pytest.mark.parametrize("kind", KINDS)
def test_rows_that_stay_are_not_written(kind):
    # all rows kept; only the last ones moved; none kept
    q, ctx = [50, 50, 50], [70, 70, 70]
    counts = [50, 48, 0]
    kept = np.concatenate([np.arange(50), np.r_[np.arange(40), np.arange(42, 50), -1, -1],
                           np.arange(50)]).astype(np.int32)
    check(R.make(4, q, ctx, 2, 1, 128), kind, kept, counts)


@pytest.mark.parametrize("kind", KINDS)
def test_tiles_with_nan_and_infinities(kind):
    b = R.make(5, [60], [60], 2, 1, 64, nan_tail=False)
    rng = np.random.default_rng(1)
    for x in (b.k, b.v):
        flat = x.reshape(-1)
        flat[rng.permutation(flat.size)[:40]] = np.nan
        flat[rng.permutation(flat.size)[:4]] = np.inf
        x[b.tables[0, 1]] = 0
    check(b, kind, some(6, [60], [45]), [45])


@pytest.mark.parametrize("kind", KINDS)
def test_many_sequences(kind):
    rng = np.random.default_rng(7)
    q = rng.integers(0, 20, 900)
    counts = rng.integers(0, q + 1)
    b = R.make(7, q, q + rng.integers(0, 30, 900), 2, 1, 64)
    check(b, kind, some(8, q, counts), counts)


def test_twice_in_a_row():
    # what is left is thinned out again, with the new lengths as lengths
    b = R.make(9, [300, 200], [300, 200], 2, 1, 64, nan_tail=False)
    first, second = [150, 120], [70, 119]
    kept = some(9, [300, 200], first)
    r = Run(b, "int8", kept, first)()
    lens, pools, _ = T.compact(b, kept, first, (b.k, b.v))
    b.k, b.v = pools
    b.ctx, b.q_lens = lens, np.asarray(first)
    b.starts = np.asarray([0, 150, 270], np.int32)
    kept = some(10, first, second)
    r2 = Run(b, "int8", kept, second, lens=r.new.cpu().numpy())()
    r2.check(b, *T.compact(b, kept, second, (b.k, b.v)))


# ------------------------------------------------------------- what is refused
@pytest.mark.parametrize("kind", KINDS)
def test_counts_and_sequences_that_do_not_fit(kind):
    b = R.make(11, [10, 12, 9], [30, 40, 50], 2, 1, 64)
    kept = some(11, b.q_lens, [4, 5, 6])
    want = T.compact(b, kept, [4, 0, 6], (b.k, b.v))

    def left_alone(r, bit, length=40):
        assert int(r.status.item()) == bit
        want[0][1] = length
        r.check(b, *want)
    for m in (-1, 13, 2 ** 31 - 1, -2 ** 31):
        left_alone(Run(b, kind, kept, [4, m, 6])(), pkv.PKV_DEV_BAD_KEEP)
    for c in (11, -5, 16 * b.tables.shape[1] + 1, 2 ** 31 - 1):
        left_alone(Run(b, kind, kept, [4, 5, 6], lens=[30, c, 50])(), pkv.PKV_DEV_BAD_CTX, c)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("starts", [[0, 10, 100, 2 ** 31 - 1], [0, 10, 4, 4], [0, 10, 10, -5],
                                    [0, 10, 32, 32]])
def test_rows_outside_the_batch(kind, starts):
    b = R.make(12, [10, 12, 9], [30, 40, 50], 2, 1, 64)
    kept = some(12, b.q_lens, [4, 5, 6])
    counts = [4, 5, 6] if starts[2] != starts[1] and starts[3] != starts[2] else [4, 5, 0]
    if starts[1] == starts[2]:
        counts = [4, 0, 6]
    r = Run(b, kind, kept, counts, starts=starts)()
    assert int(r.status.item()) == pkv.PKV_DEV_BAD_CTX
    want = T.compact(b, kept, [4, 0, 0], (b.k, b.v))
    want[0][1:] = b.ctx[1:]
    r.check(b, *want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("entry", [-1, 12, 2, 1, 2 ** 31 - 1, -2 ** 31])
def test_bad_entries_are_not_moved(kind, entry):
    # (an entry below its own number, or not above the one before)
    b = R.make(13, [10, 12], [30, 40], 2, 1, 64)
    kept = np.full(22, -1, np.int32)
    kept[:3] = [1, 2, 9]
    kept[10:15] = [0, 2, 3, entry, 11]
    r = Run(b, kind, kept, [3, 5])()
    assert int(r.status.item()) == pkv.PKV_DEV_BAD_KEEP
    assert np.array_equal(r.new.cpu().numpy(), [23, 33])
    fixed = kept.copy()
    fixed[13] = 3                          # stays where it is
    if entry > 11:
        fixed[14] = 4                      # and the next one, which is not above it
    _, pools, _ = T.compact(b, fixed, [3, 5], (b.k, b.v))
    for got, want in zip(r.pools, pools):
        got, want = (x.view(np.uint16) for x in (got.cpu().numpy(), want))
        assert np.array_equal(got[b.tables[0, :2]], want[b.tables[0, :2]])
        blk, slot = b.tables[1, 2], (28 + 4) % 16
        assert np.array_equal(got[blk, :, slot], want[blk, :, slot])
        rest = np.setdiff1d(np.arange(got.shape[0]), np.r_[b.tables[0, :2], b.tables[1, :3]])
        assert np.array_equal(got[rest], want[rest])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("value", [-1, 1 << 20, 2 ** 31 - 1, -2 ** 31])
def test_bad_blocks(kind, value):
    b = R.make(14, [40, 12], [40, 40], 2, 1, 64, nan_tail=False)
    kept = np.concatenate([np.r_[np.arange(20, 40), np.full(20, -1)], some(14, [12], [5])])
    for page, moved in ((0, range(16, 20)), (1, range(12, 16)), (2, range(0, 12))):
        tables = b.tables.copy()
        tables[0, page] = value
        r = Run(b, kind, kept, [20, 5], tables=tables)()
        assert int(r.status.item()) == pkv.PKV_DEV_BAD_BLOCK
        # rows 20 .. 39 move to 0 .. 19: those whose page or source is bad do not
        want = [x.copy() for x in T.compact(b, kept, [20, 5], (b.k, b.v))[1]]
        for x, y in zip(want, (b.k, b.v)):
            x[b.tables[0]] = y[b.tables[0]]
            for j in moved:
                x[b.tables[0, j // 16], :, j % 16] = y[b.tables[0, (j + 20) // 16], :, (j + 20) % 16]
        for got, w in zip(r.pools, want):
            assert np.array_equal(got.cpu().numpy().view(np.uint16), w.view(np.uint16))


def test_captured_and_on_another_stream():
    b = R.make(15, [64, 30], [90, 30], 2, 1, 128)
    kept = some(15, b.q_lens, [20, 10])
    want = T.compact(b, kept, [20, 10], (b.k, b.v))
    side = torch.cuda.Stream()
    r = Run(b, "fp8", kept, [20, 10], stream=side)
    torch.cuda.synchronize()
    r().check(b, *want)
    r = Run(b, "fp8", kept, [20, 10])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.kw["stream"] = torch.cuda.current_stream()
        pkv.pkv_compact_fp8(*r.args, **r.kw)
    for _ in range(2):   # the second time over the same, restored pools
        for x, y in zip(r.pools, (b.k, b.v)):
            x.copy_(dev(y))
        g.replay()
    torch.cuda.synchronize()
    r.check(b, *want)


def test_offsets_beyond_32_bits():
    ensure_built()
    b = R.make(16, [90, 40], [130, 60], 8, 8, 128, nan_tail=False)
    far = (1 << 31) // (8 * 16 * 128) + 9
    counts = [50, 20]
    kept = some(16, b.q_lens, counts)
    lens, pools, written = T.compact(b, kept, counts, (b.k, b.v))
    shape = (far + b.k.shape[0], 8, 16, 128)
    big = [torch.empty(shape, dtype=torch.float16, device="cuda") for _ in "kv"]
    codes = [torch.empty(shape, dtype=torch.int8, device="cuda") for _ in "kv"]
    scales = [torch.empty(shape[:2], device="cuda") for _ in "kv"]
    for x, y in zip(big, (b.k, b.v)):
        x[far:] = dev(y)
    new = torch.empty(2, dtype=torch.int32, device="cuda")
    tables = np.where(b.tables >= 0, b.tables + far, -1).astype(np.int32)
    pkv.pkv_compact_int8(*big, *codes, *scales, dev(kept), dev(np.asarray(counts, np.int32)), new,
                         dev(b.starts), dev(b.ctx), dev(tables))
    assert np.array_equal(new.cpu().numpy(), lens)
    for i in range(2):
        got = big[i][far:].cpu().numpy()
        assert np.array_equal(got.view(np.uint16), pools[i].view(np.uint16))
        want_c, want_s = T.tiles("int8", pools[i], written)
        assert np.array_equal(codes[i][far:].cpu().numpy()[written], want_c)
        assert np.array_equal(scales[i][far:].cpu().numpy()[written], want_s)
