"""When a prefill call splits its items over their keys, as its workspace shows:
2 * splits * rows * (head_dim + 2) floats."""
import random

import pytest

import paged_kv_cache_234_gb300 as pkv
from paged_kv_cache_234_gb300 import build as pkv_build


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


def splits(tokens, seqs, heads, kv, dim, ctx):
    part = 2 * tokens * heads * (dim + 2) * 4
    size = pkv.pkv_prefill_workspace_size(tokens, seqs, heads, kv, dim, ctx)
    assert size % part == 0
    return size // part or 1


@pytest.mark.parametrize("heads,kv,dim", [(32, 8, 128), (28, 4, 128), (14, 2, 64), (4, 4, 64)])
@pytest.mark.parametrize("seqs", [1, 2, 5])
@pytest.mark.parametrize("tokens", [2048, 4096, 8192])
def test_prompts_by_themselves_are_not_split(heads, kv, dim, seqs, tokens):
    # what the SMs wait for at the end is short items; the join would cost more
    assert splits(seqs * tokens, seqs, heads, kv, dim, tokens) == 1


def test_many_items_are_not_split():
    assert splits(4 * 8192, 4, 32, 8, 128, 32768) == 1
    rng = random.Random(0)
    for _ in range(2000):
        heads, kv = rng.choice([(32, 8), (28, 4), (14, 2), (8, 8), (16, 1)])
        seqs = rng.randrange(1, 300)
        tokens = rng.randrange(seqs, 40000 + seqs)
        items = (tokens // (256 // (heads // kv)) + seqs) * kv
        z = splits(tokens, seqs, heads, kv, 128, rng.randrange(1, 200000))
        assert 1 <= z <= 64 and (z == 1 or items < 608)


def test_few_rows_over_long_contexts_are():
    assert splits(256, 1, 32, 8, 128, 4096) == 3
    assert splits(128, 1, 32, 8, 128, 8192) >= 4
    assert splits(16, 1, 32, 8, 128, 32768) == 19    # 8 items on 152 SMs
    assert splits(160, 32, 14, 2, 64, 2048) == 2
    # too many rows to join
    assert splits(4096, 1, 32, 8, 128, 16384) == splits(1024, 1, 32, 8, 128, 8192) == 1


def test_no_sequences():
    assert pkv.pkv_prefill_workspace_size(5, 0, 8, 2, 64, 4096) == 0


@pytest.mark.parametrize("tokens,seqs,ctx", [(1, 1, 1), (1, 1, 128), (7, 7, 16), (100, 300, 5)])
def test_contexts_of_a_tile_or_two_are_not_split(tokens, seqs, ctx):
    assert splits(tokens, seqs, 8, 2, 64, ctx) == 1
