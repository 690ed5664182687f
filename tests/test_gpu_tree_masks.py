"""Tree attention with few rows: the masks of two masked tiles in a row.

A group of four score warps shares a tile's masks, which its first warp writes. A
tile whose scores exceed the references makes the group read them a second time; the
next tile's must not be written before every warp has. The debug build delays one
warp of every group at each of its waits, the second one's among them, and trees
that lie across a border of the 128-key tiles, or windows that end in two tiles, have
such tiles one behind the other."""
import numpy as np
import pytest

import paged_kv_cache_234_gb300 as pkv
import serving_reference as R
import tree_reference as T
from gpu_common import ensure_built
from test_gpu_tree import check, expand
from test_gpu_tree_waits import DebugRun

pytestmark = pytest.mark.gpu

# A bias makes the tiles behind an item's first exceed its references; so do drafted
# keys that are much larger than the context's.
OPTIONS = {
    "bias": dict(bias=True),
    "bias_cap_window": dict(bias=True, cap=20.0, window=190, prefix=3),
    "sharp": {},
}


def batch(option, dim, wide=False):
    """Trees that begin in the third tile of keys and end in the fourth, so many of them
    that most items are one piece; 5 to 24 rows of a kv head, or 35 to 60."""
    q = [12, 5, 9, 24, 17, 20] if not wide else [12, 7, 9, 11]
    ctx = [384 + n // 2 for n in q]
    heads, kv = (64, 64) if not wide else (160, 32)
    b = R.make(31, q, ctx, heads, kv, dim)
    if option == "sharp":
        for s, n in enumerate(q):
            for t in range(ctx[s] - n, ctx[s]):
                at = (b.tables[s, t // 16], slice(None), t % 16)
                b.k[at] = (b.k[at].astype(np.float32) * 6).astype(np.float16)
    return b


def small_products(b, kind, mass):
    """What `bound` leaves out: products p times V scale below 2^-14, which fp16 rounds by
    up to 2^-25 whatever their size. The row's largest is 2^6 at least, so that is 2^-31
    of it, for each of the keys, times a code (fp16: a value) of at most `most`; and
    `mass` holds the largest, times its key's largest code (value), 1 at least. It counts
    where a single key takes a row and its own code is 0."""
    most = {"fp16": 8, "int8": 127, "fp8": 448}[kind]
    return int(b.ctx.max()) * 2.0 ** -31 * most * mass.max(-1, keepdims=True)


@pytest.fixture
def slow():
    ensure_built()
    L = pkv.debug_lib()

    def put(warp=-1, ns=0):
        assert L.pkv_debug_set_tree_warp(warp, ns) == 0
    put()
    yield put
    put()


@pytest.mark.parametrize("kind,dim", [("fp16", 64), ("fp16", 128), ("int8", 64), ("int8", 128),
                                      ("fp8", 64), ("fp8", 128)])
@pytest.mark.parametrize("wide", [False, True], ids=["32rows", "64rows"])
@pytest.mark.parametrize("option", OPTIONS)
def test_one_slow_warp_of_a_group(kind, dim, wide, option, slow):
    b = batch(option, dim, wide)
    o = expand(b, OPTIONS[option])
    pools, kv64 = R.cache(b, kind)
    parents = T.trees(5, b.q_lens)
    ref, mass = T.attend(b, parents, kv64, dim ** -0.5, **o)
    tol = T.bound(b, o, ref, mass, dim ** -0.5) + small_products(b, kind, mass)
    r = DebugRun(b, kind, pools, parents, **o)
    want, status = r()
    assert status == 0 and np.all(np.abs(want - ref) <= tol)
    for warp in range(4):
        r.out.fill_(7.0)
        slow(warp, 20000)
        got, status = r()
        assert status == 0, warp
        assert np.array_equal(got, want), warp


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("n", [2, 8, 30])
def test_biased_trees_anywhere_around_a_border(kind, n):
    # the border between the second and the third tile before, in and behind the tree
    ends = [256 + e for e in (-1, 0, 1, n // 2, n - 1, n, n + 1)]
    check(R.make(32, [n] * len(ends), ends, 16, 16, 64), kind, "bias")
