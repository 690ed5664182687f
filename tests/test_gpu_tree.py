"""Attention of trees of drafted tokens over the paged cache, on the GPU, against
the 64-bit definition."""
import numpy as np
import pytest
import torch

import paged_kv_cache_234_gb300 as pkv
import serving_reference as R
import tree_reference as T
from gpu_common import dev, ensure_built

pytestmark = pytest.mark.gpu
KINDS = ["fp16", "int8", "fp8"]

OPTIONS = {
    "plain": {},
    "cap": dict(cap=8.0),
    "bias": dict(bias=True),
    "window": dict(window=40),
    "window1": dict(window=1),
    "window3": dict(window=3, prefix=17),
    "window_all": dict(window=2 ** 31 - 1, prefix=3),
    "prefix": dict(prefix=50),
    "window_prefix": dict(window=40, prefix=21),
    "all": dict(cap=20.0, bias=True, window=100, prefix=5),
}


class Run:
    def __init__(self, b, kind, pools, parents, cap=0.0, window=0, slopes=None, prefix=None,
                 tables=None, lens=None, starts=None, max_ctx=None, max_tree=None, scale=None,
                 stream=None):
        ensure_built()
        t, hq, d = b.q.shape
        n = b.ctx.size
        mcl = int(b.ctx.max()) if max_ctx is None else max_ctx
        mtl = int(b.q_lens.max()) if max_tree is None else max_tree
        self.out = torch.full((t, hq, d), 7.0, dtype=torch.float16, device="cuda")
        nbytes = pkv.pkv_tree_workspace_size(t, n, hq, b.kv_heads, d, mcl, mtl)
        # NaN in the workspace: nothing may be read before it is written
        self.ws = torch.full((max(nbytes, 16) // 4,), float("nan"), device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        up = np.full(t, -1, np.int32)
        up[:parents.size] = parents
        self.q = dev(b.q)
        self.args = (self.out, self.q, *(dev(x) for x in pools),
                     dev(b.tables if tables is None else tables),
                     dev(b.starts if starts is None else starts),
                     dev(b.ctx if lens is None else lens), dev(up), mcl, mtl,
                     d ** -0.5 if scale is None else scale, self.ws)
        self.kw = dict(logit_cap=cap, window=window, slopes=None if slopes is None else dev(slopes),
                       prefix_lens=None if prefix is None else dev(prefix),
                       dev_status=self.status, stream=stream)
        self.kind = kind

    def __call__(self):
        getattr(pkv, "pkv_paged_tree_" + self.kind)(*self.args, **self.kw)
        torch.cuda.synchronize()
        return self.out.cpu().numpy().astype(np.float64), int(self.status.item())


def expand(b, option):
    o = dict(OPTIONS[option]) if isinstance(option, str) else dict(option)
    slopes = None
    if o.pop("bias", False):
        slopes = (2.0 ** (-8.0 * np.arange(1, b.heads + 1) / b.heads)).astype(np.float32)
    prefix = o.pop("prefix", None)
    if prefix is not None:
        prefix = np.asarray([(prefix, 0, -3, prefix + 16, 10 ** 6)[i % 5]
                             for i in range(b.ctx.size)], np.int32)
    return dict(o, slopes=slopes, prefix=prefix)


def check(b, kind, option, shape="random", scale=None, seed=5, max_tree=None):
    o = expand(b, option)
    pools, kv64 = R.cache(b, kind)
    parents = T.trees(seed, b.q_lens, shape)
    got, status = Run(b, kind, pools, parents, scale=scale, max_tree=max_tree, **o)()
    scale = b.dim ** -0.5 if scale is None else scale
    ref, mass = T.attend(b, parents, kv64, scale, **o)
    rows = int(b.starts[-1])
    assert status == 0
    assert np.all(np.isfinite(got[:rows]))
    worst = np.max(np.abs(got - ref)[:rows] / T.bound(b, o, ref, mass, scale)[:rows])
    assert worst <= 1.0, worst
    assert np.all(got[rows:] == 7.0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
def test_one_small_tree(kind, dim):
    check(R.make(1, [8], [40], 4, 1, dim), kind, "plain")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("option", OPTIONS)
def test_ragged(kind, dim, option):
    q = [1, 5, 0, 64, 17, 33, 2]
    ctx = [1, 200, 40, 64, 33, 301, 150]
    check(R.make(2, q, ctx, 8, 2, dim, extra_rows=3), kind, option)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", ["chain", "star", "roots"])
@pytest.mark.parametrize("option", ["plain", "window3", "all"])
def test_shapes_of_trees(kind, shape, option):
    check(R.make(6, [20, 1, 50], [45, 30, 260], 4, 2, 128), kind, option, shape)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (4, 4), (7, 1), (16, 1), (40, 2)])
def test_group_sizes(kind, heads, kv):
    check(R.make(3, [30, 9], [150, 33], heads, kv, 128), kind, "all")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads", [1, 300])
def test_one_token_and_wide_groups(kind, heads):
    check(R.make(4, [1, 2], [5, 130], heads, 1, 64), kind, "plain")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("option", ["plain", "window_prefix", "all"])
def test_trees_of_many_rows(kind, option):
    # more tokens than a tile of keys, more rows than a work item
    check(R.make(7, [200, 131], [421, 131], 2, 1, 64), kind, option, "roots")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("option", ["plain", "cap", "all", dict(window=700, prefix=300)],
                         ids=["plain", "cap", "all", "window700"])
def test_long_contexts(kind, dim, option):
    check(R.make(5, [12, 3, 1], [4001, 2500, 1111], 4, 2, dim), kind, option)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,heads", [(64, 8), (128, 8), (128, 2)])
@pytest.mark.parametrize("option", ["plain", "all"])
def test_large_trees_over_long_contexts(kind, dim, heads, option):
    # several work items of a tree side by side, many times around the rings
    o = dict(OPTIONS[option], window=8000) if option == "all" else option
    check(R.make(22, [70, 33], [9000, 6000], heads, 1, dim), kind, o)


@pytest.mark.parametrize("kind", KINDS)
def test_every_page_boundary(kind):
    # contexts whose trees begin and end anywhere in a page and in a tile of keys
    q = [n for n in (1, 2, 15, 16, 17) for _ in range(9)]
    ctx = [n + c for n in (1, 2, 15, 16, 17) for c in (0, 1, 15, 16, 17, 111, 112, 127, 128)]
    check(R.make(8, q, ctx, 2, 1, 64), kind, "plain", "roots")


@pytest.mark.parametrize("kind", KINDS)
def test_many_sequences(kind):
    rng = np.random.default_rng(9)
    q = rng.integers(0, 4, 700)
    check(R.make(9, q, q + rng.integers(0, 40, 700), 2, 1, 64), kind, "plain")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [-0.1, 0.0, 1.0])
def test_softmax_scales(kind, scale):
    check(R.make(10, [9, 4], [90, 140], 4, 2, 64), kind, "prefix", scale=scale)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
def test_scores_that_grow_and_shrink(kind, dim):
    # later keys with ever larger, then smaller scores: the reference of the
    # exponentials has to follow
    b = R.make(11, [6, 6], [900, 900], 4, 1, dim)
    for s, up in ((0, 1.0), (1, -1.0)):
        for i, blk in enumerate(b.tables[s][:57]):
            b.k[blk] = (b.k[blk].astype(np.float32) * (0.02 + (i if up > 0 else 57 - i) / 12)
                        ).astype(np.float16)
    check(b, kind, "plain")


@pytest.mark.parametrize("kind", KINDS)
def test_a_bound_above_the_trees(kind):
    check(R.make(12, [5, 9], [50, 60], 4, 1, 64), kind, "plain", max_tree=500)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("dim", [64, 128])
def test_scales_far_apart(kind, dim):
    # V scales over 2^30 and pages of zeros: every row's largest contribution is
    # held to fp16's precision, as the bound has it.  A key's own share p |V| of a
    # page with a small scale keeps 11 bits while it is above 2^-20 of the largest.
    b = R.make(13, [6, 3], [300, 150], 4, 2, dim, nan_tail=False)
    (kc, vc, ks, vs), _ = R.cache(b, kind)
    rng = np.random.default_rng(3)
    vs = (vs * 2.0 ** rng.integers(-20, 10, vs.shape)).astype(np.float32)
    vs[b.tables[0, 2]] = 0.0
    ks = ks.copy()
    ks[b.tables[0, 3]] = 0.0
    val = [R.e4m3(c) if kind == "fp8" else c.astype(np.float64) for c in (kc, vc)]
    kv64 = tuple(v * s[:, :, None, None].astype(np.float64) for v, s in zip(val, (ks, vs)))
    parents = T.trees(4, b.q_lens)
    o = expand(b, "plain")
    got, status = Run(b, kind, (kc, vc, ks, vs), parents)()
    ref, mass = T.attend(b, parents, kv64, dim ** -0.5)
    # beyond fp16's range the output is infinite
    assert status == 0 and np.all(np.isfinite(got) | (np.abs(ref) > 65000))
    ok = np.abs(ref) < 65000
    # products below 2^-14 (the row's largest is 2^6 at least) are rounded by up to
    # 2^-25: 2^-31 of the largest p times V scale, for each of the keys, times a
    # code; that key's largest code is 1 at least, so `mass` holds the product
    extra = 300 * 2.0 ** -31 * (448 if kind == "fp8" else 127) * mass.max(-1, keepdims=True)
    assert np.all((np.abs(got - ref) <= T.bound(b, o, ref, mass, dim ** -0.5) + extra)[ok])


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("value", [np.nan, np.inf, -1.0])
def test_v_scales_that_do_not_belong_show(kind, value):
    # in the rows that see the page, and in no other
    b = R.make(14, [20], [60], 2, 1, 64)
    pools, kv64 = R.cache(b, kind)
    parents = T.trees(4, b.q_lens, "star")
    parents[18] = 17                       # slots 57 and 58 lie in the last page
    vs = pools[3].copy()
    vs[b.tables[0, 3]] = value             # slots 48 .. 63: rows 8 .. 19
    got, status = Run(b, kind, (*pools[:3], vs), parents)()
    ref, mass = T.attend(b, parents, kv64, 0.125)
    assert status == 0
    o = expand(b, "plain")
    fine = np.abs(got - ref) <= T.bound(b, o, ref, mass, 0.125)
    assert np.all(fine[:8]) and np.all(np.isnan(got[8:]))


@pytest.mark.parametrize("kind", KINDS)
def test_single_tokens_match_the_scored_decode(kind):
    b = R.make(15, [1, 1, 1], [700, 33, 16], 8, 2, 128)
    o = expand(b, "all")
    pools, _ = R.cache(b, kind)
    got, _ = Run(b, kind, pools, np.full(3, -1, np.int32), **o)()
    out = torch.empty(b.q.shape, dtype=torch.float16, device="cuda")
    ws = pkv.decode_workspace(3, 8, 2, 128, 700)
    getattr(pkv, "pkv_paged_decode_scored_" + kind)(
        out, dev(b.q), *(dev(x) for x in pools), dev(b.tables), dev(b.ctx), 700, 128 ** -0.5, ws,
        logit_cap=o["cap"], window=o["window"], slopes=dev(o["slopes"]),
        prefix_lens=dev(o["prefix"]))
    kv64 = R.cache(b, kind)[1]
    ref, mass = T.attend(b, np.full(3, -1, np.int32), kv64, 128 ** -0.5, **o)
    tol = T.bound(b, o, ref, mass, 128 ** -0.5)
    dz = R.score_error(b, kind, 128 ** -0.5, o["cap"], 700, o["slopes"])
    both = tol + R.tolerance(ref, mass, dz, 11)
    assert np.all(np.abs(got - out.cpu().numpy().astype(np.float64)) <= both)


# ------------------------------------------------------------- what is refused
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("value", [3, 4, 1000, -2, -2 ** 31, 2 ** 31 - 1])
def test_bad_parents(kind, value):
    b = R.make(16, [6, 8, 4], [30, 50, 300], 4, 2, 64)
    pools, kv64 = R.cache(b, kind)
    parents = T.trees(4, b.q_lens)
    bad = parents.copy()
    bad[6 + 3] = value                     # row 3 of sequence 1
    got, status = Run(b, kind, pools, bad)()
    ref, mass = T.attend(b, parents, kv64, 0.125)
    assert status == pkv.PKV_DEV_BAD_TREE
    ok = np.abs(got - ref) <= T.bound(b, expand(b, "plain"), ref, mass, 0.125)
    assert np.all(ok[:6]) and np.all(got[6:14] == 0) and np.all(ok[14:])


@pytest.mark.parametrize("kind", KINDS)
def test_bad_blocks(kind):
    b = R.make(17, [6, 8], [30, 500], 4, 2, 64)
    pools, kv64 = R.cache(b, kind)
    parents = T.trees(4, b.q_lens)
    ref, mass = T.attend(b, parents, kv64, 0.125)
    tol = T.bound(b, expand(b, "plain"), ref, mass, 0.125)
    for page in (0, 13, 31):
        for value in (-1, b.k.shape[0], 2 ** 31 - 1):
            tables = b.tables.copy()
            tables[1, page] = value
            got, status = Run(b, kind, pools, parents, tables=tables)()
            assert status == pkv.PKV_DEV_BAD_BLOCK
            fine = np.abs(got - ref) <= tol
            assert np.all(fine[:6])
            # rows that need the block get zeros, others may share their work item
            for r in range(8):
                path = 492 + np.asarray(T.path_to(parents[6:], r))
                assert np.all(got[6 + r] == 0) or (page > 30 and not np.any(path // 16 == page)
                                                   and np.all(fine[6 + r]))
    # pages that no row sees may have been freed
    tables = b.tables.copy()
    tables[1, 2:20] = -1
    o = dict(window=100, prefix=np.asarray([20, 20], np.int32), slopes=None)
    got, status = Run(b, kind, pools, parents, tables=tables, **o)()
    ref, mass = T.attend(b, parents, kv64, 0.125, **o)
    assert status == 0
    assert np.all(np.abs(got - ref) <= T.bound(b, o, ref, mass, 0.125))


@pytest.mark.parametrize("kind", KINDS)
def test_sequences_that_do_not_fit(kind):
    b = R.make(18, [6, 8, 3], [30, 50, 60], 4, 2, 64)
    pools, kv64 = R.cache(b, kind)
    parents = T.trees(4, b.q_lens)
    ref, mass = T.attend(b, parents, kv64, 0.125)
    ok = lambda got: np.abs(got - ref) <= T.bound(b, expand(b, "plain"), ref, mass, 0.125)  # noqa
    for lens in ([30, 7, 60], [30, 65, 60], [30, -1, 60], [30, 2 ** 31 - 1, 60]):
        got, status = Run(b, kind, pools, parents, lens=np.asarray(lens, np.int32), max_ctx=64)()
        assert status == pkv.PKV_DEV_BAD_CTX
        assert np.all(ok(got)[:6]) and np.all(got[6:14] == 0) and np.all(ok(got)[14:])
    # a tree above the bound
    got, status = Run(b, kind, pools, parents, max_tree=7)()
    assert status == pkv.PKV_DEV_BAD_CTX
    assert np.all(ok(got)[:6]) and np.all(got[6:14] == 0) and np.all(ok(got)[14:])
    # rows outside the batch
    for starts in ([0, 6, 100, 2 ** 31 - 1], [0, 6, 2, 2], [0, 6, 6, -5], [0, 6, 18, 18]):
        got, status = Run(b, kind, pools, parents, starts=np.asarray(starts, np.int32))()
        assert status == pkv.PKV_DEV_BAD_CTX
        assert np.all(ok(got)[:6])


# ---------------------------------------------------------------- ways to call
@pytest.mark.parametrize("kind", KINDS)
def test_streams_graphs_and_two_calls(kind):
    b = R.make(19, [9, 4, 30], [300, 90, 1000], 8, 2, 128)
    pools, _ = R.cache(b, kind)
    parents = T.trees(4, b.q_lens)
    want, status = Run(b, kind, pools, parents)()
    assert status == 0
    side = torch.cuda.Stream()
    one, two = Run(b, kind, pools, parents, stream=side), Run(b, kind, pools, parents)
    torch.cuda.synchronize()
    for r in (one, two):    # at the same time, with a workspace each
        getattr(pkv, "pkv_paged_tree_" + kind)(*r.args, **r.kw)
    torch.cuda.synchronize()
    for r in (one, two):
        assert np.array_equal(r.out.cpu().numpy().astype(np.float64), want)
    # two captured calls that share a workspace, replayed one after the other
    first, second = Run(b, kind, pools, parents), Run(b, kind, pools, parents)
    second.args = second.args[:-1] + (first.ws,)
    graphs = []
    for r in (first, second):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r.kw["stream"] = torch.cuda.current_stream()
            getattr(pkv, "pkv_paged_tree_" + kind)(*r.args, **r.kw)
        graphs.append(g)
    for _ in range(3):
        for r, g in zip((first, second), graphs):
            r.out.fill_(7.0)
            first.ws.fill_(float("nan"))
            g.replay()
    torch.cuda.synchronize()
    for r in (first, second):
        assert np.array_equal(r.out.cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("option", ["plain", "all"])
def test_results_depend_on_what_is_seen_alone(kind, option):
    # other values in slots that no row sees, other neighbours in the batch
    q, ctx = [5, 12], [75, 600]
    b = R.make(20, q, ctx, 4, 2, 128, nan_tail=False)
    o = expand(b, option)
    parents = T.trees(4, b.q_lens)
    pools, _ = R.cache(b, kind)
    want, _ = Run(b, kind, pools, parents, **o)()
    again, _ = Run(b, kind, pools, parents, **o)()
    assert np.array_equal(want, again)
    if kind == "fp16":
        changed = [x.copy() for x in pools]
        for x in changed:
            x[b.tables[0, 4], :, 75 % 16:] = np.nan
            x[b.tables[1, 37], :, 600 % 16:] = np.inf
        got, _ = Run(b, kind, changed, parents, **o)()
        assert np.array_equal(want, got)


def test_offsets_beyond_32_bits():
    # blocks at the end of pools of more than 2^31 values
    ensure_built()
    b = R.make(21, [7, 3], [200, 90], 16, 8, 128, nan_tail=False)
    far = (1 << 31) // (8 * 16 * 128) + 9
    nb = b.k.shape[0]
    parents = T.trees(4, b.q_lens)
    ref, mass = T.attend(b, parents, (b.k.astype(np.float64), b.v.astype(np.float64)), 128 ** -0.5)
    big = [torch.empty((far + nb, 8, 16, 128), dtype=torch.float16, device="cuda") for _ in "kv"]
    for x, y in zip(big, (b.k, b.v)):
        x[far:] = dev(y)
    out = torch.empty(b.q.shape, dtype=torch.float16, device="cuda")
    ws = pkv.tree_workspace(10, 2, 16, 8, 128, 200, 7)
    tables = np.where(b.tables >= 0, b.tables + far, -1).astype(np.int32)
    pkv.pkv_paged_tree_fp16(out, dev(b.q), *big, dev(tables), dev(b.starts), dev(b.ctx),
                            dev(parents), 200, 7, 128 ** -0.5, ws)
    got = out.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - ref) <= T.bound(b, expand(b, "plain"), ref, mass, 128 ** -0.5))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seqs,tree,heads,kv,dim,ctx", [(9, 30, 14, 2, 64, 700), (3, 40, 8, 2, 128, 1500),
                                                        (2, 70, 4, 1, 128, 5000)])
@pytest.mark.parametrize("option", ["plain", "all"])
def test_splits_of_the_keys_joined(kind, seqs, tree, heads, kv, dim, ctx, option):
    # many rows, split over the keys; uneven trees and lengths, so parts without keys
    q = [1 + (tree - 1) * (i % 3) // 2 for i in range(seqs)]
    b = R.make(60 + seqs, q, [max(n, ctx * (i + 1) // seqs) for i, n in enumerate(q)], heads, kv, dim)
    assert pkv.pkv_tree_workspace_size(sum(q), seqs, heads, kv, dim, int(b.ctx.max()), max(q)) > 0
    check(b, kind, option)
