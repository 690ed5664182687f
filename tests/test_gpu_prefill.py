"""Attention of ragged batches of new tokens over the paged cache, on the GPU,
against the 64-bit definition."""
import numpy as np
import pytest
import torch

import paged_kv_cache_234_gb300 as pkv
import serving_reference as R
from gpu_common import dev, ensure_built

pytestmark = pytest.mark.gpu


def slopes_of(heads):
    return (2.0 ** (-8.0 * np.arange(1, heads + 1) / heads)).astype(np.float32)


OPTIONS = {
    "plain": {},
    "cap": dict(cap=8.0),
    "bias": dict(bias=True),
    "window": dict(window=40),
    "window1": dict(window=1),
    "window_all": dict(window=2 ** 31 - 1, prefix=3),
    "prefix": dict(prefix=50),
    "window_prefix": dict(window=40, prefix=21),
    "all": dict(cap=20.0, bias=True, window=100, prefix=5),
}


class Run:
    def __init__(self, b, kind, pools, cap=0.0, window=0, slopes=None, prefix=None, tables=None,
                 lens=None, starts=None, max_ctx=None, scale=None, stream=None):
        ensure_built()
        t, hq, d = b.q.shape
        n = b.ctx.size
        mcl = int(b.ctx.max()) if max_ctx is None else max_ctx
        self.out = torch.full((t, hq, d), 7.0, dtype=torch.float16, device="cuda")
        nbytes = pkv.pkv_prefill_workspace_size(t, n, hq, b.kv_heads, d, mcl)
        # NaN in the workspace: nothing may be read before it is written
        self.ws = torch.full((max(nbytes, 16) // 4,), float("nan"), device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.q = dev(b.q)
        self.args = (self.out, self.q, *(dev(x) for x in pools),
                     dev(b.tables if tables is None else tables),
                     dev(b.starts if starts is None else starts),
                     dev(b.ctx if lens is None else lens), mcl,
                     d ** -0.5 if scale is None else scale, self.ws)
        self.kw = dict(logit_cap=cap, window=window, slopes=None if slopes is None else dev(slopes),
                       prefix_lens=None if prefix is None else dev(prefix),
                       dev_status=self.status, stream=stream)
        self.kind = kind

    def __call__(self):
        getattr(pkv, "pkv_paged_prefill_" + self.kind)(*self.args, **self.kw)
        torch.cuda.synchronize()
        return self.out.cpu().numpy().astype(np.float64), int(self.status.item())


def expand(b, option):
    o = dict(OPTIONS[option]) if isinstance(option, str) else dict(option)
    slopes = slopes_of(b.heads) if o.pop("bias", False) else None
    prefix = o.pop("prefix", None)
    if prefix is not None:
        prefix = np.asarray([(prefix, 0, -3, prefix + 16, 10 ** 6)[i % 5]
                             for i in range(b.ctx.size)], np.int32)
    return dict(o, slopes=slopes, prefix=prefix)


def bound(b, kind, o, ref, mass, scale=None):
    scale = b.dim ** -0.5 if scale is None else scale
    # keys enter the product as fp16 values without the decode's constant
    dz = R.score_error(b, "fp16", abs(scale), o.get("cap", 0.0), int(b.ctx.max()), o["slopes"])
    # the probabilities are rounded to fp16: half a step, 2^-11; with V scales
    # their product with the ratio is
    return R.tolerance(ref, mass, dz, 11)


def check(b, kind, option, scale=None):
    o = expand(b, option)
    pools, kv64 = R.cache(b, kind)
    got, status = Run(b, kind, pools, scale=scale, **o)()
    ref, mass = R.attend(b, kv64, b.dim ** -0.5 if scale is None else scale, **o)
    rows = int(b.starts[-1])
    assert status == 0
    assert np.all(np.isfinite(got[:rows]))
    worst = np.max(np.abs(got - ref)[:rows] / bound(b, kind, o, ref, mass, scale)[:rows])
    assert worst <= 1.0, worst
    assert np.all(got[rows:] == 7.0)


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("dim", [64, 128])
def test_one_tile(kind, dim):
    b = R.make(1, [32], [32], 4, 1, dim)
    check(b, kind, "plain")


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("option", OPTIONS)
def test_ragged(kind, dim, option):
    q = [1, 5, 0, 64, 17, 130, 2]
    ctx = [1, 200, 40, 64, 33, 301, 150]
    b = R.make(2, q, ctx, 8, 2, dim, extra_rows=3)
    check(b, kind, option)


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (4, 4), (7, 1), (16, 1), (40, 2)])
def test_group_sizes(kind, heads, kv):
    b = R.make(3, [70, 33], [150, 33], heads, kv, 128)
    check(b, kind, "all")


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("heads", [1, 300])
def test_one_token_and_wide_groups(kind, heads):
    # 300 heads of one kv head: a token's rows lie in two items
    b = R.make(4, [1, 2], [5, 130], heads, 1, 64)
    check(b, kind, "plain")


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("option", ["plain", "all"])
def test_split_over_the_keys(kind, option):
    b = R.make(5, [5, 3], [4001, 2500], 4, 1, 128)
    assert pkv.pkv_prefill_workspace_size(8, 2, 4, 1, 128, 4001) > 0
    check(b, kind, option)


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("option", ["plain", "all", "window_prefix"])
def test_long_without_a_split(kind, dim, option):
    # enough items to fill the GPU: every item walks all of its keys, many
    # times around the ring of tiles
    b = R.make(17, [9, 1, 30, 4], [2300, 1555, 1900, 800], 76, 76, dim)
    assert pkv.pkv_prefill_workspace_size(44, 4, 76, 76, dim, 2300) == 0
    # (the reference of every fourth head)
    o = expand(b, dict(OPTIONS[option], window=700) if option != "plain" else option)
    pools, kv64 = R.cache(b, kind)
    got, status = Run(b, kind, pools, **o)()
    b.heads = 19
    pick = lambda x: np.ascontiguousarray(x[:, ::4])  # noqa: E731
    b.q, b.kv_heads = pick(b.q), 19
    ref, mass = R.attend(b, tuple(pick(x) for x in kv64), b.dim ** -0.5,
                         **dict(o, slopes=None if o["slopes"] is None else o["slopes"][::4]))
    assert status == 0
    worst = np.max(np.abs(got[:, ::4] - ref) / bound(b, kind, o, ref, mass))
    assert worst <= 1.0, worst


def test_split_with_a_window_and_a_prefix_far_apart():
    # most splits of the second sequence have no keys
    b = R.make(6, [5, 9], [4001, 50], 4, 1, 64)
    check(b, "int8", dict(window=300, prefix=200))


@pytest.mark.parametrize("kind", ["fp16", "int8"])
def test_many_sequences(kind):
    n = 90
    rng = np.random.default_rng(0)
    q = rng.integers(0, 9, n)
    b = R.make(7, q, q + rng.integers(0, 60, n), 8, 2, 64)
    check(b, kind, "plain")


@pytest.mark.parametrize("cap", [0.05, 1.0, 1e4])
def test_caps_small_and_large(cap):
    b = R.make(8, [20, 64], [301, 64], 4, 2, 64, q_std=6.0)
    check(b, "fp16", dict(cap=cap))


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.5])
@pytest.mark.parametrize("kind", ["fp16", "fp8"])
def test_scales_of_any_sign(kind, scale):
    b = R.make(9, [20, 64], [201, 64], 4, 2, 64)
    check(b, kind, "window", scale=scale)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_value_scales_of_very_different_size(kind):
    # growing along the context, so that the reference of the ratios moves
    b = R.make(10, [40], [400], 4, 1, 64, nan_tail=False)
    for page in range(25):
        b.v[b.tables[0, page]] *= np.float16(2.0 ** (page % 13 - 6))
    check(b, kind, "plain")


def test_maxima_that_grow_along_the_keys():
    # the running maximum moves by far more than the lazy limit in every tile
    b = R.make(11, [40], [700], 4, 1, 64, q_std=1.0, nan_tail=False)
    for page in range(44):
        b.k[b.tables[0, page]] *= np.float16(0.1 * (1 + page))
    check(b, "fp16", "plain")
    check(b, "fp16", dict(cap=3.0))


@pytest.mark.parametrize("kind", ["fp16", "fp8"])
def test_masked_pages_are_not_read(kind):
    # blocks between prefix and window were freed; masked slots hold NaN
    b = R.make(12, [6], [333], 8, 2, 64)
    window, prefix = 50, np.asarray([20], np.int32)
    pools, kv64 = R.cache(b, kind)
    tables, pools = b.tables.copy(), [x.copy() for x in pools]
    lo = 333 - 6 - window + 1
    for page in range(21):
        t = page * 16 + np.arange(16)
        hidden = (t < lo) & (t >= 20)
        if hidden.all():
            tables[0, page] = -7
        elif hidden.any():
            for x in pools[:2]:
                x[tables[0, page]][:, hidden] = 0x7f if kind == "fp8" else np.nan
    got, status = Run(b, kind, pools, window=window, prefix=prefix, tables=tables)()
    o = dict(window=window, slopes=None, prefix=prefix)
    ref, mass = R.attend(b, kv64, 0.125, **o)
    assert status == 0 and np.all(np.isfinite(got))
    assert np.all(np.abs(got - ref) <= bound(b, kind, o, ref, mass))


@pytest.mark.parametrize("kind", ["fp16", "int8"])
@pytest.mark.parametrize("long", [False, True])
def test_bad_blocks_and_lengths_give_zeros(kind, long):
    # long: with splits over the keys
    far = 4000 if long else 0
    b = R.make(13, [6, 7, 8, 9], [60 + far, 70, 80, 90], 8, 2, 64)
    tables, lens = b.tables.copy(), b.ctx.copy()
    tables[1, 4] = 10 ** 6
    lens[2] = 7                   # eight new tokens
    pools, kv64 = R.cache(b, kind)
    assert (pkv.pkv_prefill_workspace_size(30, 4, 8, 2, 64, 96 + far) > 0) or not long
    got, status = Run(b, kind, pools, tables=tables, lens=lens, max_ctx=96 + far)()
    o = dict(slopes=None, prefix=None)
    ref, mass = R.attend(b, kv64, 0.125)
    ok = np.abs(got - ref) <= bound(b, kind, o, ref, mass)
    assert status == pkv.PKV_DEV_BAD_BLOCK | pkv.PKV_DEV_BAD_CTX
    assert np.all(got[6:21] == 0.0)
    assert np.all(ok[:6]) and np.all(ok[21:])


@pytest.mark.parametrize("start1", [-5, 40])
def test_bad_row_ranges_stay_inside_the_batch(start1):
    b = R.make(14, [4, 4, 4], [20, 30, 40], 8, 2, 64)
    pools, _ = R.cache(b, "fp16")
    starts = np.asarray([0, start1, 8, 12], np.int32)
    r = Run(b, "fp16", pools, starts=starts)
    guard = torch.full((40, 8, 64), 7.0, dtype=torch.float16, device="cuda")
    view = guard[14:26]
    r.args = (view,) + r.args[1:]
    r()
    assert torch.all(guard[:14] == 7.0) and torch.all(guard[26:] == 7.0)


@pytest.mark.parametrize("kind", ["fp16", "int8"])
def test_same_bits_every_time_and_beside_other_calls(kind):
    b = R.make(15, [100, 300], [900, 300], 8, 2, 128)
    pools, _ = R.cache(b, kind)
    r = Run(b, kind, pools)
    first, _ = r()
    s2 = torch.cuda.Stream()
    other = Run(b, kind, pools, stream=s2)
    torch.cuda.synchronize()
    for _ in range(3):
        getattr(pkv, "pkv_paged_prefill_" + kind)(*r.args, **r.kw)
        getattr(pkv, "pkv_paged_prefill_" + kind)(*other.args, **other.kw)
    torch.cuda.synchronize()
    assert np.array_equal(r.out.cpu().numpy().astype(np.float64), first)
    assert np.array_equal(other.out.cpu().numpy().astype(np.float64), first)


def test_captured_and_replayed_on_another_stream():
    b = R.make(16, [5, 1, 30], [2000, 17, 64], 8, 2, 64)
    pools, kv64 = R.cache(b, "fp8")
    st = torch.cuda.Stream()
    r = Run(b, "fp8", pools, cap=10.0, window=64, stream=st)
    torch.cuda.synchronize()
    call = pkv.prepare_paged_prefill_fp8(*r.args, **r.kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    b.q = (b.q.astype(np.float32) * 0.5).astype(np.float16)
    r.q.copy_(dev(b.q))
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    o = dict(cap=10.0, window=64, slopes=None, prefix=None)
    ref, mass = R.attend(b, kv64, 0.125, **o)
    assert np.all(np.abs(r.out.cpu().numpy() - ref) <= bound(b, "fp8", o, ref, mass))
