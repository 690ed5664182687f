"""Decode attention with capped, biased and masked scores, on the GPU, against
the 64-bit definition."""
import numpy as np
import pytest
import torch

import paged_kv_cache_234_gb300 as pkv
import serving_reference as R
from gpu_common import dev, ensure_built, persistent_workers

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
    "window_prefix": dict(window=40, prefix=21),
    "all": dict(cap=20.0, bias=True, window=100, prefix=5),
}


def run(b, kind, pools, cap=0.0, window=0, slopes=None, prefix=None, tables=None, lens=None,
        max_ctx=None, stream=None):
    ensure_built()
    n, hq, d = b.q.shape
    mcl = int(b.ctx.max()) if max_ctx is None else max_ctx
    out = torch.full((n, hq, d), float("nan"), dtype=torch.float16, device="cuda")
    ws = pkv.decode_workspace(n, hq, b.kv_heads, d, mcl)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    getattr(pkv, "pkv_paged_decode_scored_" + kind)(
        out, dev(b.q), *(dev(x) for x in pools), dev(b.tables if tables is None else tables),
        dev(b.ctx if lens is None else lens), mcl, d ** -0.5, ws, logit_cap=cap, window=window,
        slopes=None if slopes is None else dev(slopes),
        prefix_lens=None if prefix is None else dev(prefix), dev_status=status, stream=stream)
    torch.cuda.synchronize()
    return out.cpu().numpy().astype(np.float64), int(status.item())


def check(b, kind, option, seed=0, rows=None, **kw):
    o = dict(OPTIONS[option]) if isinstance(option, str) else dict(option)
    slopes = slopes_of(b.heads) if o.pop("bias", False) else None
    prefix = o.pop("prefix", None)
    if prefix is not None:
        # different lengths, none, negative and beyond the context among them
        prefix = np.asarray([(-3, 0, prefix, prefix + 16, 10 ** 6)[i % 5] if b.ctx.size > 1
                             else prefix for i in range(b.ctx.size)], np.int32)
    pools, kv64 = R.cache(b, kind)
    got, status = run(b, kind, pools, slopes=slopes, prefix=prefix, **o, **kw)
    scale = b.dim ** -0.5
    ref, mass = R.attend(b, kv64, scale, slopes=slopes, prefix=prefix, **o)
    dz = R.score_error(b, kind, scale, o.get("cap", 0.0), int(b.ctx.max()), slopes)
    # the probabilities enter the product with 22 bits
    tol = R.tolerance(ref, mass, dz, 21)
    assert status == 0
    assert np.all(np.isfinite(got))
    worst = np.max(np.abs(got - ref) / tol)
    assert worst <= 1.0, worst
    return got


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("option", OPTIONS)
def test_small_batches(kind, dim, option):
    # one item per cluster; lengths around pages and windows
    ctx = [1, 15, 16, 17, 39, 40, 41, 57, 100, 128, 0, 200]
    b = R.make(3, [1] * 12, ctx, 8, 2, dim)
    check(b, kind, option)


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("option", OPTIONS)
def test_persistent_workers(kind, option):
    ctx = [1, 15, 16, 17, 39, 40, 41, 57, 100, 128, 0, 200]
    b = R.make(4, [1] * 12, ctx, 8, 2, 64)
    for cap in (3, 13, 4096):
        with persistent_workers(cap):
            check(b, kind, option)


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (4, 4), (7, 1), (8, 1), (9, 1), (16, 1), (40, 2)])
def test_group_sizes(kind, heads, kv):
    b = R.make(5, [1] * 3, [77, 130, 30], heads, kv, 128)
    check(b, kind, "all")
    with persistent_workers(5):
        check(b, kind, "all")


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("option", ["bias", "all"])
def test_one_long_context(kind, option):
    # many pieces, merged by several CTAs per task
    b = R.make(6, [1], [20011], 8, 1, 128)
    check(b, kind, option)


def test_large_window_on_a_long_context():
    b = R.make(7, [1, 1], [9001, 5003], 4, 1, 64)
    check(b, "int8", dict(window=4097, prefix=33, cap=30.0))


@pytest.mark.parametrize("cap", [0.05, 1.0, 1e4])
def test_caps_small_and_large(cap):
    b = R.make(8, [1, 1], [301, 64], 4, 2, 64, q_std=6.0)
    check(b, "fp16", dict(cap=cap))


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("persistent", [False, True])
def test_masked_pages_are_not_read(kind, persistent):
    # blocks between the prefix and the window were freed: their table entries
    # name nothing; the masked slots of the pages at the borders hold NaN
    b = R.make(9, [1, 1], [333, 250], 8, 2, 64)
    window, prefix = 50, np.asarray([20, 0], np.int32)
    tables = b.tables.copy()
    k, v = b.k.copy(), b.v.copy()
    for s in range(2):
        lo, pre = int(b.ctx[s]) - window, int(prefix[s])
        for page in range(-(-int(b.ctx[s]) // 16)):
            t = page * 16 + np.arange(16)
            hidden = (t < lo) & (t >= pre)
            if hidden.all():
                tables[s, page] = -7
            elif hidden.any() and kind == "fp16":
                k[tables[s, page]][:, hidden] = np.nan
                v[tables[s, page]][:, hidden] = np.inf
    pools, kv64 = R.cache(b, kind)
    if kind == "fp16":
        pools = (k, v)
    elif kind == "fp8":  # NaN codes
        kc, vc = pools[0].copy(), pools[1].copy()
        for s in range(2):
            lo, pre = int(b.ctx[s]) - window, int(prefix[s])
            for page in range(-(-int(b.ctx[s]) // 16)):
                t = page * 16 + np.arange(16)
                hidden = (t < lo) & (t >= pre)
                if hidden.any() and not hidden.all():
                    kc[tables[s, page]][:, hidden] = 0x7f
                    vc[tables[s, page]][:, hidden] = 0x7f
        pools = (kc, vc) + pools[2:]
    if persistent:
        with persistent_workers(7):
            got, status = run(b, kind, pools, window=window, prefix=prefix, tables=tables)
    else:
        got, status = run(b, kind, pools, window=window, prefix=prefix, tables=tables)
    ref, mass = R.attend(b, kv64, 0.125, window=window, prefix=prefix)
    tol = R.tolerance(ref, mass, R.score_error(b, kind, 0.125, 0.0, 333, None), 21)
    assert status == 0
    assert np.all(np.isfinite(got)) and np.all(np.abs(got - ref) <= tol)


@pytest.mark.parametrize("kind", ["fp16", "int8"])
@pytest.mark.parametrize("persistent", [False, True])
def test_bad_blocks_and_lengths_give_zeros(kind, persistent):
    b = R.make(10, [1] * 4, [60, 70, 80, 90], 8, 2, 64)
    tables, lens = b.tables.copy(), b.ctx.copy()
    tables[1, 4] = 10 ** 6
    lens[2] = 97
    pools, kv64 = R.cache(b, kind)
    def call():
        return run(b, kind, pools, window=30, tables=tables, lens=lens, max_ctx=96)
    if persistent:
        with persistent_workers(6):
            got, status = call()
    else:
        got, status = call()
    ref, mass = R.attend(b, kv64, 0.125, window=30)
    assert status == pkv.PKV_DEV_BAD_BLOCK | pkv.PKV_DEV_BAD_CTX
    assert np.all(got[1:3] == 0.0)
    tol = R.tolerance(ref, mass, R.score_error(b, kind, 0.125, 0.0, 96, None), 21)
    assert np.all(np.abs(got - ref)[[0, 3]] <= tol[[0, 3]])


def test_plain_options_agree_with_the_plain_decode():
    b = R.make(11, [1] * 5, [100, 1, 64, 333, 20], 8, 2, 128)
    pools, _ = R.cache(b, "int8")
    got, _ = run(b, "int8", pools)
    out = torch.empty(b.q.shape, dtype=torch.float32, device="cuda")
    ws = pkv.decode_workspace(5, 8, 2, 128, 333)
    pkv.pkv_paged_decode_int8(out, dev(b.q), *(dev(x) for x in pools), dev(b.tables), dev(b.ctx),
                              333, 128 ** -0.5, ws)
    want = out.half().cpu().numpy().astype(np.float64)
    # the same kernel up to the splits' rounding, then one fp16 step apart at most
    assert np.all(np.abs(got - want) <= 2.0 ** -10 * np.abs(want) + 2.0 ** -20)


def test_captured_and_replayed_on_another_stream():
    b = R.make(12, [1] * 4, [100, 17, 64, 333], 8, 2, 64)
    pools, kv64 = R.cache(b, "fp8")
    ensure_built()
    out = torch.zeros(b.q.shape, dtype=torch.float16, device="cuda")
    ws = pkv.decode_workspace(4, 8, 2, 64, 400)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    q, lens = dev(b.q), dev(b.ctx)
    call = pkv.prepare_paged_decode_scored_fp8(out, q, *(dev(x) for x in pools), dev(b.tables),
                                               lens, 400, 0.125, ws, logit_cap=10.0, window=64,
                                               stream=st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    b.q = (b.q.astype(np.float32) * 0.5).astype(np.float16)
    b.ctx = np.asarray([90, 16, 5, 320], np.int32)
    q.copy_(dev(b.q))
    lens.copy_(dev(b.ctx))
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    ref, mass = R.attend(b, kv64, 0.125, cap=10.0, window=64)
    tol = R.tolerance(ref, mass, R.score_error(b, "fp8", 0.125, 10.0, 333, None), 21)
    assert np.all(np.abs(out.cpu().numpy() - ref) <= tol)
