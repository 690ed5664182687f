"""Rotation of a ragged batch on its way into the paged cache, on the GPU: the
queries, pools, codes and scales equal the fp32 steps of the definition (each
product and sum rounded, no fused multiply-add; scale = amax times the fp32
reciprocal of the largest code) bit for bit, the rotated values are within
their roundings of the 64-bit rotation, and the codes stand next to those of
the plain quantizer."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_234_gb300 as pkv
import serving_reference as R
from gpu_common import dev, ensure_built

pytestmark = pytest.mark.gpu


def table(positions, rot):
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(positions)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def qkv_of(b, seed, t):
    rng = np.random.default_rng(seed + 1000)
    return rng.standard_normal((t, b.heads + 2 * b.kv_heads, b.dim),
                               dtype=np.float32).astype(np.float16)


class Run:
    """The call's buffers on the GPU, and the call."""

    def __init__(self, b, kind, qkv, tab, positions=None, axis=None, interleaved=False,
                 tables=None, lens=None, starts=None, stream=None):
        ensure_built()
        self.b, self.kind = b, kind
        self.q_out = torch.full((qkv.shape[0], b.heads, b.dim), 7.0, dtype=torch.float16,
                                device="cuda")
        self.k, self.v = dev(b.k), dev(b.v)
        self.codes = []
        if kind != "fp16":
            quant = oracle.quantize_fp8 if kind == "fp8" else oracle.quantize
            (kc, ks), (vc, vs) = quant(b.k), quant(b.v)
            self.codes = [dev(kc), dev(vc), dev(ks), dev(vs)]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        x = dev(qkv)
        self.x = x
        h, hk = b.heads, b.kv_heads
        self.args = (self.q_out, self.k, self.v, *self.codes, x[:, :h], x[:, h:h + hk],
                     x[:, h + hk:], dev(tab), dev(b.starts if starts is None else starts),
                     dev(b.ctx if lens is None else lens),
                     dev(b.tables if tables is None else tables))
        self.kw = dict(rope_positions=None if positions is None else dev(positions),
                       axis_of_pair=axis, interleaved=interleaved, dev_status=self.status,
                       stream=stream)

    def __call__(self):
        getattr(pkv, "pkv_rope_append_" + self.kind)(*self.args, **self.kw)
        torch.cuda.synchronize()
        return self

    def check(self, q_out, k, v, written, rows=None):
        rows = slice(None) if rows is None else rows
        got = self.q_out.cpu().numpy()
        assert np.array_equal(got[rows].view(np.uint16), q_out[rows].view(np.uint16))
        for g, want in ((self.k, k), (self.v, v)):
            assert np.array_equal(g.cpu().numpy().view(np.uint16), want.view(np.uint16))
        if self.kind != "fp16":
            quant = oracle.quantize_fp8 if self.kind == "fp8" else oracle.quantize
            for x, pool, old in ((0, k, self.b.k), (1, v, self.b.v)):
                codes, scales = quant(old)
                codes[written], scales[written] = R.quantize(pool[written], self.kind)
                assert np.array_equal(self.codes[x].cpu().numpy(), codes)
                assert np.array_equal(self.codes[2 + x].cpu().numpy().view(np.uint32),
                                      scales.view(np.uint32))


SHAPES = [
    # q_lens, ctx, heads, kv_heads, dim, rot
    ([1], [1], 8, 2, 64, 64),                            # one token of an empty cache
    ([1] * 7, [1, 2, 16, 17, 31, 32, 33], 32, 8, 128, 128),   # a decode step
    ([5, 0, 16, 1, 33, 0], [5, 40, 32, 77, 33, 0], 14, 2, 64, 32),  # empty ones, half rotated
    ([17, 31, 18], [17, 46, 50], 7, 1, 128, 16),         # the smallest rotation
    ([100, 250], [300, 250], 4, 4, 128, 64),             # MHA
    ([2] * 70, [3 + i for i in range(70)], 3, 1, 64, 64),  # more sequences than a warp
]


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_bit_exact(kind, interleaved, shape):
    q_lens, ctx, heads, kv, dim, rot = SHAPES[shape]
    b = R.make(shape, q_lens, ctx, heads, kv, dim, nan_tail=False)
    tab = table(max(ctx) + 1, rot)
    qkv = qkv_of(b, shape, int(sum(q_lens)))
    r = Run(b, kind, qkv, tab, interleaved=interleaved)()
    r.check(*R.rope_append(b, qkv, tab, None, None, interleaved, (b.k, b.v)))
    assert int(r.status.item()) == 0


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes,dim,rot", [(1, 128, 128), (3, 128, 128), (3, 64, 32), (4, 64, 64)])
def test_several_axes(kind, interleaved, axes, dim, rot):
    b = R.make(50 + axes, [37, 20, 1], [50, 20, 90], 6, 2, dim, nan_tail=False)
    tab = table(64, rot)
    rng = np.random.default_rng(axes)
    positions = rng.integers(0, 64, (axes, 58)).astype(np.int32)
    axis = rng.integers(0, axes, rot // 2).astype(np.uint8)
    qkv = qkv_of(b, axes, 58)
    r = Run(b, kind, qkv, tab, positions, axis, interleaved)()
    r.check(*R.rope_append(b, qkv, tab, positions, axis, interleaved, (b.k, b.v)))
    assert int(r.status.item()) == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_against_the_64_bit_rotation(interleaved):
    # far positions: the table is fp32 (half a step 2^-25 of values up to 1),
    # each output has two products and a sum in fp32 (3 * 2^-24 of |a| + |b|)
    # and the fp16 rounding (2^-11 of the value, 2^-25 below the normals)
    b = R.make(60, [40], [200040], 4, 2, 128, nan_tail=False)
    positions = np.arange(200000, 200040, dtype=np.int32)
    rot = 128
    tab = pkv.rope_table(200040, rot).cpu().numpy()
    qkv = qkv_of(b, 60, 40)
    r = Run(b, "fp16", qkv, tab, positions, None, interleaved)()
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = positions[:, None, None] * f
    x = qkv[:, :4].astype(np.float64)
    lo, hi = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :64], x[..., 64:])
    ya, yb = lo * np.cos(a) - hi * np.sin(a), hi * np.cos(a) + lo * np.sin(a)
    want = np.stack([ya, yb], -1).reshape(x.shape) if interleaved else np.concatenate([ya, yb], -1)
    size = np.abs(lo) + np.abs(hi)
    size = np.stack([size, size], -1).reshape(x.shape) if interleaved else \
        np.concatenate([size, size], -1)
    # (the fp64 angle itself: positions * f rounded, 200040 * 2^-53, nothing)
    tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + (2.0 ** -25 + 3 * 2.0 ** -24) * 1.001 * size
    assert np.all(np.abs(r.q_out.cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_codes_next_to_the_plain_quantizers(kind):
    # With S = amax / most exactly: the plain quantizers' scale is S within
    # 2^-24 (one rounding), this one S within 2^-23 (the constant's and the
    # product's), so they are 1.5 * 2^-23 apart at most (up to 2^-46), and both
    # fp32 quotients lie within 2^-23 + 2^-24 < 2^-22 of x / S.  Two codes that
    # differ are therefore neighbours, with their midpoint within 2^-22 of it.
    b = R.make(65, [200], [200], 4, 2, 128, nan_tail=False)
    qkv = qkv_of(b, 65, 200)
    r = Run(b, kind, qkv, table(200, 128))()
    quant = oracle.quantize_fp8 if kind == "fp8" else oracle.quantize
    value = R.e4m3 if kind == "fp8" else (lambda c: c.astype(np.float64))
    most = 448.0 if kind == "fp8" else 127.0
    for x, pool in ((0, r.k), (1, r.v)):
        tiles = pool.cpu().numpy()[b.used].astype(np.float64)
        codes, scales = (a[b.used] for a in quant(pool.cpu().numpy()))
        got_c, got_s = r.codes[x].cpu().numpy()[b.used], r.codes[2 + x].cpu().numpy()[b.used]
        assert np.all(np.abs(got_s / scales.astype(np.float64) - 1) <= 1.51 * 2.0 ** -23)
        exact = tiles / (np.abs(tiles).max((2, 3), keepdims=True) / most)
        differ = got_c != codes
        mid = (value(got_c) + value(codes))[differ] / 2
        assert np.all(np.abs(got_c[differ].astype(np.int64) - codes[differ].astype(np.int64)) == 1)
        assert np.all(np.abs(exact[differ] - mid) <= 2.0 ** -22 * np.abs(mid))


@pytest.mark.parametrize("kind", ["fp16", "int8"])
def test_rows_behind_the_last_sequence_are_left_alone(kind):
    b = R.make(70, [3, 4], [20, 4], 8, 2, 64, nan_tail=False)
    tab, qkv = table(32, 64), qkv_of(b, 70, 12)
    r = Run(b, kind, qkv, tab)()
    want = R.rope_append(b, qkv, tab, None, None, False, (b.k, b.v))
    r.check(*want, rows=slice(0, 7))
    assert torch.all(r.q_out[7:] == 7.0)
    assert int(r.status.item()) == 0


@pytest.mark.parametrize("kind", ["fp16", "fp8"])
def test_bad_data_is_reported_and_writes_nothing(kind):
    b = R.make(80, [3, 20, 4, 2], [20, 30, 4, 40], 8, 2, 64, nan_tail=False)
    tab, qkv = table(39, 64), qkv_of(b, 80, 29)   # position 39 of the last one is not in the table
    tables, lens = b.tables.copy(), b.ctx.copy()
    tables[1, 1] = b.k.shape[0]                   # the page of tokens 16 .. 29 of sequence 1
    lens[2] = 3                                   # four new tokens, three cached
    r = Run(b, kind, qkv, tab, tables=tables, lens=lens)()
    # what is left of the batch: sequence 0, tokens 10 .. 15 of sequence 1 and
    # the first token of sequence 3 are appended
    q, k, v, _ = R.rope_append(b, qkv, np.concatenate([tab, tab[:1]]), None, None, False,
                               (b.k, b.v))
    bad1 = b.tables[1, 1]
    k[bad1], v[bad1] = b.k[bad1], b.v[bad1]
    for pool, old in ((k, b.k), (v, b.v)):
        pool[b.tables[2, 0]] = old[b.tables[2, 0]]
        pool[b.tables[3, 39 // 16], :, 39 % 16] = old[b.tables[3, 39 // 16], :, 39 % 16]
    q[23:27] = 0
    q[28] = 0
    written = np.asarray([b.tables[0, 1], b.tables[1, 0], b.tables[3, 2]])
    r.check(q, k, v, written)
    assert int(r.status.item()) == \
        pkv.PKV_DEV_BAD_CTX | pkv.PKV_DEV_BAD_BLOCK | pkv.PKV_DEV_BAD_POS


@pytest.mark.parametrize("start1", [-5, 2, 40])
def test_bad_row_ranges_stay_inside_the_batch(start1):
    # rows that begin before or end behind the array, or run backwards: every
    # access stays inside; where the starts only shift, sequence 2 is served
    b = R.make(85, [4, 4, 4], [20, 30, 40], 8, 2, 64, nan_tail=False)
    starts = np.asarray([0, start1, 8, 12], np.int32)
    r = Run(b, "int8", qkv_of(b, 85, 12), table(64, 64), starts=starts)()
    q, _, _, _ = R.rope_append(b, qkv_of(b, 85, 12), table(64, 64), None, None, False, (b.k, b.v))
    if start1 == 2:
        assert np.array_equal(r.q_out.cpu().numpy()[8:12], q[8:12])


def test_queries_in_place():
    b = R.make(90, [9, 2], [30, 2], 8, 2, 128, nan_tail=False)
    tab, qkv = table(32, 128), qkv_of(b, 90, 11)
    want = R.rope_append(b, qkv, tab, None, None, False, (b.k, b.v))
    ensure_built()
    q = dev(qkv[:, :8])
    k, v = dev(b.k), dev(b.v)
    pkv.pkv_rope_append_fp16(q, k, v, q, dev(qkv[:, 8:10]), dev(qkv[:, 10:]), dev(tab),
                             dev(b.starts), dev(b.ctx), dev(b.tables))
    assert np.array_equal(q.cpu().numpy().view(np.uint16), want[0].view(np.uint16))
    assert np.array_equal(k.cpu().numpy().view(np.uint16), want[1].view(np.uint16))


@pytest.mark.parametrize("kind", ["fp16", "int8"])
def test_captured_and_replayed_on_another_stream(kind):
    b = R.make(95, [9, 2, 40], [30, 2, 41], 8, 2, 64, nan_tail=False)
    tab, qkv = table(64, 64), qkv_of(b, 95, 51)
    st = torch.cuda.Stream()
    r = Run(b, kind, qkv, tab, stream=st)
    st.wait_stream(torch.cuda.current_stream())
    call = getattr(pkv, "prepare_rope_append_" + kind)(*r.args, **r.kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    fresh = qkv_of(b, 96, 51)
    r.x.copy_(dev(fresh))
    r.kw.pop("stream")
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    r.check(*R.rope_append(b, fresh, tab, None, None, False, (b.k, b.v)))
