"""What the serving operators refuse, without a GPU: the C entry points return
the documented status before any CUDA call, the Python binding raises before
it reaches the library."""
import numpy as np
import pytest
import torch

import paged_kv_cache_234_gb300 as pkv
from paged_kv_cache_234_gb300 import build as pkv_build

FAKE = 0x10000  # an aligned, never-dereferenced address
KINDS = ("fp16", "int8", "fp8")
INVALID, UNSUPPORTED = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED
MISALIGNED, WORKSPACE = pkv.PKV_ERR_MISALIGNED, pkv.PKV_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


def call(order, base, fn, **kw):
    a = dict(base)
    assert set(kw) <= set(a)
    a.update(kw)
    return getattr(pkv.lib(), fn)(*(a[n] for n in order))


DECODE = dict(out=FAKE, query=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, num_blocks=16, tables=FAKE,
              mb=4, lens=FAKE, max_ctx=64, n=2, hq=8, hkv=2, d=64, bs=16, scale=0.125, cap=0.0,
              window=0, slopes=None, prefix=None, ws=FAKE, ws_bytes=1 << 30, status=None,
              stream=None)


@pytest.mark.parametrize("kind", KINDS)
def test_scored_decode(kind):
    order = [n for n in DECODE if kind != "fp16" or n not in ("ks", "vs")]

    def c(**kw):
        return call(order, DECODE, "pkv_paged_decode_scored_" + kind, **kw)
    for name in ("out", "query", "k", "v", "tables", "lens"):
        assert c(**{name: None}) == INVALID
    assert c(cap=-1.0) == c(cap=float("nan")) == c(cap=float("inf")) == INVALID
    assert c(cap=1e-31) == c(cap=1e31) == c(scale=2.5e38) == INVALID
    assert c(window=-1) == c(n=-1) == c(hq=7) == c(num_blocks=0) == INVALID
    assert c(scale=float("nan")) == c(scale=float("inf")) == INVALID
    assert c(d=96) == c(bs=32) == c(n=9000) == UNSUPPORTED
    for name in ("slopes", "prefix", "lens", "tables", "status"):
        assert c(**{name: FAKE + 2}) == MISALIGNED
    assert c(out=FAKE + 8) == c(k=FAKE + 4) == MISALIGNED
    assert c(ws=None) == c(ws_bytes=100) == WORKSPACE
    assert c(n=0) == pkv.PKV_OK
    if kind != "fp16":
        assert c(ks=None) == INVALID


ROPE = dict(q_out=FAKE, k_cache=FAKE, v_cache=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE,
            num_blocks=16, q=FAKE, qs=512, k=FAKE, k_stride=128, v=FAKE, v_stride=128, tab=FAKE,
            max_pos=64, rot=64, inter=0, pos=None, axes=1, axis=None, starts=FAKE, lens=FAKE,
            tables=FAKE, mb=4, t=10, n=2, hq=8, hkv=2, d=64, bs=16, status=None, stream=None)


@pytest.mark.parametrize("kind", KINDS)
def test_rope_append(kind):
    order = [n for n in ROPE if kind != "fp16" or n not in ("kc", "vc", "ks", "vs")]
    axis = np.zeros(32, np.uint8)

    def c(**kw):
        return call(order, ROPE, "pkv_rope_append_" + kind, **kw)
    for name in ("q_out", "k_cache", "v_cache", "q", "k", "v", "tab", "starts", "lens", "tables"):
        assert c(**{name: None}) == INVALID
    assert c(axes=0) == c(max_pos=0) == c(rot=0) == c(rot=80) == c(t=-1) == c(n=-1) == INVALID
    assert c(axes=3) == c(axes=3, pos=FAKE) == c(axes=3, axis=axis.ctypes.data) == INVALID
    axis[31] = 3
    assert c(axes=3, pos=FAKE, axis=axis.ctypes.data) == INVALID
    assert c(qs=504) == c(k_stride=120) == c(v_stride=0) == INVALID
    assert c(rot=24) == c(rot=8) == c(d=96, rot=32) == c(bs=8) == c(mb=1 << 28) == UNSUPPORTED
    assert c(qs=516) == c(k_stride=129) == c(v=FAKE + 8) == c(q_out=FAKE + 2) == MISALIGNED
    assert c(tab=FAKE + 4) == c(starts=FAKE + 1) == c(status=FAKE + 2) == MISALIGNED
    assert c(t=0) == c(n=0) == pkv.PKV_OK
    if kind != "fp16":
        assert c(kc=None) == c(vs=None) == INVALID
        assert c(vc=FAKE + 8) == c(ks=FAKE + 2) == MISALIGNED


PREFILL = dict(out=FAKE, query=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, num_blocks=16, tables=FAKE,
               mb=4, starts=FAKE, lens=FAKE, max_ctx=64, t=10, n=2, hq=8, hkv=2, d=64, bs=16,
               scale=0.125, cap=0.0, window=0, slopes=None, prefix=None, ws=FAKE,
               ws_bytes=1 << 30, status=None, stream=None)


@pytest.mark.parametrize("kind", KINDS)
def test_prefill(kind):
    order = [n for n in PREFILL if kind != "fp16" or n not in ("ks", "vs")]

    def c(**kw):
        return call(order, PREFILL, "pkv_paged_prefill_" + kind, **kw)
    for name in ("out", "query", "k", "v", "tables", "starts", "lens"):
        assert c(**{name: None}) == INVALID
    assert c(cap=-1.0) == c(cap=float("nan")) == c(cap=float("inf")) == INVALID
    assert c(cap=1e-31) == c(cap=1e31) == c(scale=2.5e38) == INVALID
    assert c(window=-1) == c(t=-1) == c(n=-1) == c(hq=7) == c(mb=-1) == c(max_ctx=-1) == INVALID
    assert c(scale=float("nan")) == c(scale=float("-inf")) == INVALID
    assert c(d=96) == c(bs=32) == c(num_blocks=1 << 27) == c(t=1 << 30) == UNSUPPORTED
    assert c(max_ctx=(1 << 31) - 1, ws_bytes=1 << 40) == UNSUPPORTED
    for name in ("slopes", "prefix", "lens", "starts", "tables", "status"):
        assert c(**{name: FAKE + 2}) == MISALIGNED
    assert c(out=FAKE + 8) == c(k=FAKE + 4) == c(query=FAKE + 2) == MISALIGNED
    need = pkv.pkv_prefill_workspace_size(10, 2, 8, 2, 64, 6400)
    assert need > 0
    assert c(max_ctx=6400, ws=None) == c(max_ctx=6400, ws_bytes=need - 1) == WORKSPACE
    assert c(max_ctx=6400, ws=FAKE + 4) == MISALIGNED
    assert c(t=0) == c(n=0) == pkv.PKV_OK
    if kind != "fp16":
        assert c(ks=None) == INVALID and c(vs=FAKE + 1) == MISALIGNED


def test_prefill_workspace_size():
    # 2 splits * rows * (head_dim + 2) floats; none where the items fill the GPU
    one = 2 * 8 * 4 * (128 + 2) * 4
    size = pkv.pkv_prefill_workspace_size(8, 1, 4, 1, 128, 20000)
    assert size % one == 0 and 2 <= size // one <= 64
    assert pkv.pkv_prefill_workspace_size(65536, 16, 32, 8, 128, 4096) == 0
    assert pkv.pkv_prefill_workspace_size(8, 1, 4, 3, 128, 20000) == 0
    assert pkv.pkv_prefill_workspace_size(8, 1, 4, 1, 96, 20000) == 0
    assert pkv.pkv_prefill_workspace_size(0, 0, 4, 1, 64, 20000) == 0


def tensors():
    return dict(out=torch.zeros(2, 8, 64, dtype=torch.float16),
                q=torch.zeros(2, 8, 64, dtype=torch.float16),
                kv=torch.zeros(2, 2, 64, dtype=torch.float16),
                pool=torch.zeros(4, 2, 16, 64, dtype=torch.float16),
                tab=torch.zeros(32, 64), bt=torch.zeros(2, 2, dtype=torch.int32),
                cl=torch.ones(2, dtype=torch.int32), starts=torch.zeros(3, dtype=torch.int32),
                ws=torch.zeros(1024, dtype=torch.uint8))


CPU_CALLS = [
    lambda a: pkv.pkv_paged_decode_scored_fp16(a["out"], a["q"], a["pool"], a["pool"], a["bt"],
                                               a["cl"], 32, 0.125, a["ws"], logit_cap=1.0),
    lambda a: pkv.prepare_paged_decode_scored_fp16(a["out"], a["q"], a["pool"], a["pool"],
                                                   a["bt"], a["cl"], 32, 0.125, a["ws"]),
    lambda a: pkv.pkv_rope_append_fp16(a["out"], a["pool"], a["pool"], a["q"], a["kv"], a["kv"],
                                       a["tab"], a["starts"], a["cl"], a["bt"]),
    lambda a: pkv.prepare_rope_append_fp16(a["out"], a["pool"], a["pool"], a["q"], a["kv"],
                                           a["kv"], a["tab"], a["starts"], a["cl"], a["bt"]),
    lambda a: pkv.pkv_paged_prefill_fp16(a["out"], a["q"], a["pool"], a["pool"], a["bt"],
                                         a["starts"], a["cl"], 32, 0.125, a["ws"]),
    lambda a: pkv.prepare_paged_prefill_fp16(a["out"], a["q"], a["pool"], a["pool"], a["bt"],
                                             a["starts"], a["cl"], 32, 0.125, a["ws"]),
]


@pytest.mark.parametrize("i", range(len(CPU_CALLS)))
def test_cpu_tensors_are_rejected(i):
    with pytest.raises(ValueError, match="CUDA tensor"):
        CPU_CALLS[i](tensors())


def test_rope_table_is_rounded_once():
    tab = pkv.rope_table(70, 32, device="cpu").numpy()
    f = 10000.0 ** (-np.arange(0, 32, 2) / 32)
    a = np.arange(70)[:, None] * f
    want = np.concatenate([np.cos(a), np.sin(a)], 1)
    # half a step of fp32, and one of fp64 of the angle (up to 70 * 2^-52)
    assert tab.dtype == np.float32 and np.all(np.abs(tab - want) <= 2.0 ** -25 + 2.0 ** -44)
    own = pkv.rope_table(70, 32, inv_freq=f, device="cpu").numpy()
    assert np.max(np.abs(own - tab)) <= 2.0 ** -23
    with pytest.raises(ValueError):
        pkv.rope_table(70, 32, inv_freq=f[:3], device="cpu")


@pytest.mark.parametrize("kind", KINDS)
def test_scored_decode_shapes_are_checked(kind, monkeypatch):
    # the device checks aside, so that CPU tensors do; nothing is launched
    monkeypatch.setattr(pkv, "_check", lambda *a, **k: None)
    monkeypatch.setattr(pkv, "_same_device", lambda *a: None)
    monkeypatch.setattr(pkv, "_stream", lambda s: None)
    codes = {"fp16": torch.float16, "int8": torch.int8, "fp8": torch.uint8}[kind]

    def prepare(dim=64, rows=2, table_dims=2):
        a = tensors()
        pool = torch.zeros(4, 2, 16, dim, dtype=codes)
        scales = () if kind == "fp16" else (torch.ones(4, 2), torch.ones(4, 2))
        bt = torch.zeros(rows, 2, dtype=torch.int32)
        return getattr(pkv, "prepare_paged_decode_scored_" + kind)(
            a["out"], a["q"], pool, pool, *scales, bt if table_dims == 2 else bt[0], a["cl"], 32,
            0.125, a["ws"])
    prepare()
    for dim in (32, 128):
        with pytest.raises(ValueError, match="pool"):
            prepare(dim=dim)
    for kw in (dict(rows=1), dict(rows=3), dict(table_dims=1)):
        with pytest.raises(ValueError, match="block_tables"):
            prepare(**kw)
