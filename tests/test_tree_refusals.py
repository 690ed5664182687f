"""What the operators for trees of drafted tokens refuse, and batches without
tokens or sequences, without a GPU: the C entry points return the documented
status before any CUDA call, the Python binding raises before it reaches them."""
import numpy as np
import pytest
import torch

import paged_kv_cache_234_gb300 as pkv
import tree_reference as T
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


TREE = dict(out=FAKE, query=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, num_blocks=16, tables=FAKE,
            mb=4, starts=FAKE, lens=FAKE, parents=FAKE, max_ctx=64, max_tree=8, t=10, n=2, hq=8,
            hkv=2, d=64, bs=16, scale=0.125, cap=0.0, window=0, slopes=None, prefix=None, ws=FAKE,
            ws_bytes=1 << 40, status=None, stream=None)


@pytest.mark.parametrize("kind", KINDS)
def test_tree(kind):
    order = [n for n in TREE if kind != "fp16" or n not in ("ks", "vs")]

    def c(**kw):
        return call(order, TREE, "pkv_paged_tree_" + kind, **kw)
    for name in ("out", "query", "k", "v", "tables", "starts", "lens", "parents"):
        assert c(**{name: None}) == INVALID
    assert c(cap=-1.0) == c(cap=float("nan")) == c(cap=float("inf")) == INVALID
    assert c(cap=1e-31) == c(cap=1e31) == c(scale=2.5e38) == INVALID
    assert c(window=-1) == c(t=-1) == c(n=-1) == c(hq=7) == c(mb=-1) == c(max_ctx=-1) == INVALID
    assert c(max_tree=-1) == c(num_blocks=0) == c(hkv=0) == INVALID
    assert c(scale=float("nan")) == c(scale=float("-inf")) == INVALID
    assert c(d=96) == c(bs=32) == c(num_blocks=1 << 27) == UNSUPPORTED
    assert c(max_ctx=(1 << 31) - 1) == UNSUPPORTED
    for name in ("slopes", "prefix", "lens", "starts", "tables", "parents", "status"):
        assert c(**{name: FAKE + 2}) == MISALIGNED
    assert c(out=FAKE + 8) == c(k=FAKE + 4) == c(query=FAKE + 2) == MISALIGNED
    need = pkv.pkv_tree_workspace_size(10, 2, 8, 2, 64, 64, 8)
    assert need > 0 and c(ws=None) == c(ws_bytes=need - 1) == WORKSPACE
    assert c(ws=FAKE + 4) == MISALIGNED
    assert c(t=0) == c(n=0) == pkv.PKV_OK
    assert c(t=0, out=None, query=None, parents=None) == pkv.PKV_OK
    if kind != "fp16":
        assert c(ks=None) == INVALID and c(vs=FAKE + 1) == MISALIGNED


ACCEPT = dict(kept=FAKE, lens=FAKE, last=FAKE, tokens=FAKE, targets=FAKE, parents=FAKE,
              starts=FAKE, t=10, n=2, status=None, stream=None)


def test_accept():
    def c(**kw):
        return call(ACCEPT, ACCEPT, "pkv_tree_accept", **kw)
    for name in ("kept", "lens", "last", "tokens", "targets", "parents", "starts"):
        assert c(**{name: None}) == INVALID
        assert c(**{name: FAKE + 2}) == MISALIGNED
    assert c(status=FAKE + 1) == MISALIGNED
    assert c(t=-1) == c(n=-1) == INVALID
    assert c(n=0) == c(n=0, lens=None, last=None) == pkv.PKV_OK


COMPACT = dict(k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, num_blocks=16, kept=FAKE,
               kept_lens=FAKE, new=FAKE + 64, starts=FAKE, lens=FAKE, tables=FAKE, mb=4, t=10, n=2,
               hkv=2, d=64, bs=16, status=None, stream=None)


@pytest.mark.parametrize("kind", KINDS)
def test_compact(kind):
    order = [n for n in COMPACT if kind != "fp16" or n not in ("kc", "vc", "ks", "vs")]

    def c(**kw):
        return call(order, COMPACT, "pkv_compact_" + kind, **kw)
    for name in ("k", "v", "kept", "kept_lens", "starts", "lens", "tables"):
        assert c(**{name: None}) == INVALID
    assert c(new=FAKE) == INVALID            # the lengths themselves
    assert c(t=-1) == c(n=-1) == c(mb=-1) == c(hkv=0) == c(num_blocks=0) == INVALID
    assert c(d=96) == c(bs=8) == c(mb=1 << 28) == UNSUPPORTED
    for name in ("kept", "kept_lens", "new", "starts", "lens", "tables", "status"):
        assert c(**{name: FAKE + 2}) == MISALIGNED
    assert c(k=FAKE + 8) == c(v=FAKE + 2) == MISALIGNED
    assert c(n=0) == pkv.PKV_OK
    if kind != "fp16":
        assert c(kc=None) == c(vs=None) == INVALID
        assert c(vc=FAKE + 8) == c(ks=FAKE + 2) == MISALIGNED


def test_workspace_size():
    # few rows per kv head: for each of 152 pieces two parts of 32 or 64 rows, d values
    # and two numbers each, and 16 bytes that say whose they are
    def expect(rows, d):
        return 152 * (2 * rows * (d + 2) * 4 + 16)
    assert pkv.pkv_tree_workspace_size(64, 8, 8, 8, 128, 512, 8) == expect(32, 128)
    assert pkv.pkv_tree_workspace_size(64, 8, 32, 8, 128, 512, 8) == expect(32, 128)
    assert pkv.pkv_tree_workspace_size(64, 8, 32, 8, 64, 512, 9) == expect(64, 64)
    # a bound above the batch's tokens does not count
    assert pkv.pkv_tree_workspace_size(4, 1, 8, 1, 64, 512, 4096) == expect(32, 64)
    # many rows: two parts of every row for each split of the keys, if there are several
    for tree, heads in ((17, 32), (1, 80 * 8)):
        parts = 2 * 64 * heads * (128 + 2) * 4
        size = pkv.pkv_tree_workspace_size(64, 8, heads, 8, 128, 20000, tree)
        assert size % parts == 0 and 2 <= size // parts <= 32
    # 512 work items: one for every SM three times over
    assert pkv.pkv_tree_workspace_size(64 * 64, 64, 32, 8, 128, 8192, 64) == 0
    assert pkv.pkv_tree_workspace_size(8, 1, 4, 3, 128, 20000, 8) == 0
    assert pkv.pkv_tree_workspace_size(8, 1, 4, 1, 96, 20000, 8) == 0
    assert pkv.pkv_tree_workspace_size(-1, 1, 4, 1, 64, 20000, 8) == 0


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def pools(kind):
    half = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    code = torch.zeros(4, 2, 16, 64, dtype=torch.int8 if kind == "int8" else torch.uint8)
    scale = torch.ones(4, 2)
    return (half, half) if kind == "fp16" else (half, half, code, code, scale, scale)


def make_calls(kind, tokens=2, seqs=2, **other):
    a = dict(parents=ints(tokens), kept=ints(tokens), starts=ints(seqs + 1), lens=ints(seqs),
             kept_lens=ints(seqs), last=ints(seqs), new=ints(seqs), tables=ints(seqs, 2),
             ids=ints(tokens), q=torch.zeros(tokens, 8, 64, dtype=torch.float16),
             out=torch.zeros(tokens, 8, 64, dtype=torch.float16))
    a.update(other)
    p = pools(kind)
    kv = p if kind == "fp16" else p[2:]
    for prefix in ("pkv_", "prepare_"):
        yield lambda: getattr(pkv, prefix + "paged_tree_" + kind)(
            a["out"], a["q"], *kv, a["tables"], a["starts"], a["lens"], a["parents"], 32, 8, 0.125,
            torch.zeros(1 << 16, dtype=torch.uint8))
        yield lambda: getattr(pkv, prefix + "compact_" + kind)(
            *p, a["kept"], a["kept_lens"], a["new"], a["starts"], a["lens"], a["tables"])
        yield lambda: getattr(pkv, prefix + "tree_accept")(
            a["kept"], a["kept_lens"], a["last"], a["ids"], a["ids"], a["parents"], a["starts"])


@pytest.mark.parametrize("kind", KINDS)
def test_cpu_tensors_are_rejected(kind):
    for f in make_calls(kind):
        with pytest.raises(ValueError, match="CUDA tensor"):
            f()


@pytest.fixture
def no_device(monkeypatch):
    # the device checks aside, so that CPU tensors do; nothing is launched
    monkeypatch.setattr(pkv, "_check", lambda *a, **k: None)
    monkeypatch.setattr(pkv, "_same_device", lambda *a: None)
    monkeypatch.setattr(pkv, "_stream", lambda s: None)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens,seqs", [(0, 0), (5, 0)])
def test_batches_without_sequences(kind, tokens, seqs, no_device):
    for f in make_calls(kind, tokens, seqs):
        r = f()
        if r is not None:
            r()


@pytest.mark.parametrize("kind", KINDS)
def test_shapes_are_checked(kind, no_device):
    wrong = dict(parents=(ints(3), (0, 2)), starts=(ints(2), (0, 1, 2)), lens=(ints(1), (0, 1)),
                 tables=(ints(3, 2), (0, 1)), out=(torch.zeros(2, 8, 128), (0,)),
                 kept_lens=(ints(3), (1, 2)), new=(ints(1), (1,)), last=(ints(4), (2,)),
                 ids=(ints(5), (2,)))
    for name, (value, which) in wrong.items():
        calls = list(make_calls(kind, **{name: value}))
        for i in which:
            with pytest.raises(ValueError):
                calls[3 + i]()


def test_the_references_agree_with_each_other():
    # a chain is what the linear drafts' definition says
    import serving_reference as R
    b = R.make(1, [5, 3], [40, 3], 4, 2, 64)
    kv64 = (b.k.astype(np.float64), b.v.astype(np.float64))
    chain = T.trees(0, b.q_lens, "chain")
    o = dict(cap=9.0, window=12, slopes=np.full(4, 0.25, np.float32))
    for got, want in zip(T.attend(b, chain, kv64, 0.1, **o), R.attend(b, kv64, 0.1, **o)):
        assert np.allclose(got, want, rtol=1e-12, atol=0)
    kept, lens, last = T.accept(np.asarray([-1, 0, 0, 2]), np.asarray([9, 5, 5, 6]),
                                np.asarray([5, 7, 6, 8]), [0, 4])
    assert kept.tolist() == [0, 1, -1, -1] and lens.tolist() == [2] and last.tolist() == [7]
