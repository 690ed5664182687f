"""Batches without tokens or sequences, without a GPU: nothing is launched, and
the call succeeds although tensors without elements have no address."""
import numpy as np
import pytest
import torch

import paged_kv_cache_234_gb300 as pkv
from paged_kv_cache_234_gb300 import build as pkv_build

KINDS = ("fp16", "int8", "fp8")


@pytest.fixture(autouse=True)
def no_device(monkeypatch):
    # the device checks aside, so that CPU tensors do
    pkv_build.build()
    monkeypatch.setattr(pkv, "_check", lambda *a, **k: None)
    monkeypatch.setattr(pkv, "_same_device", lambda *a: None)
    monkeypatch.setattr(pkv, "_stream", lambda s: None)


class OnCuda(torch.Tensor):
    is_cuda = True


def pools(kind):
    half = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    code = torch.zeros(4, 2, 16, 64, dtype=torch.int8 if kind == "int8" else torch.uint8)
    scale = torch.ones(4, 2)
    return half, (code, code, scale, scale)


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def rows(n, heads):
    return torch.zeros(n, heads, 64, dtype=torch.float16).as_subclass(OnCuda)


@pytest.mark.parametrize("kind", KINDS)
def test_scored_decode(kind):
    half, codes = pools(kind)
    kv = (half, half) if kind == "fp16" else codes
    for name in ("pkv_paged_decode_scored_", "prepare_paged_decode_scored_"):
        r = getattr(pkv, name + kind)(rows(0, 8), rows(0, 8), *kv, ints(0, 3), ints(0), 40, 0.125,
                                      None, logit_cap=5.0, prefix_lens=ints(0))
        if r is not None:
            r()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens,seqs", [(0, 0), (0, 3), (5, 0)])
def test_prefill(kind, tokens, seqs):
    half, codes = pools(kind)
    kv = (half, half) if kind == "fp16" else codes
    for name in ("pkv_paged_prefill_", "prepare_paged_prefill_"):
        r = getattr(pkv, name + kind)(rows(tokens, 8), rows(tokens, 8), *kv, ints(seqs, 3),
                                      ints(seqs + 1), ints(seqs), 40, 0.125, None, window=9,
                                      prefix_lens=ints(seqs))
        if r is not None:
            r()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens,seqs", [(0, 0), (0, 3), (5, 0)])
@pytest.mark.parametrize("axes", [0, 1, 3])
def test_append(kind, tokens, seqs, axes):
    half, codes = pools(kind)
    codes = () if kind == "fp16" else codes
    kw = dict(rope_positions=ints(axes, tokens), axis_of_pair=np.zeros(32, np.uint8)) if axes else {}
    for name in ("pkv_rope_append_", "prepare_rope_append_"):
        r = getattr(pkv, name + kind)(rows(tokens, 8), half, half, *codes, rows(tokens, 8),
                                      rows(tokens, 2), rows(tokens, 2), torch.zeros(32, 64),
                                      ints(seqs + 1), ints(seqs), ints(seqs, 3), **kw)
        if r is not None:
            r()


def test_arrays_with_elements_are_still_required():
    half, _ = pools("fp16")
    fn, args = pkv._prefill("pkv_paged_prefill_fp16", rows(0, 8), rows(0, 8), half, half, None, None,
                            ints(2, 3), ints(3), ints(2), 40, 0.125, None, 0.0, 0, None, None, None,
                            None)
    pkv._invoke(fn, args)
    args[8] = None  # context_lens of two sequences
    with pytest.raises(pkv.PkvError):
        pkv._invoke(fn, args)
