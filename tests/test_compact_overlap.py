"""Compaction writes the new lengths while other warps still read what the call is
given: lengths that overlap it are refused, without a GPU (before any CUDA call)."""
import pytest

import paged_kv_cache_234_gb300 as pkv
from paged_kv_cache_234_gb300 import build as pkv_build

KINDS = ("fp16", "int8", "fp8")
N, T, MB = 5, 40, 6
AT = 1 << 20
# the call's arrays of int32: where they lie, and how many numbers they hold
ARRAYS = dict(kept=(AT, T), kept_lens=(AT + 0x1000, N), starts=(AT + 0x2000, N + 1),
              lens=(AT + 0x3000, N), tables=(AT + 0x4000, N * MB))
APART = AT + 0x8000


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


def call(kind, new, n=N):
    """(More kv heads than a launch can have: nothing is launched, with a GPU or without.)"""
    at = {k: v[0] for k, v in ARRAYS.items()}
    codes = [] if kind == "fp16" else [APART] * 4
    return getattr(pkv.lib(), "pkv_compact_" + kind)(
        APART, APART, *codes, 16, at["kept"], at["kept_lens"], new, at["starts"], at["lens"],
        at["tables"], MB, T, n, (1 << 31) - 1, 64, 16, None, None)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("name", ARRAYS)
def test_lengths_over_an_array_of_the_call(kind, name):
    at, count = ARRAYS[name]
    for number in {0, 1, count - 1, 1 - N, -1}:
        assert call(kind, at + 4 * number) == pkv.PKV_ERR_INVALID_ARG, number


@pytest.mark.parametrize("kind", KINDS)
def test_lengths_beside_the_arrays_are_taken(kind):
    behind = (pkv.PKV_ERR_UNSUPPORTED, pkv.PKV_ERR_CUDA)   # (the second without a GPU)
    for at, count in ARRAYS.values():
        assert call(kind, at - 4 * N) in behind and call(kind, at + 4 * count) in behind
    # without sequences there is nothing that could overlap
    assert call(kind, ARRAYS["kept"][0], n=0) == pkv.PKV_OK
    assert call(kind, None) in behind
