"""Code caches compacted: quotients at the middle of two codes and next to it.

The moved tiles' codes are found without the quantizer's division; what lies close to
the middle of two codes is settled apart. Random tiles hardly come there, so these
hold, for a largest magnitude each, the fp16 values nearest to every middle times the
scale, their neighbours, and where the scale is a power of two the middles themselves."""
import numpy as np
import pytest

import serving_reference as R
from test_gpu_compact import check

pytestmark = pytest.mark.gpu


def middles(kind):
    if kind == "int8":
        return np.arange(127) + 0.5
    codes = R.e4m3(np.arange(0x7f, dtype=np.uint8))   # 0 to 448, rising
    return (codes[1:] + codes[:-1]) / 2


def tile(kind, amax, size, rng):
    """`size` fp16 values, the largest magnitude amax."""
    top = 127.0 if kind == "int8" else 448.0
    scale = np.float32(amax) / np.float32(top)
    x = (middles(kind) * np.float64(scale)).astype(np.float16)
    up, down = np.nextafter(x, np.float16(np.inf)), np.nextafter(x, np.float16(0))
    x = np.concatenate([x, up, down, -x, -up, -down])
    x = x[np.abs(x.astype(np.float64)) <= float(amax)]
    out = np.concatenate([[np.float16(amax)], rng.permutation(x)])[:size]
    return np.concatenate([out, np.zeros(size - out.size, np.float16)])


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("pages", [3, 60, 300])   # a warp, a CTA or a cluster to a chain
def test_values_around_the_middle_of_two_codes(kind, dim, pages):
    # every page moves by one, whole
    n = 16 * (pages + 1)
    b = R.make(35, [n], [n], 2, 2, dim, nan_tail=False)
    rng = np.random.default_rng(pages)
    bits = rng.integers(1, 0x7c00, (2, pages + 4, 2)).astype(np.uint16)
    amax = bits.view(np.float16)                  # subnormal ones among them
    exact = np.float16(127.0 if kind == "int8" else 448.0)
    even = rng.random(amax.shape) < 0.4           # scales that are powers of two
    amax = np.where(even, exact * 2.0 ** rng.integers(-14, 7, amax.shape), amax).astype(np.float16)
    for x, tops in zip((b.k, b.v), amax):
        for blk in range(x.shape[0]):
            for h in range(2):
                x[blk, h] = tile(kind, tops[blk % len(tops), h], 16 * dim, rng).reshape(16, dim)
    kept = np.concatenate([np.arange(16, n), np.full(16, -1)]).astype(np.int32)
    check(b, kind, kept, [n - 16])
