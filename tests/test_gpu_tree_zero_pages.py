"""Tree attention with few rows over code caches whose pages of V have scales far
apart, zero among them (what the quantizer gives a tile of zeros), under a bias that
lifts a tile's scores far above the references that the tiles before left."""
import numpy as np
import pytest

import serving_reference as R
import tree_reference as T
from test_gpu_tree import Run, expand

pytestmark = pytest.mark.gpu


def batch(dim, small):
    """Eight sequences of 400 keys with a page of V small at every place in the second
    tile of keys, and eight whose trees begin in such a page, the last tile's."""
    n = 6
    ctx = [400] * 8 + [128 + 16 * (p + 1) + 3 for p in range(8)]
    b = R.make(33, [n] * 16, ctx, 64, 64, dim, nan_tail=False)
    for s in range(16):
        blk = b.tables[s, 8 + s % 8]
        b.v[blk] = (b.v[blk].astype(np.float32) * small).astype(np.float16)
    return b


# 0: scale 0; else the smallest values of fp16, with a scale of 2^-24 / 127 or 2^-24 / 448
@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("small", [0.0, 2.0 ** -26], ids=["zero", "least"])
@pytest.mark.parametrize("slopes", [(0.3, 1.3), (1.3, 8.0)], ids=["usual", "steep"])
def test_small_pages_under_a_bias(kind, dim, small, slopes):
    b = batch(dim, small)
    pools, kv64 = R.cache(b, kind)
    parents = T.trees(6, b.q_lens, "roots")
    o = dict(slopes=np.linspace(*slopes, b.heads).astype(np.float32))
    got, status = Run(b, kind, pools, parents, **o)()
    ref, mass = T.attend(b, parents, kv64, dim ** -0.5, **o)
    assert status == 0
    assert np.all(np.isfinite(got))
    # what test_scales_far_apart allows: of 400 keys each a product p times V scale below
    # 2^-20 of the row's largest, rounded by 2^-31 of that, times a code; `mass` holds the
    # largest times a code that is 1 at least
    extra = 400 * 2.0 ** -31 * (448 if kind == "fp8" else 127) * mass.max(-1, keepdims=True)
    assert np.all(np.abs(got - ref) <= T.bound(b, o, ref, mass, dim ** -0.5) + extra)
