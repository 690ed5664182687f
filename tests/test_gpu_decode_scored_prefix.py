"""Visible prefixes of any 32-bit length in the scored decode: a negative one
counts as 0, one beyond the context as the context."""
import numpy as np
import pytest

import serving_reference as R
from test_gpu_decode_scored import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
def test_prefix_lengths_at_the_ends_of_the_type(kind):
    # windows that begin inside a page: its tokens ahead of them are not seen
    ctx = [333, 200, 95, 333, 120]
    b = R.make(70, [1] * 5, ctx, 8, 2, 64)
    prefix = np.asarray([-2 ** 31, -2 ** 31 + 7, -1, 2 ** 31 - 1, 3], np.int32)
    pools, kv64 = R.cache(b, kind)
    got, status = run(b, kind, pools, window=41, prefix=prefix)
    ref, mass = R.attend(b, kv64, 0.125, window=41, prefix=prefix)
    dz = R.score_error(b, kind, 0.125, 0.0, max(ctx), None)
    assert status == 0
    assert np.all(np.abs(got - ref) <= R.tolerance(ref, mass, dz, 21))
