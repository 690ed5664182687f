"""Tree attention: bounds on the trees that no tree keeps to."""
import numpy as np
import pytest

import paged_kv_cache_234_gb300 as pkv
import serving_reference as R
import tree_reference as T
from test_gpu_tree import Run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("heads,kv", [(4, 2), (32, 1), (33, 1), (40, 1), (64, 1), (65, 1), (300, 1)])
def test_a_bound_of_no_rows(kind, heads, kv):
    # every tree is above it: reported, and zeros, whatever the heads
    b = R.make(34, [3, 0, 1], [40, 20, 9], heads, kv, 64, extra_rows=2)
    pools, _ = R.cache(b, kind)
    got, status = Run(b, kind, pools, T.trees(4, b.q_lens), max_tree=0)()
    assert status == pkv.PKV_DEV_BAD_CTX
    assert np.all(got[:4] == 0) and np.all(got[4:] == 7.0)
