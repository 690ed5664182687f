"""Sequences whose rows do not lie in the batch are reported, wherever they
would begin."""
import numpy as np
import pytest

import paged_kv_cache_234_gb300 as pkv
import serving_reference as R
import test_gpu_prefill as P
import test_gpu_rope_append as A

pytestmark = pytest.mark.gpu

STARTS = {
    "behind": [0, 8, 12, 12],        # sequence 1 begins behind the 8 rows
    "far": [0, 8, 100, 2 ** 31 - 1],
    "backwards": [0, 8, 4, 4],       # sequence 1 has -4 rows
    "before": [0, 8, 8, -5],
}


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("starts", STARTS)
def test_append(kind, starts):
    b = R.make(100, [8, 0, 0], [20, 30, 40], 8, 2, 64, nan_tail=False)
    tab, qkv = A.table(64, 64), A.qkv_of(b, 100, 8)
    r = A.Run(b, kind, qkv, tab, starts=np.asarray(STARTS[starts], np.int32))()
    assert int(r.status.item()) == pkv.PKV_DEV_BAD_CTX
    r.check(*R.rope_append(b, qkv, tab, None, None, False, (b.k, b.v)))


@pytest.mark.parametrize("kind,dim", [("fp16", 64), ("fp16", 128), ("int8", 64)])
@pytest.mark.parametrize("cap", [0.0, 9.0])
@pytest.mark.parametrize("starts", STARTS)
def test_prefill(kind, dim, cap, starts):
    b = R.make(101, [8, 0, 0], [20, 30, 40], 8, 2, dim)
    pools, kv64 = R.cache(b, kind)
    got, status = P.Run(b, kind, pools, starts=np.asarray(STARTS[starts], np.int32), cap=cap)()
    assert status == pkv.PKV_DEV_BAD_CTX
    ref, mass = R.attend(b, kv64, dim ** -0.5, cap=cap)
    o = dict(slopes=None, prefix=None, cap=cap)
    assert np.all(np.abs(got - ref) <= P.bound(b, kind, o, ref, mass))


@pytest.mark.parametrize("kind", ["fp16", "int8"])
def test_many_sequences_with_one_bad_one(kind):
    # more than the threads that look at them take at once
    n = 700
    b = R.make(102, [1] * n, [5] * n, 2, 1, 64, nan_tail=False)
    tab, qkv = A.table(8, 64), A.qkv_of(b, 102, n)
    for at in (None, 0, 333, n - 1):
        lens = b.ctx.copy()
        if at is not None:
            lens[at] = 0
        want = 0 if at is None else pkv.PKV_DEV_BAD_CTX
        r = A.Run(b, kind, qkv, tab, lens=lens)()
        assert int(r.status.item()) == want
        pools, _ = R.cache(b, kind)
        _, status = P.Run(b, kind, pools, lens=lens, max_ctx=5)()
        assert status == want


def test_sequences_without_rows_are_not_reported():
    # whatever their lengths say
    b = R.make(103, [4, 0, 0], [20, 30, 40], 8, 2, 64, nan_tail=False)
    lens = np.asarray([20, 10 ** 6, -3], np.int32)
    r = A.Run(b, "fp16", A.qkv_of(b, 103, 4), A.table(64, 64), lens=lens)()
    assert int(r.status.item()) == 0
    _, status = P.Run(b, "fp16", R.cache(b, "fp16")[0], lens=lens, max_ctx=40)()
    assert status == 0
