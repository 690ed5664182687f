"""The prefill kernel's waits: every one is bounded, and none is left out.

When a wait runs out, the kernel sets PKV_DEV_TIMEOUT, every role of the CTA
ends, the copies and products in flight are waited for and the tensor memory is
freed: the call returns, and the next one is right.  A copy that never lands
cannot be made safely, so the debug build (PKV_DEBUG) lets one wait of a role
give up while its copies and products are still on their way, which they then
complete.  The other setting makes every wait of a role begin later: whatever
the others then read must still be ordered behind its write.
"""
import time

import numpy as np
import pytest
import torch

import paged_kv_cache_234_gb300 as pkv
import serving_reference as R
from gpu_common import ensure_built
from test_gpu_prefill import Run, bound, expand
from test_gpu_prefill_scales import attend

pytestmark = pytest.mark.gpu

ROLES = ["rows", "products", "load_k", "load_v", "items", "widen"]


class DebugRun(Run):
    """The call on the debug build."""

    def __call__(self):
        a, k = self.args, self.kw
        kp, vp, *rest = a[2:]
        ks, vs = rest[:2] if self.kind != "fp16" else (None, None)
        rest = rest[0 if self.kind == "fp16" else 2:]
        fn, args = pkv._prefill("pkv_paged_prefill_" + self.kind, a[0], a[1], kp, vp, ks, vs, *rest,
                                k["logit_cap"], k["window"], k["slopes"], k["prefix_lens"],
                                k["dev_status"], None)
        self.status.zero_()
        assert getattr(pkv.debug_lib(), fn)(*args) == pkv.PKV_OK
        torch.cuda.synchronize()  # raises if the context were lost
        return self.out.cpu().numpy().astype(np.float64), int(self.status.item())


def batch(shape, dim):
    if shape == "queue":  # three items for an SM, one after the other
        return R.make(40, [30, 9, 30, 1, 17, 30], [300, 200, 280, 300, 17, 150], 64, 64, dim,
                      nan_tail=False)
    # splits over the keys, both tiles of a split on the same rows
    return R.make(41, [5, 3], [4001, 2500], 4, 1, dim, nan_tail=False)


@pytest.fixture
def setting():
    ensure_built()
    L = pkv.debug_lib()

    def put(give=-1, at=0, slow=-1, ns=0):
        assert L.pkv_debug_set_prefill(give, at, slow, ns) == 0
    put()
    yield put
    put()


CASES = [(kind, dim, shape, option) for kind, dim in (("fp16", 128), ("int8", 128), ("fp8", 64))
         for shape in ("queue", "split") for option in ("plain", "all")]


def make(kind, dim, shape, option):
    b = batch(shape, dim)
    o = expand(b, dict(cap=20.0, bias=True, window=700, prefix=20) if option == "all" else option)
    pools, kv64 = R.cache(b, kind)
    return b, o, kv64, DebugRun(b, kind, pools, **o)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_slow_roles_change_nothing(case, setting):
    # (V loads that begin late found the softmax reading V scales of tiles before)
    kind = case[0]
    b, o, kv64, r = make(*case)
    want, status = r()
    ref, mass = attend(b, kv64, b.dim ** -0.5, **o)
    assert status == 0
    assert np.all(np.abs(want - ref) <= bound(b, kind, o, ref, mass))
    for role in range(5 if kind == "fp16" else 6):
        r.out.fill_(7.0)
        setting(slow=role, ns=20000)
        got, status = r()
        assert status == 0, ROLES[role]
        assert np.array_equal(got, want), ROLES[role]


@pytest.mark.parametrize("role,case", [(role, c) for role in range(6) for c in CASES
                                       if c[0] != "fp16" or ROLES[role] != "widen"],
                         ids=lambda x: ROLES[x] if isinstance(x, int) else "-".join(map(str, x)))
def test_a_wait_that_runs_out(case, role, setting):
    _, _, _, r = make(*case)
    want, status = r()
    assert status == 0
    for at in (0, 1, 2, 3, 4, 6, 8, 11, 15):
        setting(give=role, at=at)
        t0 = time.monotonic()
        _, status = r()
        took = time.monotonic() - t0
        # (a role has at least two waits of an item, later ones depend on it)
        assert status == pkv.PKV_DEV_TIMEOUT if at < 2 else status in (0, pkv.PKV_DEV_TIMEOUT)
        # what is in flight lands at once: no wait behind it runs into its limit
        assert took < 0.5, (at, took)
        setting()
        r.out.fill_(7.0)
        got, status = r()
        assert status == 0
        assert np.array_equal(got, want), at
