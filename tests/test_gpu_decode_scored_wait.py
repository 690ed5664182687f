"""A stage wait of the scored decode that runs out: PKV_DEV_TIMEOUT is set, the
call returns, and the next one is right (see test_gpu_wait_timeout.py for how a
wait is made to run out without a copy that never lands)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_234_gb300 as pkv
import serving_reference as R
from gpu_common import dev, ensure_built

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("launch", ["auto", "persistent"])
@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
def test_a_stage_wait_that_runs_out(kind, launch):
    ensure_built()
    L = pkv.debug_lib()
    b = R.make(110, [1] * 6, [900, 1500, 17, 400, 1300, 777], 8, 2, 128)
    pools, kv64 = R.cache(b, kind)
    out = torch.empty(b.q.shape, dtype=torch.float16, device="cuda")
    ws = pkv.decode_workspace(6, 8, 2, 128, 1500)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    held = [dev(x) for x in pools]
    kv_t = held + [None] * (4 - len(held))
    q, tables, lens = dev(b.q), dev(b.tables), dev(b.ctx)
    fn, args = pkv._scored("pkv_paged_decode_scored_" + kind, out, q, *kv_t, tables, lens, 1500,
                           128 ** -0.5, ws, 0.0, 700, None, None, status, None)
    ref, mass = R.attend(b, kv64, 128 ** -0.5, window=700)
    tol = R.tolerance(ref, mass, R.score_error(b, kind, 128 ** -0.5, 0.0, 1500, None), 21)

    def call(lib):
        status.zero_()
        out.fill_(float("nan"))
        assert getattr(lib, fn)(*args) == pkv.PKV_OK
        torch.cuda.synchronize()  # raises if the context were lost
        return int(status.item())

    cap = 4096 if launch == "persistent" else 0
    try:
        assert L.pkv_set_decode_workers(cap) == 0
        assert L.pkv_debug_set_scored_stage_wait_ns(0) == 0
        assert call(L) & pkv.PKV_DEV_TIMEOUT
        assert L.pkv_debug_set_scored_stage_wait_ns(-1) == 0
        assert L.pkv_debug_scored_flags(1) == 0  # it stayed inside its buffers
        assert call(L) == 0
        assert np.all(np.abs(out.cpu().numpy() - ref) <= tol)
    finally:
        L.pkv_debug_set_scored_stage_wait_ns(-1)
        L.pkv_set_decode_workers(0)
    assert call(pkv.lib()) == 0
    assert np.all(np.abs(out.cpu().numpy() - ref) <= tol)
