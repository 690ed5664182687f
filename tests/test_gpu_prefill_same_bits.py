"""The results of the prefill are those of the batch's own rows and keys, to the
last bit: whatever lies in rows that belong to nobody, in slots that no row
sees, and in shared memory from calls before."""
import numpy as np
import pytest
import torch

import serving_reference as R
from test_gpu_prefill import Run, expand

pytestmark = pytest.mark.gpu

OPTIONS = {"plain": {}, "cap": dict(cap=20.0), "all": dict(cap=20.0, bias=True, window=100, prefix=5)}


def garbage(b, kind, pools, value):
    """The pools with all slots behind the last tokens, and all blocks of no
    sequence, set to a value (codes: to a byte)."""
    pools = [x.copy() for x in pools]
    byte = {0.0: 0, 30000.0: 0x7e, np.nan: 0x7f if kind == "fp8" else 0x81}[value]
    free = np.setdiff1d(np.arange(b.k.shape[0]), b.used)
    for x in pools[:2]:
        put = value if kind == "fp16" else np.asarray(byte, np.uint8).view(x.dtype)[()]
        x[free] = put
        for s in range(b.ctx.size):
            if b.ctx[s] % R.BS:
                x[b.tables[s, b.ctx[s] // R.BS], :, b.ctx[s] % R.BS:] = put
    return pools


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("heads,kv,dim", [(7, 1, 128), (3, 3, 64), (12, 4, 64)])
@pytest.mark.parametrize("option", OPTIONS)
def test_other_rows_and_slots_have_no_say(kind, heads, kv, dim, option):
    # 7 heads of a kv head: 36 tokens are 252 of an item's 256 rows
    b = R.make(20, [33, 5, 80, 1], [233, 77, 90, 145], heads, kv, dim, extra_rows=50,
               nan_tail=False)
    rows = int(b.starts[-1])
    pools, _ = R.cache(b, kind)
    o = expand(b, OPTIONS[option])
    first = None
    for value in (0.0, 30000.0, np.nan):
        b.q[rows:] = value
        got, status = Run(b, kind, garbage(b, kind, pools, value), **o)()
        assert status == 0
        # what the next call finds in shared memory
        noise = R.make(21, [40] * 40, [300] * 40, heads, kv, dim, nan_tail=False, q_std=50.0)
        Run(noise, kind, R.cache(noise, kind)[0])()
        again, _ = Run(b, kind, garbage(b, kind, pools, value), **o)()
        first = got[:rows] if first is None else first
        assert np.array_equal(got[:rows], first), value
        assert np.array_equal(again[:rows], first), value


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("option", ["cap", "all"])
def test_capped_calls_repeat_themselves(kind, option):
    # several items for an SM, in an order that differs from call to call
    b = R.make(22, [30] * 60, [300] * 60, 14, 14, 128, nan_tail=False)
    r = Run(b, kind, R.cache(b, kind)[0], **expand(b, OPTIONS[option]))
    first, _ = r()
    for _ in range(5):
        r.out.fill_(7.0)
        torch.cuda.synchronize()
        assert np.array_equal(r()[0], first)
