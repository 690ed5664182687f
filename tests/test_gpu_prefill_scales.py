"""Attention of ragged batches over code caches whose V scales differ from page
to page, on the GPU, against the 64-bit definition."""
import numpy as np
import pytest

import serving_reference as R
from test_gpu_prefill import Run, bound, expand

pytestmark = pytest.mark.gpu


def attend(b, kv64, scale, top=None, **o):
    """R.attend with the rows of a (sequence, head) at once.  top [T][Hq] gets the
    largest |V| of the keys whose probability is above 2^-40 of the row's
    largest, and of the pages these are in as far as the row sees them."""
    k64, v64 = kv64
    out, mass = np.zeros(b.q.shape), np.zeros(b.q.shape)
    for s in range(b.ctx.size):
        c, n, r = int(b.ctx[s]), int(b.q_lens[s]), int(b.starts[s])
        blk = b.tables[s, :-(-c // R.BS)]
        i, t = np.arange(c - n, c)[:, None], np.arange(c)[None]
        pre = 0 if o["prefix"] is None else int(o["prefix"][s])
        seen = R.visible(i, t, o.get("window", 0), pre)
        for h in range(b.heads):
            kk = k64[blk, h // b.group].reshape(-1, b.dim)[:c]
            vv = v64[blk, h // b.group].reshape(-1, b.dim)[:c]
            z = b.q[r:r + n, h].astype(np.float64) @ kk.T * scale
            if o.get("cap"):
                z = o["cap"] * np.tanh(z / o["cap"])
            if o["slopes"] is not None:
                z = z - float(o["slopes"][h]) * np.abs(i - t)
            z = np.where(seen, z, -np.inf)
            p = np.exp(z - z.max(1, keepdims=True))
            if top is not None:
                big = np.where(seen, np.abs(vv).max(1)[None], 0.0)
                for page in range(-(-c // R.BS)):
                    x = big[:, page * R.BS:(page + 1) * R.BS]
                    x[:] = x.max(1, keepdims=True)
                top[r:r + n, h] = np.where(p > 2.0 ** -40, big, 0.0).max(1)
            p /= p.sum(1, keepdims=True)
            out[r:r + n, h], mass[r:r + n, h] = p @ vv, p @ np.abs(vv)
    return out, mass


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("option", ["plain", "all"])
def test_value_scales_by_powers_of_two_over_thousands_of_items(kind, dim, option):
    # 40 units of tokens x 64 kv heads: every SM walks about seventeen items, tile
    # after tile.  A page's scale is never that of the page 64 before, whose
    # place in shared memory it takes: a scale that is read too early or too
    # late is off by a power of two.
    rng = np.random.default_rng(30)
    q = rng.integers(1, 40, 40)
    b = R.make(30, q, q + rng.integers(0, 700, 40), 64, 64, dim, nan_tail=False)
    steps = 6
    for s in range(40):
        for page in range(-(-int(b.ctx[s]) // 16)):
            b.v[b.tables[s, page]] *= np.float16(2.0 ** ((5 * page + s) % (2 * steps + 1) - steps))
    o = expand(b, dict(cap=20.0, bias=True, window=300, prefix=40) if option == "all" else option)
    pools, kv64 = R.cache(b, kind)
    got, status = Run(b, kind, pools, **o)()
    ref, mass = attend(b, kv64, dim ** -0.5, **o)
    # Products of a probability and a ratio of scales (2^6 in front of them, the
    # largest probability of a row at 2^6 or more) below the normal fp16 numbers
    # are rounded by up to 2^-25: 2^-31 of the largest value for each key.
    small = int(b.ctx.max()) * 2.0 ** -31 * np.abs(kv64[1][b.used]).max()
    assert status == 0
    worst = np.max(np.abs(got - ref) / (bound(b, kind, o, ref, mass) + small))
    assert worst <= 1.0, worst


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("option", ["plain", "cap"])
@pytest.mark.parametrize("why", ["ahead", "left", "outweighed"])
def test_pages_that_do_not_count_for_a_row_cost_it_no_bits(kind, option, why):
    # One page's values are 2^25 times the others'.  Rows that do not see it (it
    # lies ahead, or their window has left it), and rows whose later scores
    # outweigh it, are as exact as if it were not there.
    o = dict(cap=200.0) if option == "cap" else {}
    if why == "ahead":
        b, page = R.make(31, [40], [120], 4, 1, 64, q_std=0.05, nan_tail=False), 7
    elif why == "left":
        b, page = R.make(32, [100], [120], 4, 1, 64, q_std=0.05, nan_tail=False), 0
        o["window"] = 40
    else:
        b, page = R.make(33, [30], [160], 4, 1, 64, q_std=0.05, nan_tail=False), 0
        b.q[:, :, 0] = 8.0                                    # 40 for the keys from 128 on
        for g in range(10):
            b.k[b.tables[0, g], :, :, 0] = 0.0 if g < 8 else 40.0
    for g in range(-(-int(b.ctx[0]) // 16)):
        b.v[b.tables[0, g]] *= np.float16(2.0 ** (13 if g == page else -12))
    o = expand(b, o)
    pools, kv64 = R.cache(b, kind)
    got, status = Run(b, kind, pools, **o)()
    top = np.zeros(b.q.shape[:2])
    ref, mass = attend(b, kv64, 0.125, top, **o)
    # (small products, as above; the reference may be 8 times the largest scale
    # that counts for the row: 2^-28 of its largest value for each key)
    small = int(b.ctx[0]) * 2.0 ** -28 * top[:, :, None]
    assert status == 0
    assert (top < 1.0).sum() >= 100  # rows that the page does not count for
    worst = np.max(np.abs(got - ref) / (bound(b, kind, o, ref, mass) + small))
    assert worst <= 1.0, worst


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("option", ["plain", "all"])
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_scales_that_are_not_finite_show(kind, option, value):
    # in every row that sees the page, and not in other sequences
    b = R.make(34, [40, 9], [120, 90], 4, 1, 64, nan_tail=False)
    o = expand(b, dict(cap=20.0, bias=True) if option == "all" else option)
    pools, _ = R.cache(b, kind)
    pools[3][b.tables[0, 3]] = value                       # tokens 48 .. 63
    got, status = Run(b, kind, pools, **o)()
    assert status == 0
    assert not np.any(np.isfinite(got[:40]).all(axis=2))   # rows 80 .. 119
    assert np.all(np.isfinite(got[40:]))
