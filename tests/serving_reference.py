"""Plain 64-bit references and inputs of the serving operators' tests: the
rotation of a ragged batch on its way into the cache, and attention with
capped, biased and masked scores.  NumPy on the CPU, one row at a time."""
import dataclasses

import numpy as np

import oracle

BS = 16


@dataclasses.dataclass
class Batch:
    """A ragged batch over a paged cache.  q_lens new tokens of ctx cached ones."""
    q_lens: np.ndarray
    ctx: np.ndarray
    starts: np.ndarray     # int32 [N + 1]
    tables: np.ndarray     # int32 [N][MB]
    k: np.ndarray          # fp16 pools [NB][Hkv][16][d]
    v: np.ndarray
    q: np.ndarray          # fp16 [T][Hq][d]
    heads: int
    kv_heads: int
    dim: int

    @property
    def group(self):
        return self.heads // self.kv_heads

    @property
    def used(self):
        return np.unique(self.tables[self.tables >= 0]).astype(np.int32)


def make(seed, q_lens, ctx, heads, kv_heads, dim, q_std=2.0, extra_rows=0, nan_tail=True):
    """N(0, 1) keys and values, N(0, q_std) queries; slots behind a sequence's
    last token NaN (recycled blocks hold anything), tables -1 where unused."""
    rng = np.random.default_rng(seed)
    q_lens, ctx = np.asarray(q_lens), np.asarray(ctx)
    n = ctx.size
    pages = -(-ctx // BS)
    nb = int(pages.sum()) + 3
    perm = rng.permutation(nb)
    tables = np.full((n, max(1, int(pages.max()) if n else 1)), -1, np.int32)
    at = 0
    for s in range(n):
        tables[s, :pages[s]] = perm[at:at + pages[s]]
        at += pages[s]
    shape = (nb, kv_heads, BS, dim)
    k = rng.standard_normal(shape, dtype=np.float32).astype(np.float16)
    v = rng.standard_normal(shape, dtype=np.float32).astype(np.float16)
    if nan_tail:
        for s in range(n):
            if ctx[s] % BS:
                for x in (k, v):
                    x[tables[s, pages[s] - 1], :, ctx[s] % BS:] = np.nan
    t = int(q_lens.sum()) + extra_rows
    q = (rng.standard_normal((t, heads, dim), dtype=np.float32) * q_std).astype(np.float16)
    starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    return Batch(q_lens, ctx.astype(np.int32), starts, tables, k, v, q, heads, kv_heads, dim)


def cache(b, kind):
    """What the kind's cache holds: (pools and scales as the calls take them,
    fp64 K and V pools)."""
    if kind == "fp16":
        return (b.k, b.v), (b.k.astype(np.float64), b.v.astype(np.float64))
    quant = oracle.quantize_fp8 if kind == "fp8" else oracle.quantize
    out, vals = [], []
    for x in (b.k, b.v):
        codes, scales = quant(x, block_ids=b.used)
        c = e4m3(codes) if kind == "fp8" else codes.astype(np.float64)
        out.append((codes, scales))
        vals.append(c * scales[:, :, None, None].astype(np.float64))
    return (out[0][0], out[1][0], out[0][1], out[1][1]), tuple(vals)


def quantize(tiles, kind):
    """Codes and scales of fp16 tiles [n][Hkv][16][d] as the rotation's append
    makes them: scale = amax * fl(1 / most) in fp32, then the nearest code of
    the fp32 quotient."""
    f = tiles.astype(np.float32)
    most = np.float32(127 if kind == "int8" else 448)
    scale = np.nanmax(np.abs(f), axis=(2, 3)) * (np.float32(1) / most)
    with np.errstate(invalid="ignore", divide="ignore"):
        y = np.nan_to_num(f / scale[:, :, None, None], nan=0.0, posinf=most, neginf=-most)
    y = np.clip(y, -most, most)
    if kind == "int8":
        return np.rint(y).astype(np.int8), scale
    # nearest of the 127 finite magnitudes, ties to the even code
    mags = e4m3(np.arange(127, dtype=np.uint8))
    a = np.abs(y).astype(np.float64)
    hi = np.clip(np.searchsorted(mags, a), 1, 126)
    lo = hi - 1
    up, down = mags[hi] - a, a - mags[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(y), 128, 0)).astype(np.uint8), scale


def e4m3(codes):
    """Values of OCP E4M3 bytes (1 sign, 4 exponent, 3 mantissa bits, bias 7)."""
    c = codes.astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(c & 128, -v, v)


def visible(i, t, window, prefix):
    return ((t <= i) & ((i - t < window) if window else True)) | (t < prefix)


def attend(b, kv64, scale, cap=0.0, window=0, slopes=None, prefix=None, rows=None):
    """(out, mass) fp64 [T][Hq][d]: the definition, and sum_t p_t |V_t|, which
    the errors of the probabilities are relative to.  rows: (first token,
    context) pairs to compute, default all of the batch; the others are NaN."""
    k64, v64 = kv64
    out = np.full(b.q.shape, np.nan)
    mass = np.full(b.q.shape, np.nan)
    for s in range(b.ctx.size):
        c, n = int(b.ctx[s]), int(b.q_lens[s])
        blk = b.tables[s, :-(-c // BS)]
        for h in range(b.heads):
            kk = k64[blk, h // b.group].reshape(-1, b.dim)[:c]
            vv = v64[blk, h // b.group].reshape(-1, b.dim)[:c]
            for j in range(n):
                row, i = int(b.starts[s]) + j, c - n + j
                t = np.arange(c)
                seen = visible(i, t, window, 0 if prefix is None else int(prefix[s]))
                if not seen.any():
                    out[row, h] = mass[row, h] = 0.0
                    continue
                z = kk[seen] @ b.q[row, h].astype(np.float64) * scale
                if cap:
                    z = cap * np.tanh(z / cap)
                if slopes is not None:
                    z = z - float(slopes[h]) * np.abs(i - t[seen])
                p = np.exp(z - z.max())
                p /= p.sum()
                out[row, h] = p @ vv[seen]
                mass[row, h] = p @ np.abs(vv[seen])
    return out, mass


def score_error(b, kind, scale, cap, ctx_max, slopes):
    """Bound of the error of one score (natural units).

    The products of fp16 values are exact in fp32; the tensor core adds 16 of
    them at a time, so a score goes through d / 16 + 2 roundings of 2^-23 of
    its partial sums, which sum |q||k| bounds.  INT8 keys in the decode carry a
    constant 1152, which the sums contain until it is taken off.  The cap adds
    2^-21 of itself (see cap_score), the bias one rounding of its own size."""
    q = np.abs(b.q.astype(np.float64)).sum(-1).max()
    used = b.k[b.used].astype(np.float64)
    top = np.nanmax(np.abs(used))
    most = top + (1152 * top / 127 if kind == "int8" else 0.0)
    err = (b.dim / 16 + 2) * 2.0 ** -23 * q * most * scale + 2.0 ** -21 * cap
    if slopes is not None:
        err += 2.0 ** -22 * float(np.max(slopes)) * ctx_max
    # the score in log2 units and its exponential: a few more roundings of
    # 2^-23 of a score of at most q * top * scale
    return err + 4 * 2.0 ** -23 * q * top * scale


def tolerance(ref, mass, dz, p_bits):
    """|out - ref| allowed: half a step of fp16 (and of its smallest step), and
    the probabilities' error relative to sum p |V|: 2 dz (numerator and
    denominator), their rounding (2^-p_bits, half a step) and 2^-20 for the
    exponential and the fp32 sums."""
    return 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (2 * dz + 2.0 ** -p_bits + 2.0 ** -20) * mass


# ------------------------------------------------------------------- rotation
def rotate32(x, cos, sin, interleaved):
    """fp16 [..][rot] rotated with fp32 steps, each rounded; cos, sin [..][rot / 2]."""
    f = x.astype(np.float32)
    half = f.shape[-1] // 2
    a, b = (f[..., 0::2], f[..., 1::2]) if interleaved else (f[..., :half], f[..., half:])
    cos, sin = cos.astype(np.float32), sin.astype(np.float32)
    ya, yb = a * cos - b * sin, b * cos + a * sin
    y = np.empty_like(f)
    if interleaved:
        y[..., 0::2], y[..., 1::2] = ya, yb
    else:
        y[..., :half], y[..., half:] = ya, yb
    return y.astype(np.float16)


def rope_append(b, qkv, table, rope_positions, axis_of_pair, interleaved, pools, owners=None):
    """(q_out rows, k pool, v pool, written blocks) after the call; table fp32
    [P][rot]; qkv fp16 [T][Hq + 2 Hkv][d]."""
    rot = table.shape[1]
    half = rot // 2
    k, v = pools[0].copy(), pools[1].copy()
    q_out = np.zeros((qkv.shape[0], b.heads, b.dim), np.float16)
    written = set()
    for s in range(b.ctx.size):
        for j in range(int(b.q_lens[s])):
            row = int(b.starts[s]) + j
            pos = int(b.ctx[s]) - int(b.q_lens[s]) + j
            if rope_positions is None:
                p = np.full(half, pos)
            else:
                p = rope_positions[axis_of_pair, row]
            pair = np.arange(half)
            cos, sin = table[p, pair], table[p, half + pair]
            x = qkv[row].copy()
            x[:b.heads + b.kv_heads, :rot] = rotate32(x[:b.heads + b.kv_heads, :rot], cos, sin,
                                                      interleaved)
            q_out[row] = x[:b.heads]
            blk = b.tables[s, pos // BS]
            k[blk, :, pos % BS] = x[b.heads:b.heads + b.kv_heads]
            v[blk, :, pos % BS] = x[b.heads + b.kv_heads:]
            written.add(int(blk))
    return q_out, k, v, np.asarray(sorted(written), np.int32)
