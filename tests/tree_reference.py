"""Plain references of the operators for trees of drafted tokens: attention in 64
bits, the walk along the model's answers, and the rows that stay moved together.
NumPy on the CPU, one row at a time."""
import numpy as np

import oracle
import serving_reference as R

BS = 16


def trees(seed, q_lens, shape="random"):
    """Parents (rows within the sequence) of every token."""
    rng = np.random.default_rng(seed)
    out = []
    for n in q_lens:
        i = np.arange(n)
        if shape == "chain":
            p = i - 1
        elif shape == "star":
            p = np.where(i > 0, 0, -1)
        elif shape == "roots":      # several tokens that follow the context itself
            p = np.array([rng.integers(-1, j) if j else -1 for j in i], np.int64)
        else:
            p = np.array([rng.integers(max(0, (j - 1) // 3), j) if j else -1 for j in i], np.int64)
        out.append(np.asarray(p, np.int32).reshape(-1))
    return np.concatenate(out) if out else np.zeros(0, np.int32)


def path_to(parents, j):
    """Row j and its ancestors, from the root."""
    path = []
    while j >= 0:
        path.append(j)
        j = int(parents[j])
    return path[::-1]


def attend(b, parents, kv64, scale, cap=0.0, window=0, slopes=None, prefix=None):
    """(out, mass) fp64 [T][Hq][d]: the definition, and sum_t p_t |V_t|."""
    out, mass = np.full(b.q.shape, np.nan), np.full(b.q.shape, np.nan)
    for s in range(b.ctx.size):
        c, n, first = int(b.ctx[s]), int(b.q_lens[s]), int(b.starts[s])
        blk, base = b.tables[s, :-(-c // BS)], c - n
        pre = 0 if prefix is None else min(max(int(prefix[s]), 0), base)
        kk = [x[blk].transpose(1, 0, 2, 3).reshape(b.kv_heads, -1, b.dim)[:, :c] for x in kv64]
        for r in range(n):
            path = path_to(parents[first:first + n], r)
            i = base + len(path) - 1
            gap = np.full(c, -1)
            gap[:base] = i - np.arange(base)
            gap[base + np.asarray(path)] = np.arange(len(path))[::-1]
            seen = gap >= 0
            if window:
                seen &= (gap < window) | (np.arange(c) < pre)
            for h in range(b.heads):
                k64, v64 = (x[h // b.group][seen] for x in kk)
                z = k64 @ b.q[first + r, h].astype(np.float64) * scale
                if cap:
                    z = cap * np.tanh(z / cap)
                if slopes is not None:
                    z = z - float(slopes[h]) * gap[seen]
                p = np.exp(z - z.max())
                p /= p.sum()
                out[first + r, h], mass[first + r, h] = p @ v64, p @ np.abs(v64)
    return out, mass


def accept(parents, tokens, targets, starts):
    """(kept, kept_lens, next_tokens): children are looked for in every row."""
    kept = np.full(parents.size, -1, np.int32)
    lens, last = [], []
    for a, e in zip(starts[:-1], starts[1:]):
        path = [0] if e > a else []
        while path:
            now = path[-1]
            fits = [j for j in range(e - a) if parents[a + j] == now
                    and tokens[a + j] == targets[a + now]]
            if not fits:
                break
            path.append(fits[0])
        kept[a:a + len(path)] = path
        lens.append(len(path))
        last.append(targets[a + path[-1]] if path else -1)
    return kept, np.asarray(lens, np.int32), np.asarray(last, np.int32)


def compact(b, kept, kept_lens, pools):
    """(new lengths, pools, blocks that got a row) after the rows are moved."""
    pools = [x.copy() for x in pools]
    old = [x.copy() for x in pools]
    lens, written = [], set()
    for s in range(b.ctx.size):
        base, m = int(b.ctx[s]) - int(b.q_lens[s]), int(kept_lens[s])
        lens.append(base + m)
        for j in range(m):
            i = int(kept[int(b.starts[s]) + j])
            if i == j:
                continue
            to, of = b.tables[s, (base + j) // BS], b.tables[s, (base + i) // BS]
            written.add(int(to))
            for x, y in zip(pools, old):
                x[to, :, (base + j) % BS] = y[of, :, (base + i) % BS]
    return np.asarray(lens, np.int32), pools, np.asarray(sorted(written), np.int32)


def tiles(kind, x, blocks):
    """Codes and scales that the quantizer gives the blocks of an fp16 pool."""
    quant = oracle.quantize_fp8 if kind == "fp8" else oracle.quantize
    codes, scales = quant(x, block_ids=blocks)
    return codes[blocks], scales[blocks]


def bound(b, o, ref, mass, scale):
    """As for the prefill: the probabilities (with codes times the V scale) are
    rounded to fp16, half a step of 2^-11."""
    dz = R.score_error(b, "fp16", abs(scale), o.get("cap", 0.0), int(b.ctx.max()), o["slopes"])
    return R.tolerance(ref, mass, dz, 11)
