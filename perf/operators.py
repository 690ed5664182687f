"""Workloads of the serving operators around the paged KV cache.

Three operators, each over fp16, INT8 and FP8 (E4M3) caches:

* append:  rotate the queries and keys of a ragged batch of new tokens (one
           position axis, or several for images and video) and write the keys
           and values into the paged cache;
* prefill: attention of a ragged batch of new tokens, causal over the paged
           cache, with an optional tanh cap, distance bias, window and prefix;
* decode:  the same attention for one new token per sequence.

``listed()`` names the measured cases and ``draw()`` gives further ones of the
same ranges.  ``run()`` makes one pass: the library's calls where ``own`` is
true, elementary torch operations otherwise.
"""
import math

import numpy as np
import torch

own = False

BS = 16          # tokens per block
BASE = 10000.0   # rotary base of the tables


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of a serving batch: 64 sequences get their token
        _append("append step 64", "fp16", 64, 1, 2048, (32, 8, 128)),
        # a chunk of prompt tokens of several sequences, each going on in the
        # middle of its cache, into an INT8 cache
        _append("append chunk int8", "int8", 24, 683, 4096, (32, 8, 128), ragged=11),
        # whole prompts
        _append("append prompts", "fp16", 16, 4096, 4096, (32, 8, 128)),
        # image tokens with (time, height, width) positions, half of each head
        # rotated, neighbouring values paired, FP8 cache, odd lengths
        _append("append image fp8", "fp8", 9, 1177, 1200, (14, 2, 64), ragged=12, axes=3,
                rot=32, paired=True),
        # the smallest attention call: a small batch, where latency counts
        _attend("decode 8x512 int8 capped", "decode", "int8", 8, 1, 512, (8, 8, 128), cap=30.0),
        # a serving batch with capped scores
        _attend("decode 64x2048 capped", "decode", "fp16", 64, 1, 2048, (32, 8, 128), cap=50.0),
        # a large ragged batch that attends to a window and to the first tokens
        _attend("decode 256 ragged int8 window", "decode", "int8", 256, 1, 4096, (32, 8, 128),
                ragged=13, window=1024, prefix=16),
        # one long context with a bias by distance
        _attend("decode 1x131072 fp8 bias", "decode", "fp8", 1, 1, 131072, (32, 8, 128),
                bias=True),
        # a few drafted tokens per sequence to be verified
        _attend("verify 32x5 over 2048", "prefill", "fp16", 32, 5, 2048, (14, 2, 64)),
        # prompts of a new batch
        _attend("prefill 8x2048", "prefill", "fp16", 8, 2048, 2048, (32, 8, 128)),
        # ragged chunks over INT8 caches, prefix visible to everyone, window
        _attend("prefill ragged int8 window", "prefill", "int8", 12, 1500, 5000, (28, 4, 128),
                ragged=14, window=1024, prefix=100, bias=True),
        # a chunk of a long document, capped scores
        _attend("prefill 4096 over 16384 capped", "prefill", "fp16", 1, 4096, 16384,
                (32, 8, 128), cap=30.0),
    ]


def _append(name, kind, seqs, new, ctx, heads, ragged=0, axes=1, rot=0, paired=False):
    c = {"op": "append", "kind": kind, "seqs": seqs, "new": new, "ctx": ctx,
         "heads": heads[0], "kv_heads": heads[1], "dim": heads[2], "ragged": ragged,
         "axes": axes, "rot": rot or heads[2], "paired": paired}
    return dict(c, name=name) if name else c


def _attend(name, op, kind, seqs, new, ctx, heads, ragged=0, cap=0.0, window=0, prefix=0,
            bias=False):
    c = {"op": op, "kind": kind, "seqs": seqs, "new": new, "ctx": ctx, "heads": heads[0],
         "kv_heads": heads[1], "dim": heads[2], "ragged": ragged, "cap": cap,
         "window": window, "prefix": prefix, "bias": bias}
    return dict(c, name=name) if name else c


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "decode", "prefill"])
    kind = rng.choice(["fp16", "int8", "fp8"])
    ragged = rng.choice([0, rng.randrange(1, 1 << 20)])
    if op == "append":
        heads = rng.choice([(32, 8, 128), (14, 2, 64), (16, 2, 128), (28, 4, 128), (8, 2, 64)])
        tokens = log(8, 65536)
        seqs = log(1, min(256, tokens))
        new = max(1, tokens // seqs)
        ctx = new + log(1, 4096)
        rot = rng.choice([heads[2], heads[2] // 2, heads[2] // 4])
        return _append("", kind, seqs, new, ctx, heads, ragged, rng.choice([1, 3]), rot,
                       rng.choice([False, True]))
    heads = rng.choice([(32, 8, 128), (14, 2, 64), (8, 8, 128), (28, 4, 128), (16, 1, 128),
                        (12, 4, 64)])
    cap = rng.choice([0.0, round(rng.uniform(10.0, 60.0), 1)])
    window = rng.choice([0, log(16, 4096)])
    prefix = rng.choice([0, 0, log(1, 1000)])
    bias = rng.choice([False, False, True])
    if op == "decode":
        total = log(1 << 12, 1 << 19)
        seqs = log(1, 256)
        return _attend("", op, kind, seqs, 1, max(17, total // seqs), heads, ragged, cap,
                       window, prefix, bias)
    scores = log(1 << 22, 1 << 31)  # query tokens x keys x heads of the padded batch
    ctx = log(64, 16384)
    most = max(2, scores // (heads[0] * ctx))
    new = min(ctx, log(2, min(4096, most)))
    seqs = max(1, min(64, scores // (heads[0] * ctx * new)))
    return _attend("", op, kind, seqs, new, ctx, heads, ragged, cap, window, prefix, bias)


def _lengths(case):
    """New tokens and context lengths (with the new tokens) of the sequences."""
    n, new, ctx = case["seqs"], case["new"], case["ctx"]
    if not case["ragged"]:
        return np.full(n, new, np.int64), np.full(n, ctx, np.int64)
    r = np.random.RandomState(case["ragged"])
    q = r.randint(max(1, new // 8), new + 1, n)
    old = r.randint(0, ctx - new + 1, n)
    if new == 1:
        old = r.randint(0, ctx, n)
    return q.astype(np.int64), (q + old).astype(np.int64)


def _visible(case, q, ctx):
    """(pairs of a query token and a key it sees, keys that some token of the
    sequence sees), summed over the sequences."""
    pairs = keys = 0
    for n, c in zip(q.tolist(), ctx.tolist()):
        p = np.arange(c - n, c, dtype=np.int64)
        lo = np.maximum(0, p - case["window"] + 1) if case["window"] else np.zeros_like(p)
        pre = min(case["prefix"], c)
        pairs += int((p - lo + 1).sum() + np.where(pre <= lo, pre, np.maximum(lo, pre - p - 1 + lo)).sum())
        keys += c if pre >= lo[0] else pre + c - int(lo[0])
    return pairs, keys


def work(case):
    q, ctx = _lengths(case)
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    elem = 2 if case["kind"] == "fp16" else 1
    t = int(q.sum())
    if case["op"] == "append":
        bytes_ = t * ((h + 2 * hk) * d * 2 * 2 + 4 * case["rot"] + 4 * case["axes"])
        if case["kind"] != "fp16":
            # the written tiles' codes, and the rows that were there before
            first, last = (ctx - q) // BS, (ctx - 1) // BS
            tiles = int((last - first + 1).sum())
            bytes_ += tiles * hk * 2 * (BS * d + 4) + (tiles * BS - t) * hk * 2 * d * 2
        return {"bytes": bytes_, "flops": t * (h + hk) * case["rot"] * 3}
    pairs, keys = _visible(case, q, ctx)
    bytes_ = 2 * t * h * d * 2 + keys * hk * 2 * d * elem + keys // BS * 4
    if case["kind"] != "fp16":
        bytes_ += keys // BS * hk * 2 * 4
    return {"bytes": bytes_, "flops": 4 * d * h * pairs}


# ------------------------------------------------------------------ the inputs
def _codes(kind, x):
    """Codes and per-(block, kv head) scales of fp16 tiles [n][Hkv][16][d]."""
    f = x.float()
    most = 127.0 if kind == "int8" else 448.0
    scale = torch.nan_to_num(f.abs(), nan=0.0).amax(dim=(2, 3)) / most
    y = torch.nan_to_num(f / scale[:, :, None, None], nan=0.0).clamp(-most, most)
    if kind == "int8":
        return y.round().to(torch.int8), scale
    return y.to(torch.float8_e4m3fn).view(torch.uint8), scale


def _normal(shape, gen, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16).mul_(std)


def prepare(case, seed):
    q, ctx = _lengths(case)
    n, t = case["seqs"], int(q.sum())
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pages = (ctx + BS - 1) // BS
    blocks = int(pages.sum()) + 7
    # the sequences' blocks lie anywhere in the pool; unused table entries -1
    perm = torch.randperm(blocks, generator=gen, device="cuda", dtype=torch.int32)
    width = int(pages.max())
    used = torch.from_numpy(np.arange(width)[None, :] < pages[:, None]).cuda()
    tables = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    tables[used] = perm[: int(pages.sum())]
    starts = np.concatenate([[0], np.cumsum(q)])
    s = {"case": case, "tables": tables, "max_ctx": int(ctx.max()), "seqs": n,
         "starts": torch.from_numpy(starts.astype(np.int32)).cuda(),
         "lens": torch.from_numpy(ctx.astype(np.int32)).cuda(),
         "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    shape = (blocks, hk, BS, d)
    k, v = _normal(shape, gen), _normal(shape, gen)
    if case["op"] == "append":
        s["qkv"] = _normal((t, (h + 2 * hk) * d), gen)
        s["k"], s["v"] = k, v
        if case["kind"] != "fp16":
            for x in "kv":
                s[x + "_codes"], s[x + "_scales"] = _codes(case["kind"], s[x])
        s["table"] = _rotation_table(int(ctx.max()) + 64, case["rot"])
        pairs = case["rot"] // 2
        at = np.concatenate([np.arange(c - m, c) for m, c in zip(q.tolist(), ctx.tolist())])
        if case["axes"] == 1:
            s["positions"], s["axis"] = None, None
        else:
            # images of 32 x 32 tokens that follow one another: time, height,
            # width; the time axis takes the first pairs
            pos = np.stack([at // 1024, at // 32 % 32, at % 32])
            s["positions"] = torch.from_numpy(pos.astype(np.int32)).cuda()
            cut = [pairs // 4, pairs // 4 + (pairs - pairs // 4) // 2]
            s["axis"] = np.searchsorted(cut, np.arange(pairs), side="right").astype(np.uint8)
        return s
    # slots behind a sequence's last token hold whatever was there before
    rest = torch.from_numpy((pages * BS - ctx).astype(np.int64)).cuda()
    last = tables.gather(1, torch.from_numpy(pages - 1)[:, None].cuda())[:, 0].long()
    stale = torch.arange(BS, device="cuda")[None, :] >= BS - rest[:, None]
    if case["kind"] == "fp16":
        for x in (k, v):
            x[last] = torch.where(stale[:, None, :, None], torch.nan, x[last])
        s["k"], s["v"] = k, v
    else:
        s["k"], s["k_scales"] = _codes(case["kind"], k)
        s["v"], s["v_scales"] = _codes(case["kind"], v)
    # queries whose scores spread over several units, as sharp heads' do
    s["q"] = _normal((t, h, d), gen, 2.0)
    s["slopes"] = None
    if case["bias"]:
        s["slopes"] = torch.pow(2.0, -8.0 * torch.arange(1, h + 1, device="cuda") / h)
    s["prefix"] = None
    if case["prefix"]:
        s["prefix"] = torch.full((n,), case["prefix"], dtype=torch.int32, device="cuda")
    return s


def _rotation_table(positions, rot):
    """fp32 [positions][rot]: the cosines of all pairs, then the sines."""
    freq = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([a.cos(), a.sin()], dim=1).float()


# ------------------------------------------------------------------- one pass
def run(state):
    if own:
        return _run_own(state)
    if state["case"]["op"] == "append":
        return _plain_append(state)
    return _plain_attend(state)


def _run_own(s):
    import paged_kv_cache_234_gb300 as pkv

    c = s["case"]
    if "call" not in s:
        # a serving loop keeps its output buffers and its prepared call, and
        # updates the inputs in place from step to step
        h, hk, d, scale = c["heads"], c["kv_heads"], c["dim"], c["dim"] ** -0.5
        if c["op"] == "append":
            x = s["qkv"].view(s["qkv"].shape[0], h + 2 * hk, d)
            s["out"] = torch.empty((x.shape[0], h, d), dtype=torch.float16, device="cuda")
            codes = [s[n] for n in ("k_codes", "v_codes", "k_scales", "v_scales")
                     if c["kind"] != "fp16"]
            make = getattr(pkv, "prepare_rope_append_" + c["kind"])
            s["call"] = make(s["out"], s["k"], s["v"], *codes, x[:, :h], x[:, h:h + hk],
                             x[:, h + hk:], s["table"], s["starts"], s["lens"], s["tables"],
                             rope_positions=s["positions"], axis_of_pair=s["axis"],
                             interleaved=c["paired"], dev_status=s["status"])
        else:
            s["out"] = torch.empty_like(s["q"])
            kv = [s["k"], s["v"]]
            kv += [s["k_scales"], s["v_scales"]] if c["kind"] != "fp16" else []
            options = dict(logit_cap=c["cap"], window=c["window"], slopes=s["slopes"],
                           prefix_lens=s["prefix"], dev_status=s["status"])
            if c["op"] == "decode":
                make = getattr(pkv, "prepare_paged_decode_scored_" + c["kind"])
                ws = pkv.decode_workspace(s["seqs"], h, hk, d, s["max_ctx"])
                s["call"] = make(s["out"], s["q"], *kv, s["tables"], s["lens"], s["max_ctx"],
                                 scale, ws, **options)
            else:
                make = getattr(pkv, "prepare_paged_prefill_" + c["kind"])
                ws = pkv.prefill_workspace(s["q"].shape[0], s["seqs"], h, hk, d, s["max_ctx"])
                s["call"] = make(s["out"], s["q"], *kv, s["tables"], s["starts"], s["lens"],
                                 s["max_ctx"], scale, ws, **options)
    s["call"]()
    if c["op"] == "append":
        return _append_outputs(s, s["out"])
    return s["out"]


def _append_outputs(s, q):
    out = {"q": q, "k": s["k"], "v": s["v"]}
    if s["case"]["kind"] != "fp16":
        # codes and scales: codes * scales are the values that the cache holds
        out.update({n: s[n] for n in ("k_codes", "v_codes", "k_scales", "v_scales")})
    return out


def _token_map(s):
    """Sequence and cache position of every new token."""
    starts, lens = s["starts"].long(), s["lens"].long()
    t = s["qkv"].shape[0] if "qkv" in s else s["q"].shape[0]
    token = torch.arange(t, device="cuda")
    seq = torch.searchsorted(starts, token, right=True) - 1
    row = token - starts[seq]
    return seq, row, lens[seq] - (starts[seq + 1] - starts[seq]) + row


def _plain_append(s):
    c = s["case"]
    h, hk, d, half = c["heads"], c["kv_heads"], c["dim"], c["rot"] // 2
    seq, _, pos = _token_map(s)
    x = s["qkv"].view(-1, h + 2 * hk, d)
    pair = torch.arange(half, device="cuda")
    if s["positions"] is None:
        at = pos[:, None].expand(-1, half)
    else:
        at = s["positions"].long().t()[:, torch.from_numpy(s["axis"]).long().cuda()]
    cos, sin = s["table"][at, pair][:, None], s["table"][at, pair + half][:, None]
    r = x[:, :h + hk, :c["rot"]].float()
    a, b = (r[..., 0::2], r[..., 1::2]) if c["paired"] else (r[..., :half], r[..., half:])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if c["paired"] else torch.cat([a, b], -1)
    turned = torch.cat([turned.half(), x[:, :h + hk, c["rot"]:]], -1)
    block = s["tables"][seq, pos // BS].long()
    s["k"][block, :, pos % BS] = turned[:, h:]
    s["v"][block, :, pos % BS] = x[:, h + hk:]
    if c["kind"] != "fp16":
        block = torch.unique(block)
        for n in "kv":
            s[n + "_codes"][block], s[n + "_scales"][block] = _codes(c["kind"], s[n][block])
    return _append_outputs(s, turned[:, :h].contiguous())


def _values(s, name, block):
    """The fp32 values [...][Hkv][16][d] of the pool's blocks."""
    x = s[name][block]
    if s["case"]["kind"] == "fp16":
        return x.float()
    if s["case"]["kind"] == "fp8":
        x = x.view(torch.float8_e4m3fn)
    return x.float() * s[name + "_scales"][block][..., None, None]


def _plain_attend(s):
    c = s["case"]
    n, h, hk, d, g = s["seqs"], c["heads"], c["kv_heads"], c["dim"], c["heads"] // c["kv_heads"]
    seq, row, pos = _token_map(s)
    lens = s["lens"].long()
    m = c["new"]
    q = torch.zeros((n, m, h, d), device="cuda")
    q[seq, row] = s["q"].float()
    q = q.view(n, m, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, g * m, d)
    block = s["tables"].clamp(min=0).long()
    key = torch.arange(block.shape[1] * BS, device="cuda")
    held = key[None, :] < lens[:, None]                                    # [n][keys]

    def gather(name):
        x = _values(s, name, block).permute(0, 2, 1, 3, 4).reshape(n, hk, -1, d)
        return torch.where(held[:, None, :, None], x, 0.0)

    z = q @ gather("k").transpose(2, 3)
    z = z.mul_(d ** -0.5).view(n, hk, g, m, -1)
    if c["cap"]:
        z = z.div_(c["cap"]).tanh_().mul_(c["cap"])
    at = torch.zeros((n, m), dtype=torch.long, device="cuda")
    at[seq, row] = pos
    gap = at[:, :, None] - key[None, None, :]                              # [n][m][keys]
    if s["slopes"] is not None:
        z -= s["slopes"].view(hk, g, 1, 1) * gap.abs()[:, None, None]
    seen = gap >= 0
    if c["window"]:
        seen &= gap < c["window"]
    if s["prefix"] is not None:
        seen |= key[None, None, :] < s["prefix"].long()[:, None, None]
    seen &= held[:, None, :]
    z = torch.where(seen[:, None, None], z, -torch.inf)
    z = z.sub_(z.amax(-1, keepdim=True)).exp_()
    z /= z.sum(-1, keepdim=True)
    o = z.view(n, hk, g * m, -1) @ gather("v")
    o = o.view(n, hk, g, m, d).permute(0, 3, 1, 2, 4).reshape(n, m, h, d)
    return o[seq, row].half()


# ------------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    q_lens, ctx = _lengths(case)
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    g = h // hk
    f64 = torch.float64
    if case["op"] == "append":
        half = case["rot"] // 2
        i = torch.arange(half, device="cuda")
        lo, hi = (2 * i, 2 * i + 1) if case["paired"] else (i, i + half)
        axis = torch.zeros(half, dtype=torch.long, device="cuda")
        if s["axis"] is not None:
            axis = torch.from_numpy(s["axis"]).long().cuda()
        q = torch.empty((int(q_lens.sum()), h, d), dtype=f64, device="cuda")
        k, v = s["k"].double(), s["v"].double()
        t0 = 0
        for b, (n, c) in enumerate(zip(q_lens.tolist(), ctx.tolist())):
            x = s["qkv"][t0:t0 + n].double().view(n, h + 2 * hk, d)
            where = torch.arange(c - n, c, device="cuda")
            p = where[None] if s["positions"] is None else s["positions"][:, t0:t0 + n].long()
            table = s["table"].double()
            co = torch.stack([table[p[a], j] for j, a in enumerate(axis.tolist())], 1)[:, None]
            si = torch.stack([table[p[a], j + half] for j, a in enumerate(axis.tolist())], 1)[:, None]
            turned = x[:, :h + hk].clone()
            turned[..., lo] = x[:, :h + hk, lo] * co - x[:, :h + hk, hi] * si
            turned[..., hi] = x[:, :h + hk, lo] * si + x[:, :h + hk, hi] * co
            q[t0:t0 + n] = turned[:, :h]
            blk = s["tables"][b].long()[where // BS]
            k[blk, :, where % BS] = turned[:, h:]
            v[blk, :, where % BS] = x[:, h + hk:]
            t0 += n
        out = {"q": q, "k": k, "v": v}
        if case["kind"] != "fp16":
            out.update(k_codes=None, v_codes=None, k_scales=None, v_scales=None)
        return out
    if 4 * d * h * float((q_lens * ctx).sum()) > 4e12:
        return None
    out, t0 = [], 0
    for b, (n, c) in enumerate(zip(q_lens.tolist(), ctx.tolist())):
        blk = s["tables"][b, :(c + BS - 1) // BS].long()
        kv = []
        for name in "kv":
            x = s[name][blk]
            x = x.view(torch.float8_e4m3fn).float().double() if case["kind"] == "fp8" else x.double()
            if case["kind"] != "fp16":
                x = x * s[name + "_scales"][blk].double()[:, :, None, None]
            kv.append(x.transpose(0, 1).reshape(hk, -1, d)[:, :c])
        i = torch.arange(c - n, c, device="cuda")[:, None]
        j = torch.arange(c, device="cuda")[None]
        hidden = (j > i) | ((i - j >= case["window"]) if case["window"] else (j < 0))
        hidden &= j >= case["prefix"]
        rows = torch.empty((n, h, d), dtype=f64, device="cuda")
        for head in range(h):
            z = s["q"][t0:t0 + n, head].double() @ kv[0][head // g].t() / math.sqrt(d)
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
            if case["bias"]:
                z = z - s["slopes"][head].double() * (i - j).abs()
            z = z.masked_fill(hidden, -math.inf)
            rows[:, head] = torch.softmax(z, -1) @ kv[1][head // g]
        out.append(rows)
        t0 += n
    return torch.cat(out)
