"""Workloads of speculative decoding over the paged KV cache.

Three operators, one step of a serving loop that drafts a tree of tokens:

* tree:    attention of the drafted tokens, each over the cached context and its
           own ancestors in the tree, for fp16, INT8 and FP8 (E4M3) caches, with
           an optional tanh cap, distance bias, window and visible prefix;
* accept:  the walk from each tree's root along the tokens that the model
           answered with;
* compact: the rows of the tokens that stay, moved together in the paged cache
           (the accepted path of a tree, or what is left of a whole context),
           and for code caches the moved tiles' codes and scales.

``listed()`` names the measured cases and ``draw()`` gives further ones of the
same ranges.  ``run()`` makes one pass: the library's calls where ``own`` is
true, elementary torch operations otherwise.
"""
import math

import numpy as np
import torch

own = False

BS = 16          # tokens per block
VOCAB = 32000    # token ids of the accepted trees


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the smallest attention call: a small batch of small trees, where latency counts
        _tree("tree 8x8 over 512 int8", "int8", 8, 8, 512, (8, 8, 128)),
        # a serving batch with a tree of 16 tokens each
        _tree("tree 64x16 over 2048", "fp16", 64, 16, 2048, (32, 8, 128)),
        # small heads, a bias by distance, an odd number of tokens
        _tree("tree 32x25 over 2048 bias", "fp16", 32, 25, 2048, (14, 2, 64), bias=True),
        # a ragged batch that attends to a window and to the first tokens, FP8 cache
        _tree("tree ragged fp8 window", "fp8", 24, 60, 5000, (28, 4, 128), ragged=21, window=1024,
              prefix=64),
        # one long context, capped scores, INT8 cache
        _tree("tree 1x64 over 131072 int8 capped", "int8", 1, 64, 131072, (32, 8, 128), cap=30.0),
        # large trees over long contexts
        _tree("tree 16x64 over 8192", "fp16", 16, 64, 8192, (32, 8, 128)),
        # the walk through the trees of a small and of a very large batch
        _accept("accept 8x8", 8, 8),
        _accept("accept 4096x64", 4096, 64, ragged=22),
        # the accepted paths of a serving batch
        _compact("compact paths 64x16", "fp16", 64, 16, 2048, 5, (32, 8, 128)),
        # the accepted paths of ragged trees in an INT8 cache
        _compact("compact paths int8", "int8", 256, 60, 1500, 9, (28, 4, 128), ragged=23),
        # half of every context dropped
        _compact("compact 8x16384 half", "fp16", 8, 16384, 16384, 8192, (32, 8, 128)),
        # one long context in an FP8 cache, a quarter dropped
        _compact("compact 1x131072 fp8", "fp8", 1, 131072, 131072, 98304, (32, 8, 128)),
    ]


def _tree(name, kind, seqs, new, ctx, heads, ragged=0, cap=0.0, window=0, prefix=0, bias=False):
    c = {"op": "tree", "kind": kind, "seqs": seqs, "new": new, "ctx": ctx, "heads": heads[0],
         "kv_heads": heads[1], "dim": heads[2], "ragged": ragged, "cap": cap, "window": window,
         "prefix": prefix, "bias": bias}
    return dict(c, name=name) if name else c


def _accept(name, seqs, new, ragged=0):
    c = {"op": "accept", "kind": "ids", "seqs": seqs, "new": new, "ctx": new, "ragged": ragged}
    return dict(c, name=name) if name else c


def _compact(name, kind, seqs, new, ctx, keep, heads, ragged=0):
    # new: tokens of a sequence that may go (its last ones), keep: of them stay
    c = {"op": "compact", "kind": kind, "seqs": seqs, "new": new, "ctx": ctx, "keep": keep,
         "heads": heads[0], "kv_heads": heads[1], "dim": heads[2], "ragged": ragged}
    return dict(c, name=name) if name else c


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["tree", "tree", "accept", "compact"])
    kind = rng.choice(["fp16", "int8", "fp8"])
    ragged = rng.choice([0, rng.randrange(1, 1 << 20)])
    if op == "accept":
        return _accept("", log(1, 4096), log(1, 64), ragged)
    heads = rng.choice([(32, 8, 128), (14, 2, 64), (8, 8, 128), (28, 4, 128), (16, 1, 128),
                        (12, 4, 64)])
    if op == "tree":
        new = log(1, 128)
        total = log(1 << 12, 1 << 17)                    # tokens of all contexts
        seqs = log(1, 256)
        # the padded scores of the plain form: at most those of the largest case
        total = min(total, (1 << 28) // (new * heads[0]))
        seqs = max(1, min(seqs, total // (new + 16)))
        return _tree("", kind, seqs, new, max(new, total // seqs), heads, ragged,
                     rng.choice([0.0, 0.0, round(rng.uniform(10.0, 60.0), 1)]),
                     rng.choice([0, 0, log(16, 4096)]), rng.choice([0, 0, log(1, 1000)]),
                     rng.choice([False, False, True]))
    total = log(64, 131072)
    if rng.random() < 0.5:                               # accepted paths
        new = log(1, 128)
        seqs = max(1, min(256, total // new))
        ctx = new + log(1, 4096)
        return _compact("", kind, seqs, new, ctx, rng.randint(1, min(new, 12)), heads, ragged)
    seqs = log(1, 32)                                    # whole contexts
    ctx = max(1, total // seqs)
    return _compact("", kind, seqs, ctx, ctx, max(1, int(ctx * rng.uniform(0.1, 0.95))), heads,
                    ragged)


def _lengths(case):
    """New tokens and context lengths (with the new tokens) of the sequences."""
    n, new, ctx = case["seqs"], case["new"], case["ctx"]
    if not case["ragged"]:
        return np.full(n, new, np.int64), np.full(n, ctx, np.int64)
    r = np.random.RandomState(case["ragged"])
    q = r.randint(max(1, new // 8), new + 1, n)
    return q.astype(np.int64), (q + r.randint(0, ctx - new + 1, n)).astype(np.int64)


def _parents(case):
    """A drafted tree for every sequence: token 0 is the root, and the others
    hang on earlier ones, so that depths grow like a logarithm."""
    q, _ = _lengths(case)
    r = np.random.RandomState(case["ragged"] + 1)
    i = np.concatenate([np.arange(n) for n in q.tolist()])
    low, high = (i - 1) // 3, (i + 1) // 2
    p = low + (r.rand(len(i)) * np.maximum(high - low, 1)).astype(np.int64)
    return np.where(i == 0, -1, np.minimum(np.maximum(p, 0), i - 1)).astype(np.int32)


def _ancestors(parents):
    """bool [n][n]: whether token j is token i or one of its ancestors."""
    n = len(parents)
    a = np.zeros((n, n), bool)
    for i, p in enumerate(parents.tolist()):
        if p >= 0:
            a[i] = a[p]
        a[i, i] = True
    return a


def _kept_counts(case):
    """Tokens of each sequence that stay."""
    q, _ = _lengths(case)
    return np.maximum(1, np.minimum(q, q * case["keep"] // case["new"]))


def work(case):
    q, ctx = _lengths(case)
    t = int(q.sum())
    if case["op"] == "accept":
        # token, answer and parent in, the path out, and two numbers a tree
        return {"bytes": 16 * t + 12 * case["seqs"], "flops": 0}
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    elem = 2 if case["kind"] == "fp16" else 1
    if case["op"] == "compact":
        m = _kept_counts(case)
        rows = int(m.sum())
        bytes_ = rows * hk * 2 * d * 2 * 2 + 4 * rows
        if case["kind"] != "fp16":
            # the written tiles' codes and scales, and the rows that were there before
            base = ctx - q
            tiles = int(((base + m - 1) // BS - base // BS + 1).sum())
            bytes_ += tiles * hk * 2 * (BS * d + 4) + (tiles * BS - rows) * hk * 2 * d * 2
        return {"bytes": bytes_, "flops": 0}
    parents, pairs, keys, t0 = _parents(case), 0, 0, 0
    for n, c in zip(q.tolist(), ctx.tolist()):
        a = _ancestors(parents[t0:t0 + n])
        depth = a.sum(1) - 1
        base, pre = c - n, min(case["prefix"], c - n)
        w = case["window"] or c + 1
        lo = np.clip(base + depth - w + 1, 0, base)     # context from here on, and below pre
        pairs += int((base - lo + np.minimum(pre, lo)).sum())
        pairs += int((a & (depth[:, None] - depth[None] < w)).sum())
        keys += n + base - int(lo.min()) + min(pre, int(lo.min()))
        t0 += n
    bytes_ = 2 * t * h * d * 2 + 4 * t + keys * hk * 2 * d * elem + keys // BS * 4
    if case["kind"] != "fp16":
        bytes_ += keys // BS * hk * 2 * 4
    return {"bytes": bytes_, "flops": 4 * d * h * pairs}


# ------------------------------------------------------------------ the inputs
def _codes(kind, x):
    """Codes and per-(block, kv head) scales of fp16 tiles [n][Hkv][16][d]."""
    f = x.float()
    most = torch.tensor(127.0 if kind == "int8" else 448.0, device=x.device)
    scale = f.abs().amax(dim=(2, 3)) / most
    y = torch.nan_to_num(f / scale[:, :, None, None], nan=0.0)
    y = torch.minimum(torch.maximum(y, -most), most)
    if kind == "int8":
        return y.round().to(torch.int8), scale
    return y.to(torch.float8_e4m3fn).view(torch.uint8), scale


def _normal(shape, gen, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16).mul_(std)


def prepare(case, seed):
    q, ctx = _lengths(case)
    n, t = case["seqs"], int(q.sum())
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = np.random.RandomState(seed)
    starts = np.concatenate([[0], np.cumsum(q)])
    s = {"case": case, "seqs": n, "tokens": t,
         "starts": torch.from_numpy(starts.astype(np.int32)).cuda(),
         "lens": torch.from_numpy(ctx.astype(np.int32)).cuda(),
         "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if case["op"] == "accept":
        # drafted tokens, and answers that follow one child of most tokens
        p = _parents(case)
        ids, answers = rand.randint(0, VOCAB, t), rand.randint(0, VOCAB, t)
        up = np.repeat(starts[:-1], q) + p
        right = np.flatnonzero((p >= 0) & (rand.rand(t) < 0.7))
        answers[up[right]] = ids[right]
        for name, x in (("parents", p), ("ids", ids), ("answers", answers)):
            s[name] = torch.from_numpy(x.astype(np.int32)).cuda()
        return s
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    pages = (ctx + BS - 1) // BS
    blocks = int(pages.sum()) + 7
    # the sequences' blocks lie anywhere in the pool; unused table entries -1
    perm = torch.randperm(blocks, generator=gen, device="cuda", dtype=torch.int32)
    width = int(pages.max())
    used = torch.from_numpy(np.arange(width)[None, :] < pages[:, None]).cuda()
    s["tables"] = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    s["tables"][used] = perm[: int(pages.sum())]
    k, v = _normal((blocks, hk, BS, d), gen), _normal((blocks, hk, BS, d), gen)
    if case["op"] == "compact":
        kept = np.full(t, -1, np.int32)
        counts = _kept_counts(case)
        for b, (m, c) in enumerate(zip(q.tolist(), counts.tolist())):
            # the first token of a path is the root; a context loses any of its own
            pick = np.zeros(m, bool)
            pick[rand.permutation(m)[:c]] = True
            if case["new"] < case["ctx"] and not pick[0]:
                pick[np.flatnonzero(pick)[0]], pick[0] = False, True
            kept[starts[b]:starts[b] + c] = np.flatnonzero(pick)
        s["kept"] = torch.from_numpy(kept).cuda()
        s["kept_lens"] = torch.from_numpy(counts.astype(np.int32)).cuda()
        s["k"], s["v"] = k, v
        if case["kind"] != "fp16":
            for x in "kv":
                s[x + "_codes"], s[x + "_scales"] = _codes(case["kind"], s[x])
        return s
    s["max_ctx"], s["max_new"] = int(ctx.max()), int(q.max())
    s["parents"] = torch.from_numpy(_parents(case)).cuda()
    # slots behind a sequence's last token hold whatever was there before
    rest = torch.from_numpy((pages * BS - ctx).astype(np.int64)).cuda()
    last = s["tables"].gather(1, torch.from_numpy(pages - 1)[:, None].cuda())[:, 0].long()
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


# ------------------------------------------------------------------- one pass
def run(state):
    if own:
        return _run_own(state)
    return {"tree": _plain_tree, "accept": _plain_accept,
            "compact": _plain_compact}[state["case"]["op"]](state)


def _run_own(s):
    import paged_kv_cache_234_gb300 as pkv

    c = s["case"]
    if "call" not in s:
        # a serving loop keeps its output buffers and its prepared call, and
        # updates the inputs in place from step to step
        if c["op"] == "accept":
            s["kept"] = torch.empty(s["tokens"], dtype=torch.int32, device="cuda")
            s["kept_lens"] = torch.empty(s["seqs"], dtype=torch.int32, device="cuda")
            s["next"] = torch.empty(s["seqs"], dtype=torch.int32, device="cuda")
            s["call"] = pkv.prepare_tree_accept(s["kept"], s["kept_lens"], s["next"], s["ids"],
                                                s["answers"], s["parents"], s["starts"],
                                                dev_status=s["status"])
        elif c["op"] == "compact":
            s["new_lens"] = torch.empty_like(s["lens"])
            codes = [s[n] for n in ("k_codes", "v_codes", "k_scales", "v_scales")
                     if c["kind"] != "fp16"]
            make = getattr(pkv, "prepare_compact_" + c["kind"])
            s["call"] = make(s["k"], s["v"], *codes, s["kept"], s["kept_lens"], s["new_lens"],
                             s["starts"], s["lens"], s["tables"], dev_status=s["status"])
        else:
            h, hk, d = c["heads"], c["kv_heads"], c["dim"]
            s["out"] = torch.empty_like(s["q"])
            kv = [s["k"], s["v"]]
            kv += [s["k_scales"], s["v_scales"]] if c["kind"] != "fp16" else []
            ws = pkv.tree_workspace(s["tokens"], s["seqs"], h, hk, d, s["max_ctx"], s["max_new"])
            make = getattr(pkv, "prepare_paged_tree_" + c["kind"])
            s["call"] = make(s["out"], s["q"], *kv, s["tables"], s["starts"], s["lens"],
                             s["parents"], s["max_ctx"], s["max_new"], d ** -0.5, ws,
                             logit_cap=c["cap"], window=c["window"], slopes=s["slopes"],
                             prefix_lens=s["prefix"], dev_status=s["status"])
    s["call"]()
    if c["op"] == "accept":
        return {"kept": s["kept"], "kept_lens": s["kept_lens"], "next": s["next"]}
    if c["op"] == "compact":
        return _compact_outputs(s, s["new_lens"])
    return s["out"]


def _compact_outputs(s, new_lens):
    out = {"lens": new_lens, "k": s["k"], "v": s["v"]}
    if s["case"]["kind"] != "fp16":
        # codes and scales: codes * scales are the values that the cache holds
        out.update({n: s[n] for n in ("k_codes", "v_codes", "k_scales", "v_scales")})
    return out


def _token_map(s):
    """Sequence and row of every token of the batch."""
    starts = s["starts"].long()
    token = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(starts, token, right=True) - 1
    return seq, token - starts[seq]


def _plain_accept(s):
    seq, row = _token_map(s)
    n, t = s["seqs"], s["tokens"]
    starts = s["starts"].long()
    here = torch.zeros(n, dtype=torch.long, device="cuda")      # the walk's token, by its row
    lens = torch.ones_like(here)
    kept = torch.full((t,), -1, dtype=torch.int32, device="cuda")
    kept[starts[:-1]] = 0
    ids, answers = s["ids"], s["answers"]
    parents = s["parents"].long()
    for _ in range(s["case"]["new"] - 1):
        fits = (parents == here[seq]) & (ids == answers[starts[:-1] + here][seq])
        first = torch.full((n,), t, dtype=torch.long, device="cuda")
        first = first.scatter_reduce(0, seq, torch.where(fits, row, t), "amin")
        on = first < t
        at = starts[:-1] + lens
        kept[at[on]] = first[on].int()
        here, lens = torch.where(on, first, here), lens + on
    return {"kept": kept, "kept_lens": lens.int(), "next": answers[starts[:-1] + here]}


def _plain_compact(s):
    seq, row = _token_map(s)
    lens, starts = s["lens"].long(), s["starts"].long()
    base = lens - (starts[1:] - starts[:-1])
    stays = row < s["kept_lens"].long()[seq]
    seq, row, source = seq[stays], row[stays], s["kept"].long()[stays]
    moves = source != row
    seq, row, source = seq[moves], base[seq[moves]] + row[moves], base[seq[moves]] + source[moves]
    to = s["tables"][seq, row // BS].long()
    of = s["tables"][seq, source // BS].long()
    for n in "kv":
        s[n][to, :, row % BS] = s[n][of, :, source % BS]
    if s["case"]["kind"] != "fp16":
        block = torch.unique(to)
        for n in "kv":
            s[n + "_codes"][block], s[n + "_scales"][block] = _codes(s["case"]["kind"], s[n][block])
    return _compact_outputs(s, (base + s["kept_lens"].long()).int())


def _values(s, name, block):
    """The fp32 values [...][Hkv][16][d] of the pool's blocks."""
    x = s[name][block]
    if s["case"]["kind"] == "fp16":
        return x.float()
    if s["case"]["kind"] == "fp8":
        x = x.view(torch.float8_e4m3fn)
    return x.float() * s[name + "_scales"][block][..., None, None]


def _plain_tree(s):
    c = s["case"]
    n, h, hk, d, g = s["seqs"], c["heads"], c["kv_heads"], c["dim"], c["heads"] // c["kv_heads"]
    seq, row = _token_map(s)
    lens, m = s["lens"].long(), s["max_new"]
    count = (s["starts"][1:] - s["starts"][:-1]).long()
    base = lens - count
    q = torch.zeros((n, m, h, d), device="cuda")
    q[seq, row] = s["q"].float()
    q = q.view(n, m, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, g * m, d)
    # tokens and their ancestors: the closure of "is my parent", by squaring
    tree = torch.eye(m, device="cuda").repeat(n, 1, 1)
    has = s["parents"] >= 0
    tree[seq[has], row[has], s["parents"].long()[has]] = 1.0
    for _ in range(max(1, m - 1).bit_length()):
        tree = (tree @ tree).clamp_(max=1.0)
    depth = tree.sum(-1).long() - 1                                        # [n][m]
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
    # a cached key's row in the tree, or one that is none of it; its position
    node = (key[None, :] - base[:, None]).clamp(0, m - 1)
    drafted = (key[None, :] >= base[:, None]) & held
    at = torch.where(drafted, base[:, None] + depth.gather(1, node), key[None, :])
    gap = (base[:, None] + depth)[:, :, None] - at[:, None, :]             # [n][m][keys]
    if s["slopes"] is not None:
        z -= s["slopes"].view(hk, g, 1, 1) * gap[:, None, None]
    near = gap < c["window"] if c["window"] else torch.ones_like(gap, dtype=torch.bool)
    context = near
    if s["prefix"] is not None:
        context = near | (key[None, None, :] < s["prefix"].long()[:, None, None])
    above = tree.gather(2, node[:, None, :].expand(n, m, -1)) > 0
    seen = torch.where(drafted[:, None, :], above & near, context) & held[:, None, :]
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
    starts = np.concatenate([[0], np.cumsum(q_lens)])
    if case["op"] == "accept":
        return _exact_accept(s, starts)
    if case["op"] == "compact":
        return _exact_compact(s, case, starts, q_lens, ctx)
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    g = h // hk
    if 4 * d * h * float((q_lens * ctx).sum()) > 4e12:
        return None
    parents, out = s["parents"].cpu().numpy(), []
    for b, (n, c) in enumerate(zip(q_lens.tolist(), ctx.tolist())):
        blk = s["tables"][b, :(c + BS - 1) // BS].long()
        kv = []
        for name in "kv":
            x = s[name][blk]
            x = x.view(torch.float8_e4m3fn).float().double() if case["kind"] == "fp8" else x.double()
            if case["kind"] != "fp16":
                x = x * s[name + "_scales"][blk].double()[:, :, None, None]
            kv.append(x.transpose(0, 1).reshape(hk, -1, d)[:, :c])
        up = torch.from_numpy(_ancestors(parents[starts[b]:starts[b] + n])).cuda()
        place = torch.arange(c, device="cuda")
        place[c - n:] = c - n + up.sum(1) - 1
        gap = place[c - n:, None] - place[None]
        hidden = gap >= (case["window"] or c + 1)
        hidden[:, :min(case["prefix"], c - n)] = False
        hidden[:, c - n:] |= ~up
        rows = torch.empty((n, h, d), dtype=torch.float64, device="cuda")
        for head in range(h):
            z = s["q"][starts[b]:starts[b] + n, head].double() @ kv[0][head // g].t() / math.sqrt(d)
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
            if case["bias"]:
                z = z - s["slopes"][head].double() * gap
            rows[:, head] = torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ kv[1][head // g]
        out.append(rows)
    return torch.cat(out)


def _exact_accept(s, starts):
    p, ids, answers = (s[n].cpu().tolist() for n in ("parents", "ids", "answers"))
    kept, lens, last = np.full(s["tokens"], -1, np.int32), [], []
    for a, b in zip(starts[:-1].tolist(), starts[1:].tolist()):
        path = [0]
        for j in range(1, b - a):
            if p[a + j] == path[-1] and ids[a + j] == answers[a + path[-1]]:
                path.append(j)
        kept[a:a + len(path)] = path
        lens.append(len(path))
        last.append(answers[a + path[-1]])
    return {n: torch.from_numpy(np.asarray(x, np.int32)).cuda()
            for n, x in (("kept", kept), ("kept_lens", lens), ("next", last))}


def _exact_compact(s, case, starts, q_lens, ctx):
    kept, counts = s["kept"].cpu().numpy(), s["kept_lens"].cpu().numpy()
    k, v = s["k"].clone(), s["v"].clone()
    lens = []
    for b, (n, c) in enumerate(zip(q_lens.tolist(), ctx.tolist())):
        m = int(counts[b])
        lens.append(c - n + m)
        j = torch.arange(m, device="cuda") + (c - n)
        i = torch.from_numpy(kept[starts[b]:starts[b] + m].astype(np.int64)).cuda() + (c - n)
        table = s["tables"][b].long()
        for new, old in ((k, s["k"]), (v, s["v"])):
            new[table[j // BS], :, j % BS] = old[table[i // BS], :, i % BS]
    out = {"lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "k": k.double(),
           "v": v.double()}
    if case["kind"] != "fp16":
        out.update(k_codes=None, v_codes=None, k_scales=None, v_scales=None)
    return out
