"""A speculative serving loop on the GPU: prompts, then steps that append a tree of
drafted tokens (rotated to their depths), attend, walk along the model's answers
and move the accepted rows together.  After every step the cache holds what
appending the accepted tokens one by one would have put there."""
import numpy as np
import pytest
import torch

import paged_kv_cache_234_gb300 as pkv
import serving_reference as R
import tree_reference as T
from gpu_common import dev, ensure_built

pytestmark = pytest.mark.gpu

HEADS, KV, DIM, BLOCKS, WIDTH, VOCAB = 8, 2, 64, 64, 24, 40
SCALE = DIM ** -0.5


class Server:
    def __init__(self, kind, seqs, options):
        ensure_built()
        self.kind, self.options, self.seqs = kind, options, seqs
        self.tables = np.random.default_rng(3).permutation(BLOCKS)[:seqs * 20].reshape(seqs, 20)
        self.tables = self.tables.astype(np.int32)
        self.ctx = np.zeros(seqs, np.int32)
        shape = (BLOCKS, KV, 16, DIM)
        self.k = torch.zeros(shape, dtype=torch.float16, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.codes = []
        if kind != "fp16":
            t = torch.int8 if kind == "int8" else torch.uint8
            self.codes = [torch.zeros(shape, dtype=t, device="cuda") for _ in "kv"]
            self.codes += [torch.zeros(shape[:2], device="cuda") for _ in "kv"]
        self.table = pkv.rope_table(400, DIM)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.rng = np.random.default_rng(7)
        self.rows = [[] for _ in range(seqs)]    # (K, V) rows of every token, as they should be

    def append(self, new, positions):
        self.ctx = (self.ctx + new).astype(np.int32)
        t = int(new.sum())
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        qkv = self.rng.standard_normal((t, HEADS + 2 * KV, DIM), dtype=np.float32).astype(np.float16)
        x = dev(qkv)
        self.q = torch.empty((t, HEADS, DIM), dtype=torch.float16, device="cuda")
        self.dev = dict(st=dev(self.starts), lens=dev(self.ctx), tables=dev(self.tables))
        getattr(pkv, "pkv_rope_append_" + self.kind)(
            self.q, self.k, self.v, *self.codes, x[:, :HEADS], x[:, HEADS:HEADS + KV],
            x[:, HEADS + KV:], self.table, self.dev["st"], self.dev["lens"], self.dev["tables"],
            rope_positions=dev(positions.astype(np.int32)), dev_status=self.status)
        tab = self.table.cpu().numpy()[positions]
        k = R.rotate32(qkv[:, HEADS:HEADS + KV], tab[:, None, :DIM // 2], tab[:, None, DIM // 2:],
                       False)
        return k, qkv[:, HEADS + KV:]

    def prompts(self, new):
        new = np.asarray(new, np.int32)
        positions = np.concatenate([np.arange(n) for n in new])
        k, v = self.append(new, positions)
        for s in range(self.seqs):
            a, e = self.starts[s], self.starts[s + 1]
            self.rows[s] = list(zip(k[a:e], v[a:e]))

    def draft(self, new, seed):
        """One speculative step with trees of new[s] tokens."""
        new = np.asarray(new, np.int32)
        old = self.ctx.copy()
        parents = T.trees(seed, new)
        starts = np.concatenate([[0], np.cumsum(new)])
        depth = np.concatenate([[len(T.path_to(parents[a:e], r)) - 1 for r in range(e - a)]
                                for a, e in zip(starts[:-1], starts[1:])]).astype(np.int64)
        k, v = self.append(new, np.repeat(old, new) + depth)
        t, n, mcl = int(new.sum()), self.seqs, int(self.ctx.max())
        ws = pkv.tree_workspace(t, n, HEADS, KV, DIM, mcl, int(new.max()))
        out = torch.empty_like(self.q)
        pools = (self.k, self.v) if self.kind == "fp16" else tuple(self.codes)
        d, up = self.dev, dev(parents)
        cap, window = self.options.get("cap", 0.0), self.options.get("window", 0)
        getattr(pkv, "pkv_paged_tree_" + self.kind)(
            out, self.q, *pools, d["tables"], d["st"], d["lens"], up, mcl, int(new.max()), SCALE,
            ws, logit_cap=cap, window=window, dev_status=self.status)
        before = [x.cpu().numpy().copy() for x in (self.k, self.v, *self.codes)]
        # the model's answers: one child of most tokens is the right one
        tokens = self.rng.integers(0, VOCAB, t).astype(np.int32)
        targets = self.rng.integers(0, VOCAB, t).astype(np.int32)
        right = np.flatnonzero((parents >= 0) & (self.rng.random(t) < 0.8))
        targets[(np.repeat(starts[:-1], new) + parents)[right]] = tokens[right]
        kept = torch.empty(t, dtype=torch.int32, device="cuda")
        kept_lens, last, lens = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(3))
        pkv.pkv_tree_accept(kept, kept_lens, last, dev(tokens), dev(targets), up, d["st"],
                            dev_status=self.status)
        getattr(pkv, "pkv_compact_" + self.kind)(
            self.k, self.v, *self.codes, kept, kept_lens, lens, d["st"], d["lens"], d["tables"],
            dev_status=self.status)
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        # the attention, over what the cache held
        b = R.Batch(new, self.ctx, self.starts, self.tables, before[0], before[1],
                    self.q.cpu().numpy(), HEADS, KV, DIM)
        kv64 = [x.astype(np.float64) for x in before[:2]]
        if self.kind != "fp16":
            kv64 = [(R.e4m3(c) if self.kind == "fp8" else c.astype(np.float64)) *
                    s[:, :, None, None].astype(np.float64)
                    for c, s in zip(before[2:4], before[4:6])]
        o = dict(cap=cap, window=window, slopes=None)
        ref, mass = T.attend(b, parents, kv64, SCALE, **o)
        got = out.cpu().numpy().astype(np.float64)
        assert np.max(np.abs(got - ref) / T.bound(b, o, ref, mass, SCALE)) <= 1.0
        # the path, and the cache behind it
        want = T.accept(parents, tokens, targets, self.starts)
        for x, y in zip((kept, kept_lens, last), want):
            assert np.array_equal(x.cpu().numpy(), y)
        self.ctx = (old + want[1]).astype(np.int32)
        assert np.array_equal(lens.cpu().numpy(), self.ctx)
        for s in range(self.seqs):
            path = self.starts[s] + want[0][self.starts[s]:self.starts[s] + want[1][s]]
            self.rows[s] += [(k[i], v[i]) for i in path]
        self.check_cache()
        return want[1]

    def check_cache(self):
        k, v = self.k.cpu().numpy(), self.v.cpu().numpy()
        for s in range(self.seqs):
            for t, (kr, vr) in enumerate(self.rows[s]):
                at = (self.tables[s, t // 16], slice(None), t % 16)
                assert np.array_equal(k[at].view(np.uint16), kr.view(np.uint16))
                assert np.array_equal(v[at].view(np.uint16), vr.view(np.uint16))
        if self.kind != "fp16":
            # the code tiles stand for the fp16 tiles: half a step of INT8, 2^-4 of an
            # E4M3 value or half its smallest step, and the scale's own rounding
            used = np.unique(np.concatenate([self.tables[s, :-(-int(self.ctx[s]) // 16)]
                                             for s in range(self.seqs)]))
            for i, x in ((0, k), (1, v)):
                c, sc = self.codes[i].cpu().numpy()[used], self.codes[2 + i].cpu().numpy()[used]
                sc = sc[:, :, None, None].astype(np.float64)
                x = x[used].astype(np.float64)
                if self.kind == "int8":
                    assert np.all(np.abs(c * sc - x) <= sc * (0.5 + 2.0 ** -15))
                else:
                    step = np.maximum(np.abs(x) * 2.0 ** -4, sc * 2.0 ** -10)
                    assert np.all(np.abs(R.e4m3(c) * sc - x) <= step * (1 + 2.0 ** -15))


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("options", [{}, dict(cap=10.0, window=50)], ids=["plain", "cap_window"])
def test_speculative_steps(kind, options):
    srv = Server(kind, 3, options)
    srv.prompts([40, 7, 130])
    moved = 0
    for step, new in enumerate(([8, 8, 8], [20, 1, 33], [5, 16, 9], [12, 12, 12])):
        moved += int(srv.draft(new, step).sum())
    assert moved > 12    # (roots alone would be 12)
