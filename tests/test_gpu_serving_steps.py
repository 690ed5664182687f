"""The serving operators as a serving loop uses them, on the GPU: prompts are
rotated and appended, attended to, a second chunk follows, then single tokens
(append, decode), all over one paged cache whose blocks the block manager
hands out.  Every step's output is held to the 64-bit definition over what the
cache holds by then, and the cache to the appended rows."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_234_gb300 as pkv
import serving_reference as R
from gpu_common import dev, ensure_built

pytestmark = pytest.mark.gpu

HEADS, KV, DIM, BLOCKS, WIDTH = 8, 2, 64, 64, 20
SCALE = DIM ** -0.5


class Server:
    def __init__(self, kind, seqs, options):
        ensure_built()
        self.kind, self.options = kind, options
        self.bm = pkv.BlockManager(BLOCKS)
        self.tables = np.full((seqs, WIDTH), -1, np.int32)
        self.ctx = np.zeros(seqs, np.int32)
        shape = (BLOCKS, KV, 16, DIM)
        self.k = torch.zeros(shape, dtype=torch.float16, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.codes = []
        if kind != "fp16":
            t = torch.int8 if kind == "int8" else torch.uint8
            self.codes = [torch.zeros(shape, dtype=t, device="cuda") for _ in range(2)]
            self.codes += [torch.zeros(shape[:2], device="cuda") for _ in range(2)]
        self.table = pkv.rope_table(400, DIM)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.rng = np.random.default_rng(7)
        slopes = (2.0 ** -np.arange(1, HEADS + 1)).astype(np.float32)
        self.slopes = slopes if options.get("bias") else None
        self.mirror_k, self.mirror_v = (np.zeros(shape, np.float16) for _ in range(2))

    def grow(self, new):
        for s, n in enumerate(new):
            have, need = -(-int(self.ctx[s]) // 16), -(-int(self.ctx[s] + n) // 16)
            if need > have:
                self.tables[s, have:need] = self.bm.allocate(need - have)
        self.ctx = (self.ctx + new).astype(np.int32)

    def step(self, new):
        """new[s] tokens of every sequence: append, attend, check."""
        new = np.asarray(new, np.int32)
        self.grow(new)
        t = int(new.sum())
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        qkv = self.rng.standard_normal((t, HEADS + 2 * KV, DIM), dtype=np.float32).astype(np.float16)
        x = dev(qkv)
        q = torch.empty((t, HEADS, DIM), dtype=torch.float16, device="cuda")
        tables, lens, st = dev(self.tables), dev(self.ctx), dev(starts)
        getattr(pkv, "pkv_rope_append_" + self.kind)(
            q, self.k, self.v, *self.codes, x[:, :HEADS], x[:, HEADS:HEADS + KV],
            x[:, HEADS + KV:], self.table, st, lens, tables, dev_status=self.status)
        out = torch.empty_like(q)
        pools = (self.k, self.v) if self.kind == "fp16" else tuple(self.codes)
        kw = dict(logit_cap=self.options.get("cap", 0.0), window=self.options.get("window", 0),
                  slopes=None if self.slopes is None else dev(self.slopes),
                  dev_status=self.status)
        mcl = int(self.ctx.max())
        if np.all(new == 1):
            ws = pkv.decode_workspace(new.size, HEADS, KV, DIM, mcl)
            getattr(pkv, "pkv_paged_decode_scored_" + self.kind)(
                out, q, *pools, tables, lens, mcl, SCALE, ws, **kw)
        else:
            ws = pkv.prefill_workspace(t, new.size, HEADS, KV, DIM, mcl)
            getattr(pkv, "pkv_paged_prefill_" + self.kind)(
                out, q, *pools, tables, st, lens, mcl, SCALE, ws, **kw)
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        self.check(new, starts, qkv, q.cpu().numpy(), out.cpu().numpy().astype(np.float64))

    def check(self, new, starts, qkv, q, out):
        b = R.Batch(new, self.ctx, starts, self.tables, self.mirror_k, self.mirror_v, q, HEADS, KV,
                    DIM)
        want_q, self.mirror_k, self.mirror_v, written = R.rope_append(
            b, qkv, self.table.cpu().numpy(), None, None, False, (self.mirror_k, self.mirror_v))
        assert np.array_equal(q.view(np.uint16), want_q.view(np.uint16))
        for got, want in ((self.k, self.mirror_k), (self.v, self.mirror_v)):
            assert np.array_equal(got.cpu().numpy().view(np.uint16), want.view(np.uint16))
        b.k, b.v = self.mirror_k, self.mirror_v
        if self.kind == "fp16":
            kv64 = (b.k.astype(np.float64), b.v.astype(np.float64))
        else:
            kv64 = []
            for i, pool in ((0, b.k), (1, b.v)):
                c, s = self.codes[i].cpu().numpy(), self.codes[2 + i].cpu().numpy()
                wc, ws = R.quantize(pool[written], self.kind)
                assert np.array_equal(c[written], wc)
                assert np.array_equal(s[written].view(np.uint32), ws.view(np.uint32))
                val = R.e4m3(c) if self.kind == "fp8" else c.astype(np.float64)
                kv64.append(val * s[:, :, None, None].astype(np.float64))
        cap, window = self.options.get("cap", 0.0), self.options.get("window", 0)
        ref, mass = R.attend(b, kv64, SCALE, cap=cap, window=window, slopes=self.slopes)
        dz = R.score_error(b, self.kind, SCALE, cap, int(self.ctx.max()), self.slopes)
        tol = R.tolerance(ref, mass, dz, 11)
        assert np.max(np.abs(out - ref) / tol) <= 1.0


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("options", [{}, dict(cap=10.0, window=50), dict(bias=True)],
                         ids=["plain", "cap_window", "bias"])
def test_prompts_chunks_and_single_tokens(kind, options):
    srv = Server(kind, 3, options)
    srv.step([40, 7, 130])      # prompts
    srv.step([33, 1, 0])        # a second chunk, one token, none
    for _ in range(3):
        srv.step([1, 1, 1])     # decode steps, across a page border
    srv.step([5, 4, 1])         # drafted tokens beside a single one


def test_scored_decode_stays_inside_its_memory():
    # the debug build checks every shared-memory address and table index
    import ctypes
    ensure_built()
    L = pkv.debug_lib()
    flags = L.pkv_debug_scored_flags
    flags.restype, flags.argtypes = ctypes.c_uint, [ctypes.c_int]
    for kind in ("fp16", "int8", "fp8"):
        for heads, kv, dim, workers in ((8, 2, 64, 0), (20, 1, 128, 0), (8, 2, 128, 5)):
            b = R.make(3, [1] * 5, [1, 300, 17, 0, 128], heads, kv, dim)
            pools, _ = R.cache(b, kind)
            out = torch.empty(b.q.shape, dtype=torch.float16, device="cuda")
            ws = pkv.decode_workspace(5, heads, kv, dim, 300)
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            q, tables, lens = dev(b.q), dev(b.tables), dev(b.ctx)
            prefix = dev(np.asarray([5, 20, 0, 3, 40], np.int32))
            kv_t = [dev(x) for x in pools] + [None] * (4 - len(pools))
            name, args = pkv._scored("pkv_paged_decode_scored_" + kind, out, q, *kv_t, tables,
                                     lens, 300, dim ** -0.5, ws, 9.0, 100, None, prefix, status,
                                     None)
            L.pkv_set_decode_workers(workers)
            try:
                flags(1)
                assert getattr(L, name)(*args) == pkv.PKV_OK
                torch.cuda.synchronize()
            finally:
                L.pkv_set_decode_workers(0)
            assert flags(1) == 0 and int(status.item()) == 0
