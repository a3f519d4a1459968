"""The latent-cache operators as a forward pass uses them together: a turn's
tokens appended and attended in the expanded form, completed pages offloaded
and their device copies dropped, then a decode step -- rows appended, the
selected ones resolved (host copies among them), sparse attention over the
resolved rows and dense attention through the block table -- eagerly, captured
into a graph, and on two streams.  Bounds: those of each operator's own tests
(see there); the query rotation's rounding does not enter, the oracle attends
with the rotated queries read back."""

from __future__ import annotations

import os

import numpy as np
import pytest
import torch

from oracle import latent as ol
from oracle import sparse_mla as sm
from test_gpu_latent_decode import bits, bound, compare, dev, f64
from test_gpu_prefill import check as check_prefill

pytestmark = pytest.mark.gpu
FREQ = 10000.0 ** (-np.arange(32) / 32)
PAGE, PAGES, R, L, P, K, H, C = 64, 7, 3, 2, 2, 96, 16, 256
SCALE = 0.06


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import serving_memory_tier_amd as hs
    if not os.path.exists(hs.LIB_PATH):
        from serving_memory_tier_amd import build
        build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    hs.lib()


class Serving:
    """Three requests: a turn of `turn` tokens, then a decode step of P tokens."""

    def __init__(self, fmt, seed=11):
        import serving_memory_tier_amd as hs
        self.hs, self.fmt = hs, fmt
        rs = self.rs = np.random.default_rng(seed)
        self.turn = np.array([400, 130, 64], np.int32)
        self.ctx = self.turn + P
        lat, kr = bits(rs, R, PAGES * PAGE, 512), bits(rs, R, PAGES * PAGE, 64)
        self.lat, self.kr = lat, kr
        t = np.arange(PAGES * PAGE)
        # the row of every token, as the oracle builds it
        self.logical = np.stack([ol.encode_rows(lat[r], ol.to_bf16(
            ol.rotate(sm.bf16_to_float(kr[r]), t, FREQ, True)), fmt) for r in range(R)])
        blocks = R * PAGES + R * C // PAGE + 3
        order = rs.permutation(blocks)
        self.bt = order[:R * PAGES].reshape(R, PAGES).astype(np.int32)
        hot = order[R * PAGES:R * PAGES + R * C // PAGE].reshape(R, -1).astype(np.int32)
        self.rows, self.host_blocks = blocks * PAGE, R * PAGES
        self.lay = hs.layout_of(PAGE, fmt, L, C, self.rows, self.host_blocks * PAGE)
        self.host = hs.HostPool(L * self.host_blocks * PAGE * fmt)
        self.host.array[:] = 0xFF
        self.pool = torch.full((L, self.rows, fmt), 255, dtype=torch.uint8, device="cuda")
        self.gbt, self.ghbt = dev(self.bt), dev(np.full((R, PAGES), -1, np.int32))
        self.gctx, self.hot = dev(self.turn.copy()), dev(hot)
        self.tok = torch.full((R, L, C), -1, dtype=torch.int32, device="cuda")
        self.stp = torch.zeros((R, L, C), dtype=torch.int32, device="cuda")
        self.batch = hs.batch_of(R, PAGES, self.pool, self.host, self.gbt, self.ghbt, self.gctx,
                                 self.hot, self.tok, self.stp)

    def append(self, layer, req, pos, q_rope, q_out, row_ids=None, stream=None):
        r, n = np.asarray(req, np.int32), np.asarray(pos, np.int32)
        call = self.hs.append_of(len(r), dev(r), dev(n), dev(self.lat[r, n]), dev(self.kr[r, n]),
                                 dev(FREQ), True, q_rope, q_out)
        self.hs.hs_mla_append(self.lay, self.batch, layer, call, row_ids, None, stream)
        return call

    def prompt(self):
        """The turn's rows into both layers and its attention in layer 1."""
        hs, rs = self.hs, self.rs
        req = np.repeat(np.arange(R), self.turn)
        pos = np.concatenate([np.arange(n) for n in self.turn])
        N = len(req)
        q = dev(bits(rs, N, H, 192))
        raw = q[:, :, 128:].clone()
        for layer in range(L):
            self.append(layer, req, pos, raw, q[:, :, 128:])
        start = np.concatenate([[0], np.cumsum(self.turn)]).astype(np.int32)
        w = bits(rs, H, 256, 512, mult=0.05)
        out = torch.empty((N, H, 128), dtype=torch.int16, device="cuda")
        ws = torch.empty(hs.hs_mla_prefill_workspace_bytes(R, N, N, H), dtype=torch.uint8,
                         device="cuda")
        print(f"[prompt] fmt={self.fmt} N={N}", flush=True)
        hs.hs_mla_prefill(self.lay, self.batch, 1, dev(start), N, N, q, H, dev(w), SCALE, out, ws)
        torch.cuda.synchronize()
        pool = np.full((self.rows, self.fmt), 255, np.uint8)
        for r in range(R):
            t = np.arange(self.turn[r])
            pool[self.bt[r, t // PAGE].astype(np.int64) * PAGE + t % PAGE] = self.logical[r, t]
        got = self.pool.cpu().numpy()
        assert (got == pool[None]).all()
        check_prefill(f64(out), pool, self.bt, self.turn, start,
                      q.cpu().numpy().view(np.uint16), w, PAGE, SCALE)

    def offload(self):
        """All complete pages but each request's first: to the host, then dropped."""
        gone = [(r, j) for r in range(R) for j in range(1, self.turn[r] // PAGE)]
        pairs = np.array([(self.bt[r, j], i) for i, (r, j) in enumerate(gone)], np.int32)
        self.hs.hs_offload_prefix_pages(self.lay, self.pool, self.host, dev(pairs), len(pairs))
        torch.cuda.synchronize()
        hbt = np.full((R, PAGES), -1, np.int32)
        for i, (r, j) in enumerate(gone):
            blk = int(self.bt[r, j])
            self.pool[:, blk * PAGE:(blk + 1) * PAGE] = 255        # whoever reads it gets NaN
            self.bt[r, j], hbt[r, j] = -1, i
        self.gbt.copy_(dev(self.bt))
        self.ghbt.copy_(dev(hbt))
        self.gctx.copy_(dev(self.ctx))
        assert len(gone) > 4

    def buffers(self):
        """The decode step's operands, made once as a serving loop does."""
        hs, rs = self.hs, self.rs
        topk = np.full((R, L, P, K), -1, np.int32)
        for r in range(R):
            for p in range(P):
                n = int(min(K - 3, self.ctx[r] - P + p + 1))
                topk[r, :, p, :n] = rs.permutation(self.ctx[r] - P + p + 1)[:n]
        q = bits(rs, R, P, H, 576)
        g = dict(topk=dev(topk), q0=dev(q), q=dev(q),
                 ids=torch.empty((R, L, P, K), dtype=torch.int32, device="cuda"),
                 one=torch.empty((R, P, K), dtype=torch.int32, device="cuda"),
                 staging=torch.empty((R, L, P, K, self.fmt), dtype=torch.uint8, device="cuda"),
                 stats=torch.empty((R, L, 8), dtype=torch.int32, device="cuda"),
                 lse=torch.empty((R, P, H), device="cuda"),
                 out=torch.empty((R, P, H, 512), device="cuda",
                                 dtype=torch.int16 if self.fmt == 400 else torch.float32),
                 dense=torch.empty((R, P, H, 512), dtype=torch.int16, device="cuda"),
                 dlse=torch.empty((R, P, H), device="cuda"),
                 new=torch.empty((R * P,), dtype=torch.int32, device="cuda"))
        g["topk_host"] = topk
        size = (hs.hs_sparse_mla_fp4_workspace_bytes if self.fmt == 400 else
                hs.hs_sparse_mla_workspace_bytes)
        g["ws"] = torch.empty(max(size(R * P, H, K), 16), dtype=torch.uint8, device="cuda")
        self.max_ctx = PAGES * PAGE
        g["dws"] = torch.empty(max(hs.hs_paged_mla_workspace_bytes(R, P, H, self.max_ctx), 16),
                               dtype=torch.uint8, device="cuda")
        req = np.repeat(np.arange(R), P).astype(np.int32)
        pos = (self.ctx[:, None] - P + np.arange(P)).reshape(-1).astype(np.int32)
        g["call"] = hs.append_of(R * P, dev(req), dev(pos), dev(self.lat[req, pos]),
                                 dev(self.kr[req, pos]), dev(FREQ), True,
                                 g["q0"].view(R * P, H, 576)[:, :, 512:],
                                 g["q"].view(R * P, H, 576)[:, :, 512:])
        self.g = g

    def step(self, stream=None):
        """One decode step: layer 1 sparse, layer 0 dense."""
        hs, g = self.hs, self.g
        for layer in range(L):
            hs.hs_mla_append(self.lay, self.batch, layer, g["call"], g["new"], None, stream)
        hs.hs_resolve_in_place(self.lay, self.batch, g["topk"], P, K, 5, g["ids"], g["staging"],
                               g["stats"], None, 0, stream)
        g["one"].copy_(g["ids"][:, 1])
        attend = hs.hs_sparse_mla_decode_fp4 if self.fmt == 400 else hs.hs_sparse_mla_decode
        attend(self.lay, self.pool[1], g["one"], R * P, K, g["q"], H, SCALE, g["out"], g["lse"],
               g["ws"], stream)
        hs.hs_paged_mla_decode(self.lay, self.batch, 0, g["q"], P, H, self.max_ctx, SCALE,
                               g["dense"], g["dlse"], g["dws"], stream)

    def results(self):
        torch.cuda.synchronize()
        return {k: self.g[k].clone() for k in ("ids", "out", "lse", "dense", "dlse", "q", "new",
                                               "stats")}

    def check_step(self):
        g = self.results()
        q = g["q"].cpu().numpy().view(np.uint16)
        out = f64(g["out"]) if self.fmt == 400 else g["out"].cpu().numpy().astype(np.float64)
        lse, dlse = (g[k].cpu().numpy().astype(np.float64) for k in ("lse", "dlse"))
        dense, topk = f64(g["dense"]), self.g["topk_host"]
        assert (g["stats"][:, :, 2] > 0).any() and (g["stats"][:, :, 3:5] == 0).all()
        for r in range(R):
            ref, refl = ol.sparse_mla_decode(self.logical[r], topk[r, 1], q[r], SCALE)
            for p in range(P):
                ids = topk[r, 1, p]
                seen = np.broadcast_to(ids >= 0, (H, K))
                tol, toll = bound(sm.bf16_to_float(q[r, p]), ids, self.logical[r], seen, SCALE,
                                  ref[p], refl[p])
                compare(out[r, p], lse[r, p], ref[p], refl[p], tol, toll, ("sparse", r, p))
            # the dense layer sees what is resident
            t = np.arange(self.ctx[r])
            ids = np.where(self.bt[r, t // PAGE] >= 0, t, -1)
            k, v = ol.decode_rows(self.logical[r, t])
            for p in range(P):
                seen = np.broadcast_to((ids >= 0) & (t <= self.ctx[r] - P + p), (H, len(t)))
                ref, refl = ol.attend(sm.bf16_to_float(q[r, p]), k, v, seen, SCALE)
                tol, toll = bound(sm.bf16_to_float(q[r, p]), ids, self.logical[r], seen, SCALE,
                                  ref, refl)
                compare(dense[r, p], dlse[r, p], ref, refl, tol, toll, ("dense", r, p))


@pytest.mark.parametrize("fmt", [656, 400])
def test_turn_then_decode(fmt):
    s = Serving(fmt)
    s.prompt()
    s.offload()
    s.buffers()
    print(f"[step] fmt={fmt}", flush=True)
    s.step()
    s.check_step()


@pytest.mark.parametrize("fmt", [656, 400])
def test_decode_step_replays(fmt):
    """Captured once, replayed four times with eager work between; every replay
    gives the eager call's results byte for byte, from the same state."""
    from serving_memory_tier_amd.hipgraph import HipRuntime
    s = Serving(fmt)
    s.prompt()
    s.offload()
    s.buffers()
    keep = {k: getattr(s, k).clone() for k in ("pool", "tok", "stp")}

    def restore():
        for k, v in keep.items():
            getattr(s, k).copy_(v)
        for k in ("ids", "out", "lse", "dense", "dlse", "q", "new", "stats", "ws", "dws"):
            s.g[k].fill_(7)
        s.g["q"].copy_(s.g["q0"])
        torch.cuda.synchronize()

    restore()
    s.step()
    want = s.results()
    pool = s.pool.clone()
    rt = HipRuntime()
    stream = torch.cuda.Stream()
    restore()
    with torch.cuda.stream(stream):
        rt.begin_capture(stream.cuda_stream)
        s.step(stream.cuda_stream)
        rt.end_capture(stream.cuda_stream)
    try:
        for i in range(4):
            restore()
            torch.randn(300, 300, device="cuda").mm(torch.randn(300, 300, device="cuda")).sum()
            torch.cuda.synchronize()
            print(f"[replay] fmt={fmt} {i}", flush=True)
            rt.launch(stream.cuda_stream)
            got = s.results()
            for k, v in want.items():
                assert torch.equal(got[k].view(torch.uint8), v.view(torch.uint8)), (i, k)
            assert torch.equal(s.pool, pool), i
    finally:
        torch.cuda.synchronize()
        rt.close()


@pytest.mark.parametrize("fmt", [656, 400])
def test_prefill_captured(fmt):
    """The expanded form in a graph, new contents at the same addresses between replays."""
    import serving_memory_tier_amd as hs
    from serving_memory_tier_amd.hipgraph import HipRuntime
    rs = np.random.default_rng(5)
    ctx = [[300, 700], [700, 64], [1, 699]]
    start = [[0, 100, 150], [0, 20, 84], [0, 1, 150]]
    pools = [ol.encode_rows(bits(rs, 1600, 512), bits(rs, 1600, 64), fmt) for _ in ctx]
    lay = hs.layout_of(64, fmt, 1, 64, 1600, 0)
    bt = rs.permutation(25)[:22].reshape(2, 11).astype(np.int32)
    q, w = bits(rs, 150, 4, 192), bits(rs, 4, 256, 512, mult=0.05)
    g = [dev(pools[0]), dev(bt), dev(np.array(ctx[0], np.int32)), dev(np.array(start[0], np.int32)),
         dev(q), dev(w)]
    out = torch.empty((150, 4, 128), dtype=torch.int16, device="cuda")
    ws = torch.empty(hs.hs_mla_prefill_workspace_bytes(2, 150, 1000, 4), dtype=torch.uint8,
                     device="cuda")
    batch = hs.batch_of(2, 11, g[0], None, g[1], None, g[2], None, None, None)
    call = lambda st=None: hs.hs_mla_prefill(lay, batch, 0, g[3], 150, 1000, g[4], 4, g[5], SCALE,
                                             out, ws, st)
    rt, stream = HipRuntime(), torch.cuda.Stream()
    rt.begin_capture(stream.cuda_stream)
    call(stream.cuda_stream)
    rt.end_capture(stream.cuda_stream)
    try:
        for i in (0, 1, 2, 0):
            g[0].copy_(dev(pools[i]))
            g[2].copy_(dev(np.array(ctx[i], np.int32)))
            g[3].copy_(dev(np.array(start[i], np.int32)))
            both = []
            for run in (call, lambda: rt.launch(stream.cuda_stream)):
                out.fill_(0x1234)
                ws.fill_(255)
                torch.cuda.synchronize()
                print(f"[prefill] fmt={fmt} inputs {i}", flush=True)
                run()
                torch.cuda.synchronize()
                both.append(out.clone())
            assert torch.equal(both[0], both[1]), i
            check_prefill(f64(out), pools[i], bt, np.array(ctx[i]), np.array(start[i]), q, w, 64,
                          SCALE)
    finally:
        rt.close()


def test_two_streams():
    """Calls of every kind on two streams at once, a workspace each: what they
    give alone."""
    import serving_memory_tier_amd as hs
    rs = np.random.default_rng(9)
    Rn, ctx, Hn, Kn = 2, 5000, 64, 1500
    jobs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for fmt in (656, 400):
        rows = 64 * 180
        pool = dev(ol.encode_rows(bits(rs, rows, 512), bits(rs, rows, 64), fmt))
        bt = dev(rs.permutation(180)[:160].reshape(Rn, 80).astype(np.int32))
        cl = dev(np.array([ctx, ctx - 77], np.int32))
        lay = hs.layout_of(64, fmt, 1, 64, rows, 0)
        batch = hs.batch_of(Rn, 80, pool, None, bt, None, cl, None, None, None)
        q = dev(bits(rs, Rn, Hn, 576))
        ids = dev(rs.integers(-1, rows, (Rn, Kn)).astype(np.int32))
        qp, w = dev(bits(rs, 200, 8, 192)), dev(bits(rs, 8, 256, 512, mult=0.05))
        start = dev(np.array([0, 150, 200], np.int32))
        o = [torch.empty((Rn, Hn, 512), dtype=torch.int16, device="cuda") for _ in range(2)]
        l = [torch.empty((Rn, Hn), device="cuda") for _ in range(2)]
        op = torch.empty((200, 8, 128), dtype=torch.int16, device="cuda")
        ws = [torch.empty(max(n, 16), dtype=torch.uint8, device="cuda") for n in (
            hs.hs_paged_mla_workspace_bytes(Rn, 1, Hn, ctx),
            hs.hs_sparse_mla_fp4_workspace_bytes(Rn, Hn, Kn),
            hs.hs_mla_prefill_workspace_bytes(Rn, 200, 2 * ctx, 8))]

        def job(st, fmt=fmt, lay=lay, batch=batch, pool=pool, q=q, ids=ids, qp=qp, w=w,
                start=start, o=o, l=l, op=op, ws=ws):
            hs.hs_paged_mla_decode(lay, batch, 0, q, 1, Hn, ctx, SCALE, o[0], l[0], ws[0], st)
            if fmt == 400:
                hs.hs_sparse_mla_decode_fp4(lay, pool, ids, Rn, Kn, q, Hn, SCALE, o[1], l[1],
                                            ws[1], st)
            hs.hs_mla_prefill(lay, batch, 0, start, 200, 2 * ctx, qp, 8, w, SCALE, op, ws[2], st)

        jobs.append((job, [o[0], l[0], op] + ([o[1], l[1]] if fmt == 400 else []), bt, cl))
    want = []
    for job, outs, *_ in jobs:
        job(None)
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
        for t in outs:
            t.fill_(3)
    torch.cuda.synchronize()
    for i in range(6):
        print(f"[streams] pass {i}", flush=True)
        for (job, *_), st in zip(jobs, streams):
            job(st.cuda_stream)
    torch.cuda.synchronize()
    for (_, outs, *_), w in zip(jobs, want):
        for t, x in zip(outs, w):
            assert torch.equal(t, x)
