"""The operators around the latent (MLA) cache, as cases to measure: appending rows to the paged
pool with the position rotation on the way, sparse decode over 4-bit rows, dense decode through
the block table (absorbed form), and the prefill of a chunk of new tokens (expanded form).

With ``own`` false ``run`` computes each operator in its plain form with elementary torch
operations; with ``own`` true it calls the framework.  ``exact`` states the same in 64 bits.

Two row formats: "fp8", 656 bytes (512 E4M3 values, 4 float32 scales, 64 bfloat16 rope values),
and "fp4", 400 bytes (512 E2M1 values, 16 E8M0 scales, 64 bfloat16 rope values).
"""

import math
import random

import torch

own = False

LATENT, ROPE, DIM = 512, 64, 576
NOPE, VDIM = 128, 128               # expanded heads: 128 + 64 query/key values, 128 value dimensions
PAGE = 64
ROW = {"fp8": 656, "fp4": 400}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one new token for each of the 32 requests of a decode step, all heads on one GPU
        {"name": "append_decode_fp8", "op": "append", "fmt": "fp8", "tokens": 32, "heads": 128,
         "requests": 32, "longest": 74160, "interleaved": True},
        # a verify step: 128 requests x 4 positions of contexts up to a million tokens, a
        # tensor-parallel rank's 16 heads, 4-bit rows
        {"name": "append_verify_fp4", "op": "append", "fmt": "fp4", "tokens": 512, "heads": 16,
         "requests": 128, "longest": 1000000, "interleaved": False},
        # sixteen requests' next turns of 753 tokens in one prefill batch
        {"name": "append_turns_fp8", "op": "append", "fmt": "fp8", "tokens": 16 * 753, "heads": 128,
         "requests": 16, "longest": 142000, "interleaved": True},
        # a few requests on a tensor-parallel rank, ragged lists
        {"name": "sparse_fp4_ragged", "op": "sparse", "tokens": 5, "heads": 16, "top_k": 1000,
         "rows": 20000, "holes": 0.2},
        # the decode step: 32 requests x 128 heads x top-2048
        {"name": "sparse_fp4_decode", "op": "sparse", "tokens": 32, "heads": 128, "top_k": 2048,
         "rows": 200000, "holes": 0.0},
        # a speculative step: 128 requests x 4 positions x top-2048
        {"name": "sparse_fp4_plan", "op": "sparse", "tokens": 512, "heads": 128, "top_k": 2048,
         "rows": 400000, "holes": 0.02},
        # short contexts on a tensor-parallel rank: latency
        {"name": "paged_short_fp8", "op": "paged", "fmt": "fp8", "requests": 3, "positions": 1,
         "heads": 16, "context": 500, "holes": 0.0},
        # dense decode of a batch with middling contexts
        {"name": "paged_decode_fp8", "op": "paged", "fmt": "fp8", "requests": 32, "positions": 1,
         "heads": 128, "context": 8192, "holes": 0.0},
        # a verify step of long contexts from 4-bit rows, a few pages only on the host
        {"name": "paged_verify_fp4", "op": "paged", "fmt": "fp4", "requests": 8, "positions": 4,
         "heads": 128, "context": 74160, "holes": 0.02},
        # short prompts on a tensor-parallel rank
        {"name": "prefill_short_fp8", "op": "prefill", "fmt": "fp8", "requests": 3, "new": 130,
         "context": 500, "heads": 16},
        # four requests' next turns of 753 tokens behind 4,096 cached ones
        {"name": "prefill_turns_fp4", "op": "prefill", "fmt": "fp4", "requests": 4, "new": 753,
         "context": 4849, "heads": 64},
        # a chunk of a long prompt, all heads
        {"name": "prefill_chunk_fp8", "op": "prefill", "fmt": "fp8", "requests": 1, "new": 2048,
         "context": 8192, "heads": 128},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    return rng.choice((128, 64, 32, 16, 8, rng.randint(1, 128)))


def draw(rng):
    op = rng.choice(("append", "sparse", "paged", "prefill"))
    fmt = rng.choice(("fp8", "fp4"))
    if op == "append":
        tokens = _log(rng, 1, 12048)
        return {"op": op, "fmt": fmt, "tokens": tokens, "heads": _heads(rng),
                "requests": rng.randint(1, min(tokens, 128)), "longest": _log(rng, 64, 1000000),
                "interleaved": rng.random() < 0.5}
    if op == "sparse":
        heads, tokens = _heads(rng), _log(rng, 1, 512)
        top_k = _log(rng, 1, 4096)
        while tokens * heads * top_k > 512 * 128 * 2048 or tokens * top_k > 512 * 2048:
            tokens = max(1, tokens // 2)
        return {"op": op, "tokens": tokens, "heads": heads, "top_k": top_k,
                "rows": PAGE * _log(rng, 8, 6000), "holes": rng.choice((0.0, 0.05, 0.6))}
    if op == "paged":
        heads, positions, context = _heads(rng), rng.randint(1, 4), _log(rng, 1, 74160)
        requests = _log(rng, 1, 64)
        while (requests * positions * heads * context > 8 * 4 * 128 * 74160
               or requests * context > 8 * 74160):
            requests = max(1, requests // 2)
        return {"op": op, "fmt": fmt, "requests": requests, "positions": positions,
                "heads": heads, "context": context, "holes": rng.choice((0.0, 0.0, 0.1))}
    heads, requests, new = _heads(rng), rng.randint(1, 6), _log(rng, 2, 2048)
    context = new + rng.choice((0, _log(rng, 1, 6144)))
    while (requests * heads * new * context > 128 * 2048 * 8192
           or requests * context * heads > 8192 * 128):
        if requests > 1:
            requests -= 1
        else:
            heads = max(1, heads // 2)
    return {"op": op, "fmt": fmt, "requests": requests, "new": new, "context": context,
            "heads": heads}


def _spread(most, n):
    """n lengths from `most` down to about half of it."""
    return [max(1, most - (most * r) // (2 * n)) for r in range(n)]


def _contexts(case):
    return _spread(case["context"], case["requests"])


def _news(case):
    """New tokens of each request of a prefill, at most its context."""
    return [min(n, c) for n, c in zip(_spread(case["new"], case["requests"]), _contexts(case))]


def work(case):
    H = case["heads"]
    if case["op"] == "append":
        T = case["tokens"]
        return {"bytes": T * (2 * DIM + ROW[case["fmt"]] + 2 * DIM + 12 + H * ROPE * 4) + 256,
                "flops": T * (H + 1) * ROPE * 3}
    if case["op"] == "sparse":
        T, K = case["tokens"], case["top_k"]
        rows = T * K * (1 - case["holes"])
        seen = min(rows, case["rows"])
        return {"bytes": seen * ROW["fp4"] + T * K * 4 + T * H * (2 * DIM + 2 * LATENT + 4),
                "flops": 2 * H * rows * (DIM + LATENT)}
    if case["op"] == "paged":
        P, ctx = case["positions"], _contexts(case)
        pairs = sum(max(0, c - P + p + 1) for c in ctx for p in range(P)) * (1 - case["holes"])
        return {"bytes": sum(ctx) * (1 - case["holes"]) * ROW[case["fmt"]]
                + len(ctx) * P * H * (2 * DIM + 2 * LATENT + 4) + 4 * (sum(ctx) // PAGE),
                "flops": 2 * H * pairs * (DIM + LATENT)}
    ctx, new = _contexts(case), _news(case)
    pairs = sum(n * c - n * (n - 1) // 2 for n, c in zip(new, ctx))
    return {"bytes": sum(ctx) * ROW[case["fmt"]] + H * (NOPE + VDIM) * LATENT * 2
            + sum(new) * H * (2 * (NOPE + ROPE) + 2 * VDIM),
            "flops": 2 * sum(ctx) * LATENT * H * (NOPE + VDIM)
            + 2 * H * pairs * (NOPE + ROPE + VDIM)}


# ----------------------------------------------------------------- inputs

def _freq(device):
    j = torch.arange(ROPE // 2, dtype=torch.float64, device=device)
    return 10000.0 ** (-2.0 * j / ROPE)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _pool(g, rows, fmt):
    """A pool of `rows` rows, encoded from unit normal latents (as a normalised latent has)."""
    out = torch.empty((rows, ROW[fmt]), dtype=torch.uint8, device="cuda")
    for lo in range(0, rows, 1 << 17):
        n = min(1 << 17, rows - lo)
        out[lo:lo + n] = _encode(_normal(g, n, LATENT), _normal(g, n, ROPE), fmt)
    return out


def _tables(g, pages, blocks, holes=0.0):
    """A block table [R][max pages] of distinct random blocks, some of them null placeholders."""
    R, most = len(pages), max(pages)
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    bt = torch.full((R, most), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, n in enumerate(pages):
        bt[r, :n] = order[at:at + n]
        at += n
    if holes:
        bt[torch.rand((R, most), generator=g, device="cuda") < holes] = -1
    return bt


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    H, i32, dev = case["heads"], torch.int32, "cuda"
    s = dict(case)
    s["scale"] = (NOPE + ROPE) ** -0.5
    if case["op"] == "append":
        # runs of consecutive positions, one run a request, ending at a random position below
        # `longest`; the last token of the batch is padding (request -1), as in a step padded to
        # a captured size
        T, R = case["tokens"], case["requests"]
        per = -(-T // R)
        rnd = random.Random(seed)
        last = [rnd.randrange(case["longest"]) + per for _ in range(R)]
        pages = [n // PAGE + 1 for n in last]
        first = [max(0, (n - per) // PAGE) for n in last]
        used = [p - f for p, f in zip(pages, first)]
        blocks = R * (per // PAGE + 2)        # a run touches this many pages at most
        order = torch.randperm(blocks, generator=g, device=dev).to(i32)
        bt = torch.full((R, max(pages)), -1, dtype=i32, device=dev)
        at = 0
        for r in range(R):
            bt[r, first[r]:pages[r]] = order[at:at + used[r]]
            at += used[r]
        req = torch.arange(T, dtype=i32, device=dev) // per
        ends = torch.tensor(last, dtype=i32, device=dev)
        pos = ends[req.long()] - per + torch.arange(T, dtype=i32, device=dev) % per
        if T > 1:
            req[-1] = -1
        kv = _normal(g, T, DIM)               # the down-projection's output: latent and rope parts
        q = _normal(g, T, H, NOPE + ROPE)     # the queries: their rope part is rotated
        rows = blocks * PAGE
        pool = torch.zeros((rows + 1, ROW[case["fmt"]]), dtype=torch.uint8, device=dev)
        s.update(rows=rows, pool=pool, bt=bt, req=req, pos=pos, latent=_normal(g, T, LATENT),
                 rope=kv[:, LATENT:], q_rope=q[:, :, NOPE:], freq=_freq(dev),
                 q_out=torch.zeros((T, H, DIM), dtype=torch.bfloat16, device=dev),
                 values=torch.zeros((T, DIM), dtype=torch.bfloat16, device=dev),
                 row_ids=torch.zeros(T, dtype=i32, device=dev))
        if own:
            import serving_memory_tier_amd as hs
            s["layout"] = hs.layout_of(PAGE, ROW[case["fmt"]], 1, PAGE, rows, 0)
            s["batch"] = hs.batch_of(R, bt.shape[1], pool, None, bt, None, None, None, None, None)
            s["call"] = hs.append_of(T, req, pos, s["latent"], s["rope"], s["freq"],
                                     case["interleaved"], s["q_rope"], s["q_out"][:, :, LATENT:])
        return s
    if case["op"] == "sparse":
        T, K = case["tokens"], case["top_k"]
        rows = -(-case["rows"] // PAGE) * PAGE
        ids = torch.randint(0, rows, (T, K), generator=g, device=dev, dtype=i32)
        if case["holes"]:
            ids[torch.rand((T, K), generator=g, device=dev) < case["holes"]] = -1
        s.update(pool=_pool(g, rows, "fp4"), ids=ids, q=_normal(g, T, H, DIM), rows=rows,
                 out=torch.empty((T, H, LATENT), dtype=torch.bfloat16, device=dev),
                 lse=torch.empty((T, H), device=dev))
        if own:
            import serving_memory_tier_amd as hs
            s["layout"] = hs.layout_of(PAGE, ROW["fp4"], 1, PAGE, rows, 0)
            need = hs.hs_sparse_mla_fp4_workspace_bytes(T, H, K)
            s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        return s
    ctx = _contexts(case)
    pages = [-(-c // PAGE) for c in ctx]
    blocks = sum(pages) + 3
    R = len(ctx)
    bt = _tables(g, pages, blocks, case.get("holes", 0.0))
    s.update(pool=_pool(g, blocks * PAGE, case["fmt"]), bt=bt, rows=blocks * PAGE,
             ctx=torch.tensor(ctx, dtype=i32, device=dev), longest=max(ctx))
    if case["op"] == "paged":
        P = case["positions"]
        s.update(q=_normal(g, R, P, H, DIM),
                 out=torch.empty((R, P, H, LATENT), dtype=torch.bfloat16, device=dev),
                 lse=torch.empty((R, P, H), device=dev))
    else:
        new = _news(case)
        start = [0]
        for n in new:
            start.append(start[-1] + n)
        # the up-projection's weights [H][128 key + 128 value dimensions][512]: unit variance
        # latents give unit variance keys and values
        s.update(q=_normal(g, start[-1], H, NOPE + ROPE), new=new, total=sum(ctx),
                 w=(torch.randn((H, NOPE + VDIM, LATENT), generator=g, device=dev)
                    * LATENT ** -0.5).to(torch.bfloat16),
                 q_start=torch.tensor(start, dtype=i32, device=dev),
                 out=torch.empty((start[-1], H, VDIM), dtype=torch.bfloat16, device=dev))
    if own:
        import serving_memory_tier_amd as hs
        s["layout"] = hs.layout_of(PAGE, ROW[case["fmt"]], 1, PAGE, s["rows"], 0)
        s["batch"] = hs.batch_of(R, bt.shape[1], s["pool"], None, bt, None, s["ctx"], None, None,
                                 None)
        need = (hs.hs_paged_mla_workspace_bytes(R, P, H, s["longest"]) if case["op"] == "paged"
                else hs.hs_mla_prefill_workspace_bytes(R, s["q"].shape[0], s["total"], H))
        s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------ plain forms

def _encode(latent, rope, fmt):
    """bfloat16 latents [n, 512] and rope values [n, 64] as the rows' bytes.  A group's scale is
    the smallest power of two (from 2^-126) under which its largest value stays within 448 (E4M3)
    or rounds to at most 6 (E2M1); 1 for a group of zeros."""
    group, top = (128, 448.0) if fmt == "fp8" else (32, 7.0)
    x = latent.float().unflatten(-1, (-1, group))
    most = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(most / top)
    e = torch.where(m == 0.5, e - 1, e).clamp(min=-126)
    e = torch.where(most == 0, torch.zeros_like(e), e)
    y = torch.ldexp(x, -e)
    if fmt == "fp8":
        codes = y.to(torch.float8_e4m3fn).flatten(-2).view(torch.uint8)
        scales = torch.ldexp(torch.ones_like(most), e).flatten(-2).view(torch.uint8)
    else:
        a = y.abs()
        c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
             + (a >= 3.5) + (a > 5)) | (torch.signbit(y).to(torch.uint8) << 3)
        c = c.flatten(-2)
        codes = c[..., 0::2] | (c[..., 1::2] << 4)
        scales = (e + 127).to(torch.uint8).flatten(-2)
    return torch.cat([codes, scales, rope.contiguous().view(torch.uint8)], -1)


def _decode(rows, fmt):
    """Rows' bytes [..., n] to their float32 latents [..., 512] and rope values [..., 64]."""
    if fmt == "fp8":
        lat = rows[..., :512].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (4, 128))
        scale = rows[..., 512:528].contiguous().view(torch.float32)
        rope = rows[..., 528:]
    else:
        b = rows[..., :256]
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=rows.device)
        lat = table[torch.stack([b & 15, b >> 4], -1).flatten(-2).int()].unflatten(-1, (16, 32))
        scale = torch.exp2(rows[..., 256:272].float() - 127.0)
        rope = rows[..., 272:]
    return ((lat * scale[..., None]).flatten(-2),
            rope.contiguous().view(torch.bfloat16).float())


def _rotate(x, cos, sin, interleaved):
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)


def _append(s):
    angle = s["pos"].double()[:, None] * s["freq"]
    cos, sin = torch.cos(angle), torch.sin(angle)
    # the cached keys' rotation in 64 bits, rounded once: bytes that do not depend on who rotates
    rope = _rotate(s["rope"].double(), cos, sin, s["interleaved"]).to(torch.bfloat16)
    rows = _encode(s["latent"], rope, s["fmt"])
    req, pos = s["req"].long(), s["pos"].long()
    block = s["bt"][req.clamp(min=0), pos // PAGE].long()
    ok = (req >= 0) & (block >= 0)
    at = block * PAGE + pos % PAGE
    s["pool"][torch.where(ok, at, s["rows"])] = rows     # the row behind the pool takes the padding
    lat, _ = _decode(rows, s["fmt"])
    values = torch.cat([lat.to(torch.bfloat16), rope], -1)
    s["values"].copy_(torch.where(ok[:, None], values, s["values"]))
    q = _rotate(s["q_rope"].float(), cos.float()[:, None], sin.float()[:, None], s["interleaved"])
    part = s["q_out"][:, :, LATENT:]
    part.copy_(torch.where(ok[:, None, None], q.to(torch.bfloat16), part))
    s["row_ids"].copy_(torch.where(ok, at, torch.where(req < 0, -1, -3)))
    return _append_outputs(s)


def _append_outputs(s):
    return {"row_ids": s["row_ids"], "values": s["values"], "q": s["q_out"][:, :, LATENT:],
            "pool": s["pool"][:s["rows"]]}


def _softmax_av(scores, v):
    """softmax(scores) v and its log sum, rows without any key giving 0 and -inf."""
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(m == -math.inf, torch.zeros_like(m), m))
    z = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(z > 0, z, torch.ones_like(z))
    return out.to(torch.bfloat16), (m + torch.log(z))[..., 0]


def _sparse(s):
    ids = s["ids"]
    lat, rope = _decode(s["pool"][ids.clamp(min=0).long()], "fp4")
    k = torch.cat([lat, rope], -1)
    scores = torch.matmul(s["q"].float(), k.transpose(1, 2)) * s["scale"]
    scores.masked_fill_((ids < 0)[:, None], -math.inf)
    out, lse = _softmax_av(scores, lat)
    return {"out": out, "lse": lse}


def _context_rows(s):
    """Every request's rows, padded to the longest, and which of them are there."""
    t = torch.arange(s["longest"], device="cuda")
    block = s["bt"][:, t // PAGE].long()
    ok = (block >= 0) & (t < s["ctx"][:, None])
    return torch.where(ok, block * PAGE + t % PAGE, torch.zeros_like(block)), ok, t


def _paged(s):
    at, ok, t = _context_rows(s)
    lat, rope = _decode(s["pool"][at], s["fmt"])
    k = torch.cat([lat, rope], -1)
    R, P, H = s["q"].shape[:3]
    last = s["ctx"][:, None] - P + torch.arange(P, device="cuda", dtype=torch.int32)
    seen = ok[:, None] & (t <= last[:, :, None])                       # [R][P][tokens]
    scores = torch.matmul(s["q"].float().flatten(1, 2), k.transpose(1, 2)) * s["scale"]
    scores = scores.unflatten(1, (P, H)).masked_fill(~seen[:, :, None], -math.inf)
    out, lse = _softmax_av(scores.flatten(1, 2), lat)
    return {"out": out.unflatten(1, (P, H)), "lse": lse.unflatten(1, (P, H))}


def _prefill(s):
    at, ok, t = _context_rows(s)
    lat, rope = _decode(s["pool"][at], s["fmt"])                       # [R][tokens][...]
    H = s["heads"]
    kv = torch.matmul(lat, s["w"].float().flatten(0, 1).t()).unflatten(-1, (H, NOPE + VDIM))
    k = torch.cat([kv[..., :NOPE], rope[:, :, None].expand(-1, -1, H, -1)], -1)
    v = kv[..., NOPE:].transpose(1, 2)                                 # [R][H][tokens][128]
    most = max(s["new"])
    i = torch.arange(most, device="cuda")
    new = s["q_start"][1:] - s["q_start"][:-1]
    live = i < new[:, None]                                            # [R][queries]
    src = torch.where(live, s["q_start"][:-1, None] + i, torch.zeros_like(i)).long()
    q = s["q"][src].float().transpose(1, 2)                            # [R][H][queries][192]
    last = s["ctx"][:, None] - new[:, None] + i
    seen = ok[:, None] & (t <= last[:, :, None])                       # [R][queries][tokens]
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]
    scores.masked_fill_(~seen[:, None], -math.inf)
    out, _ = _softmax_av(scores, v)
    # back to the packed order of the queries
    flat = torch.arange(s["q"].shape[0], device="cuda", dtype=torch.int32)
    r = (torch.searchsorted(s["q_start"], flat, right=True) - 1)
    n = (flat - s["q_start"][r]).long()
    return {"out": out[r, :, n]}


def run(s):
    op = s["op"]
    if not own:
        return {"append": _append, "sparse": _sparse, "paged": _paged, "prefill": _prefill}[op](s)
    import serving_memory_tier_amd as hs
    if op == "append":
        hs.hs_mla_append(s["layout"], s["batch"], 0, s["call"], s["row_ids"], s["values"])
        return _append_outputs(s)
    if op == "sparse":
        hs.hs_sparse_mla_decode_fp4(s["layout"], s["pool"], s["ids"], s["tokens"], s["top_k"],
                                    s["q"], s["heads"], s["scale"], s["out"], s["lse"], s["ws"])
    elif op == "paged":
        hs.hs_paged_mla_decode(s["layout"], s["batch"], 0, s["q"], s["positions"], s["heads"],
                               s["longest"], s["scale"], s["out"], s["lse"], s["ws"])
    else:
        hs.hs_mla_prefill(s["layout"], s["batch"], 0, s["q_start"], s["q"].shape[0], s["total"],
                          s["q"], s["heads"], s["w"], s["scale"], s["out"], s["ws"])
        return {"out": s["out"]}
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------ in 64 bits, apart

def exact(case, seed):
    s = prepare(case, seed)
    f64, dev = torch.float64, "cuda"

    def grid(x, bias, mantissa, top):
        """x rounded to the nearest value of a small float format, ties to even."""
        e = torch.frexp(x)[1] - 1
        step = torch.ldexp(torch.ones_like(x), e.clamp(min=1 - bias) - mantissa)
        return (torch.round(x / step) * step).clamp(-top, top)

    def decode(rows, fmt):
        n = rows.shape[0]
        if fmt == "fp8":
            b = rows[:, :512].to(torch.int64)
            e, m = (b >> 3) & 15, (b & 7).to(f64)
            mag = torch.where(e == 0, m * 2.0 ** -9,
                              torch.ldexp(1 + m / 8, e.to(torch.int32) - 7))
            lat = torch.where(b >= 128, -mag, mag)
            scale = rows[:, 512:528].contiguous().view(torch.float32).to(f64)
            return ((lat.view(n, 4, 128) * scale[:, :, None]).view(n, 512),
                    rows[:, 528:].contiguous().view(torch.bfloat16).to(f64))
        b = rows[:, :256].to(torch.int64)
        c = torch.stack([b % 16, b // 16], 2).view(n, 512)
        e, m = (c >> 1) & 3, (c & 1).to(f64)
        mag = torch.where(e == 0, m / 2, torch.ldexp(1 + m / 2, e.to(torch.int32) - 1))
        lat = torch.where(c >= 8, -mag, mag)
        scale = torch.ldexp(torch.ones((n, 16), dtype=f64, device=dev),
                            rows[:, 256:272].to(torch.int32) - 127)
        return ((lat.view(n, 16, 32) * scale[:, :, None]).view(n, 512),
                rows[:, 272:].contiguous().view(torch.bfloat16).to(f64))

    def attend(q, k, v, seen):
        """q [m, d], k [n, d], v [n, e], seen [m, n] or [n]."""
        sc = (q @ k.t()) * s["scale"]
        sc = torch.where(seen, sc, torch.full_like(sc, -math.inf))
        lse = torch.logsumexp(sc, -1)
        p = torch.where(seen, torch.exp(sc - torch.where(lse == -math.inf, 0.0, lse)[:, None]), 0.0)
        return p @ v, lse

    if case["op"] == "append":
        T, H = case["tokens"], case["heads"]
        size, top, bias, mantissa = (128, 448.0, 7, 3) if case["fmt"] == "fp8" else (32, 6.0, 1, 1)
        x = s["latent"].to(f64).view(T, -1, size)
        limit = 448.0 if case["fmt"] == "fp8" else 7.0
        most = x.abs().amax(-1)
        e = torch.ceil(torch.log2(most / limit))
        e = torch.where(most > limit * 2 ** e, e + 1, e)
        e = torch.where(most <= limit * 2 ** (e - 1), e - 1, e).clamp(min=-126)
        unit = torch.where(most == 0, torch.ones_like(e), 2 ** e)[:, :, None]
        lat = (grid(x / unit, bias, mantissa, top) * unit).view(T, 512)
        t = s["pos"].to(f64)[:, None] * s["freq"]

        def turn(x):
            z = (torch.view_as_complex(x.unflatten(-1, (32, 2)).contiguous())
                 if case["interleaved"] else torch.complex(x[..., :32], x[..., 32:]))
            z = z * torch.polar(torch.ones_like(t), t).view(T, *(1,) * (x.dim() - 2), 32)
            return (torch.view_as_real(z).flatten(-2) if case["interleaved"]
                    else torch.cat([z.real, z.imag], -1))

        values = torch.cat([lat, turn(s["rope"].to(f64))], 1)
        q = turn(s["q_rope"].to(f64))
        there = s["req"] >= 0
        values[~there] = 0
        q[~there] = 0
        return {"row_ids": None, "values": values, "q": q, "pool": None}
    if case["op"] == "sparse":
        out, lse = [], []
        for t in range(case["tokens"]):
            ids = s["ids"][t]
            lat, rope = decode(s["pool"][ids.clamp(min=0).long()], "fp4")
            o, l = attend(s["q"][t].to(f64), torch.cat([lat, rope], 1), lat, (ids >= 0)[None])
            out.append(o)
            lse.append(l)
        return {"out": torch.stack(out), "lse": torch.stack(lse)}
    out, lse = [], []
    for r, c in enumerate(_contexts(case)):
        tok = torch.arange(c, device=dev)
        block = s["bt"][r][tok // PAGE].long()
        lat, rope = decode(s["pool"][block.clamp(min=0) * PAGE + tok % PAGE], case["fmt"])
        H = case["heads"]
        if case["op"] == "paged":
            P = case["positions"]
            for p in range(P):
                o, l = attend(s["q"][r, p].to(f64), torch.cat([lat, rope], 1), lat,
                              ((block >= 0) & (tok <= c - P + p))[None])
                out.append(o)
                lse.append(l)
            continue
        n, at = s["new"][r], int(s["q_start"][r])
        seen = tok[None] <= (c - n + torch.arange(n, device=dev))[:, None]
        for h in range(H):
            w = s["w"][h].to(f64)
            out.append(attend(s["q"][at:at + n, h].to(f64),
                              torch.cat([lat @ w[:NOPE].t(), rope], 1), lat @ w[NOPE:].t(),
                              seen)[0])
    if case["op"] == "paged":
        shape = s["q"].shape[:3]
        return {"out": torch.stack(out).view(*shape, LATENT), "lse": torch.stack(lse).view(shape)}
    H, R = case["heads"], case["requests"]
    return {"out": torch.cat([torch.stack(out[r * H:(r + 1) * H], 1) for r in range(R)])}
