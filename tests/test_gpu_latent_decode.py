"""GPU parity of hs_sparse_mla_decode_fp4 and hs_paged_mla_decode with the float64
oracle, within bounds the arithmetic fixes.  With A = sum_j p_j |v_j| (each
value dimension) and S the largest scale * <|q|, |k_j|>:
  - scores accumulate 576 float32 products: off by at most 600 * 2^-24 * S = e;
  - the probabilities times scales are rounded to bfloat16: 2^-8 A;
  - a split's normalised output is rounded to half precision, scaled so that its
    largest value is in [1, 2): 2^-11 A, or half a step of its least, 2^-25 of
    that scale, which is at most the row's largest A;
  - the output is rounded to bfloat16: 2^-8 |out|;
so |d out| <= (2^-8 + 2^-11 + 2 e) A + 2^-25 max A + 2^-8 |out| + 2^-30
(probabilities below float32's range), and |d lse| <= e + 2^-20 |lse| + 2^-20
(the sum, its logarithm and the two products with log2 e)."""

from __future__ import annotations

import math
import os
import zlib

import numpy as np
import pytest
import torch

from oracle import latent as ol
from oracle import sparse_mla as sm

pytestmark = pytest.mark.gpu
FORMATS = [656, 400]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import serving_memory_tier_amd as hs
    if not os.path.exists(hs.LIB_PATH):
        from serving_memory_tier_amd import build
        build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    hs.lib()


def dev(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


def bits(rs, *shape, mult=1.0):
    return ol.to_bf16(rs.standard_normal(shape) * mult)


def make_pool(rs, rows, fmt, spread=2):
    """Rows of random codes and scales (FP8 scales are any float, not powers of two)."""
    pool = rs.integers(0, 256, (rows, fmt)).astype(np.uint8)
    if fmt == 400:
        pool[:, 256:272] = 127 + rs.integers(-spread - 1, spread, (rows, 16))
        at = 272
    else:
        pool[:, :512] &= 0xBF                      # |value| < 2, no NaN
        pool[:, 512:528] = rs.uniform(0.2, 1.0, (rows, 4)).astype("<f4").view(np.uint8)
        at = 528
    pool[:, at:] = bits(rs, rows, 64).view(np.uint8)
    return pool


def bound(q, ids, pool, seen, scale, out, lse):
    """The docstring's bounds for one query row group: q [m, 576] float64."""
    k, v = ol.decode_rows(pool[np.maximum(ids, 0)])
    k, v = np.where((ids >= 0)[:, None], k, 0), np.where((ids >= 0)[:, None], v, 0)
    a, _ = ol.attend(q, k, np.abs(v), seen, scale)
    s = (np.where(seen, abs(scale) * (np.abs(q) @ np.abs(k).T), 0)).max(1, initial=0)
    e = 600 * 2.0 ** -24 * s[:, None]
    return ((2.0 ** -8 + 2.0 ** -11 + 2 * e) * a + 2.0 ** -25 * a.max(1, keepdims=True)
            + 2.0 ** -8 * np.abs(out) + 2.0 ** -30,
            e[:, 0] + 2.0 ** -20 * np.abs(np.where(np.isfinite(lse), lse, 0)) + 2.0 ** -20)


def compare(got, gotl, ref, refl, tol, toll, what):
    empty = np.isneginf(refl)
    assert (np.isneginf(gotl) == empty).all(), what
    assert (got[empty] == 0).all(), what
    assert (np.abs(got - ref) <= tol).all(), (what, np.abs(got - ref).max(), tol.min())
    assert (np.abs(gotl[~empty] - refl[~empty]) <= toll[~empty]).all(), (
        what, np.abs(gotl[~empty] - refl[~empty]).max())


def f64(t):
    return sm.bf16_to_float(t.cpu().numpy().view(np.uint16))


def run_sparse(pool, ids, q, scale, stream=None):
    import serving_memory_tier_amd as hs
    T, K = ids.shape
    H = q.shape[1]
    lay = hs.layout_of(1, 400, 1, 64, pool.shape[0], 0)
    out = torch.full((T, H, 512), -1, dtype=torch.int16, device="cuda")
    lse = torch.full((T, H), float("nan"), device="cuda")
    need = hs.hs_sparse_mla_fp4_workspace_bytes(T, H, K)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if need else None
    args = dev(pool), dev(ids), dev(q)
    print(f"[sparse] T={T} H={H} K={K} rows={pool.shape[0]} ws={need}", flush=True)
    hs.hs_sparse_mla_decode_fp4(lay, args[0], args[1], T, K, args[2], H, scale, out, lse, ws,
                                stream)
    torch.cuda.synchronize()
    return f64(out), lse.cpu().numpy().astype(np.float64)


def check_sparse(pool, ids, q, scale):
    out, lse = run_sparse(pool, ids, q, scale)
    ref, refl = ol.sparse_mla_decode(pool, ids, q, scale)
    for t in range(ids.shape[0]):
        there = np.where((ids[t] >= 0) & (ids[t] < pool.shape[0]), ids[t], -1)
        seen = np.broadcast_to(there >= 0, (q.shape[1], len(there)))
        tol, toll = bound(sm.bf16_to_float(q[t]), there, pool, seen, scale, ref[t], refl[t])
        compare(out[t], lse[t], ref[t], refl[t], tol, toll, t)


SPARSE = {  # tokens, heads, list length, pool rows, query multiplier, share without a row
    "one": (1, 1, 1, 3, 1.0, 0.0), "k31": (2, 3, 31, 50, 1.0, 0.1), "k33": (2, 17, 33, 50, 1.0, 0.1),
    "k64_holes": (3, 32, 64, 90, 1.0, 0.9), "k1000": (2, 33, 1000, 3000, 1.0, 0.05),
    "k2048": (1, 128, 2048, 5000, 2.0, 0.0), "h129": (1, 129, 300, 700, 1.0, 0.02),
    "h300_k5000": (1, 300, 5000, 6000, 0.5, 0.02), "t300": (300, 16, 40, 500, 1.0, 0.1),
    "peaky": (2, 64, 777, 2000, 8.0, 0.02), "k9000": (1, 5, 9000, 20000, 1.0, 0.3),
}


@pytest.mark.parametrize("name", sorted(SPARSE))
def test_sparse(name):
    T, H, K, n, mult, holes = SPARSE[name]
    rs = np.random.default_rng(zlib.crc32(name.encode()))
    pool = make_pool(rs, n, 400)
    ids = rs.integers(0, n, (T, K)).astype(np.int32)
    gone = rs.random((T, K)) < holes
    ids[gone] = rs.choice(np.array([-1, -2, -3, n, 2 ** 31 - 1], np.int32), gone.sum())
    if K > 4:
        ids[0, 1] = ids[0, 0]                      # a duplicate counts twice
    check_sparse(pool, ids, bits(rs, T, H, 576, mult=mult), 1 / math.sqrt(192))


def test_sparse_nothing_selected():
    rs = np.random.default_rng(1)
    pool = make_pool(rs, 10, 400)
    pool[:, 256:272] = 255                         # every row NaN: none is selected
    ids = np.full((3, 70), -1, np.int32)
    out, lse = run_sparse(pool, ids, bits(rs, 3, 5, 576), 0.1)
    assert (out == 0).all() and np.isneginf(lse).all()
    out, lse = run_sparse(pool, np.zeros((2, 0), np.int32), bits(rs, 2, 5, 576), 0.1)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_sparse_nan_rows_and_large_scales():
    """A NaN row poisons the tokens that select it and no other; scales near both
    ends of E8M0 do not overflow what is finite."""
    rs = np.random.default_rng(2)
    pool = make_pool(rs, 200, 400)
    pool[7, 256 + 5] = 255
    ids = rs.integers(8, 200, (3, 100)).astype(np.int32)
    ids[1, 60] = 7
    q = bits(rs, 3, 20, 576)
    out, lse = run_sparse(pool, ids, q, 0.1)
    assert np.isnan(out[1]).all() and np.isnan(lse[1]).all()
    assert np.isfinite(out[[0, 2]]).all()
    pool[:, 256:272] = 127 - 60
    pool[3, 256:272] = 1                           # 2^-126
    check_sparse(pool, ids, q, 1.0)


def table(rs, R, pages, blocks, holes=0.0):
    bt = np.full((R, pages), -1, np.int32)
    flat = rs.permutation(blocks)[:R * pages]
    bt.reshape(-1)[:len(flat)] = flat
    gone = rs.random(bt.shape) < holes
    bt[gone] = rs.choice(np.array([-1, -5, blocks, 2 ** 31 - 1], np.int32), gone.sum())
    return bt


def run_paged(pool, bt, ctx, q, page, scale, max_ctx=None, layers=1, layer=0, stream=None):
    import serving_memory_tier_amd as hs
    R, P, H = q.shape[:3]
    rows = pool.shape[-2]
    max_ctx = int(max(list(ctx) + [0])) if max_ctx is None else max_ctx
    lay = hs.layout_of(page, pool.shape[-1], layers, page, rows, 0)
    gp, gb, gc, gq = dev(pool), dev(bt), dev(np.asarray(ctx, np.int32)), dev(q)
    batch = hs.batch_of(R, bt.shape[1], gp, None, gb, None, gc, None, None, None)
    out = torch.full((R, P, H, 512), -1, dtype=torch.int16, device="cuda")
    lse = torch.full((R, P, H), float("nan"), device="cuda")
    need = hs.hs_paged_mla_workspace_bytes(R, P, H, max_ctx)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if need else None
    print(f"[paged] fmt={pool.shape[-1]} R={R} P={P} H={H} max_ctx={max_ctx} page={page} ws={need}",
          flush=True)
    hs.hs_paged_mla_decode(lay, batch, layer, gq, P, H, max_ctx, scale, out, lse, ws, stream)
    torch.cuda.synchronize()
    return f64(out), lse.cpu().numpy().astype(np.float64)


def check_paged(pool, bt, ctx, q, page, scale, got=None, **kw):
    out, lse = run_paged(pool, bt, ctx, q, page, scale, **kw) if got is None else got
    if pool.ndim == 3:
        pool = pool[kw.get("layer", 0)]
    ref, refl = ol.paged_mla_decode(pool, bt, ctx, q, page, scale)
    R, P, H = q.shape[:3]
    for r in range(R):
        ids = ol.table_rows(bt[r], int(ctx[r]), page, pool.shape[0])
        t = np.arange(len(ids))
        for p in range(P):
            seen = np.broadcast_to((ids >= 0) & (t <= int(ctx[r]) - P + p), (H, len(ids)))
            tol, toll = bound(sm.bf16_to_float(q[r, p]), ids, pool, seen, scale, ref[r, p],
                              refl[r, p])
            compare(out[r, p], lse[r, p], ref[r, p], refl[r, p], tol, toll, (r, p))


PAGED = {  # contexts, positions, heads, page, share of pages without a block, query multiplier
    "one": ([1], 1, 1, 64, 0.0, 1.0), "empty": ([0, 5, 0], 1, 16, 64, 0.0, 1.0),
    "short": ([1, 2, 3, 4, 5], 4, 3, 16, 0.0, 1.0), "page1": ([70, 33], 2, 5, 1, 0.1, 1.0),
    "pages_inside_blocks": ([100, 257, 31], 3, 20, 8, 0.2, 1.0),
    "ragged": ([500, 333, 64, 65, 1023], 1, 16, 64, 0.0, 1.0),
    "verify_holes": ([700, 1500], 4, 64, 64, 0.3, 1.0), "h129": ([300], 1, 129, 64, 0.0, 1.0),
    "p9": ([40, 400], 9, 30, 64, 0.0, 1.0), "p70": ([100, 50], 70, 3, 64, 0.0, 1.0),
    "long": ([9000], 2, 70, 4096, 0.0, 1.0), "peaky": ([600, 601], 2, 40, 32, 0.05, 8.0),
    "many": ([37 * (i % 9) for i in range(300)], 1, 8, 16, 0.1, 1.0),
    "nothing_resident": ([100, 200], 2, 8, 64, 1.0, 1.0),
}


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", sorted(PAGED))
def test_paged(name, fmt):
    ctx, P, H, page, holes, mult = PAGED[name]
    rs = np.random.default_rng(zlib.crc32(name.encode()))
    R, pages = len(ctx), max(1, -(-max(ctx) // page))
    blocks = R * pages + 3
    pool = make_pool(rs, blocks * page, fmt)
    check_paged(pool, table(rs, R, pages, blocks, holes), ctx, bits(rs, R, P, H, 576, mult=mult),
                page, 1 / math.sqrt(192))


@pytest.mark.parametrize("fmt", FORMATS)
def test_paged_bounds_and_layers(fmt):
    """A context past the table or past max_ctx is cut; a loose max_ctx changes only
    rounding; another layer of the pool."""
    rs = np.random.default_rng(3)
    pool = make_pool(rs, 20 * 16, fmt)
    bt = table(rs, 2, 6, 20)
    q = bits(rs, 2, 2, 24, 576)
    check_paged(pool, bt, [96, 90], q, 16, 0.1, max_ctx=100000)
    # 110 tokens, 96 in the table: both positions see all of it
    out, lse = run_paged(pool, bt, [110, 110], q, 16, 0.1)
    ref, refl = ol.paged_mla_decode(pool, bt, [110, 110], q, 16, 0.1)
    assert np.abs(lse - refl).max() < 1e-4 and np.abs(out - ref).max() < 0.1
    # max_ctx 50 of 96 tokens: the first 50
    out, lse = run_paged(pool, bt, [96, 96], q, 16, 0.1, max_ctx=50)
    cut = np.full_like(bt, -1)
    cut[:, :3] = bt[:, :3]
    keep = pool.copy()
    refs = [ol.attend(sm.bf16_to_float(q[r, p]), *ol.decode_rows(
        keep[ol.table_rows(bt[r], 50, 16, 320)]), np.ones((24, 50), bool), 0.1)
        for r in range(2) for p in range(2)]
    assert np.abs(lse - np.stack([x[1] for x in refs]).reshape(2, 2, 24)).max() < 1e-4
    two = np.stack([pool[::-1], pool])
    check_paged(two, bt, [96, 90], q, 16, 0.1, layers=2, layer=1)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("R,H,longest,bound_", [(1, 8, 900, 900), (3, 8, 700, 60000), (3, 130, 900, 60000),
                                               (64, 5, 300, 3000), (64, 40, 200, 20000),
                                               (65, 5, 300, 3000), (33, 64, 400, 401),
                                               (130, 40, 200, 9000), (512, 3, 100, 3000),
                                               (513, 3, 100, 3000)])
def test_paged_splits_follow_contexts(fmt, R, H, longest, bound_):
    """Ragged contexts, none at all among them, under tight and loose bounds."""
    import serving_memory_tier_amd as hs
    rs = np.random.default_rng(R + H)
    assert hs.hs_paged_mla_workspace_bytes(R, 1, H, bound_) > 0
    page = 16
    ctx = [longest] + [int(x) for x in rs.integers(0, longest, R - 1)]
    if R > 2:
        ctx[1], ctx[-1] = 0, 1
    pages = -(-longest // page)
    pool = make_pool(rs, (R * pages + 1) * page, fmt)
    check_paged(pool, table(rs, R, pages, R * pages + 1), ctx, bits(rs, R, 1, H, 576), page, 0.05,
                max_ctx=bound_)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("where", ["latent", "rope", "scale"])
def test_paged_nan_rows(fmt, where):
    """A row with a NaN or an infinity makes the positions that see it NaN and leaves
    the earlier ones, and other requests, as they are; rows of pages that are not
    resident, or past the context, do not count at all."""
    if fmt == 400 and where == "latent":
        pytest.skip("E2M1 has no NaN")
    rs = np.random.default_rng(4)
    page, ctx, P, H = 16, [50, 60], 3, 20
    pool = make_pool(rs, 12 * page, fmt)
    bt = table(rs, 2, 4, 9)
    q = bits(rs, 2, P, H, 576)

    def poison(row):
        if where == "latent":
            pool[row, 300] = 0x7F
        elif where == "rope":
            pool[row, fmt - 10:fmt - 8] = [0x80, 0x7F]        # infinity
        elif fmt == 656:
            pool[row, 516:520] = np.array([np.inf], "<f4").view(np.uint8)
        else:
            pool[row, 256 + 9] = 255

    clean = run_paged(pool, bt, ctx, q, page, 0.1)
    for row in range(9 * page, 12 * page):                    # blocks of nobody
        poison(row)
    poison(bt[0, 3] * page + 2)                               # token 50: past the context
    same = run_paged(pool, bt, ctx, q, page, 0.1)
    assert (same[0] == clean[0]).all() and (same[1] == clean[1]).all()
    poison(bt[0, 49 // page] * page + 49 % page)              # seen by position 2 alone
    out, lse = run_paged(pool, bt, ctx, q, page, 0.1)
    # an infinite key may give a score of either infinity: not a number, or weight 1 or 0
    assert not np.isfinite(out[0, 2]).all(-1).any()
    assert (out[0, :2] == clean[0][0, :2]).all() and (lse[0, :2] == clean[1][0, :2]).all()
    assert (out[1] == clean[0][1]).all() and (lse[1] == clean[1][1]).all()


@pytest.mark.parametrize("power", [-60, 40])
@pytest.mark.parametrize("H", [5, 20, 40, 128])
@pytest.mark.parametrize("fmt", FORMATS)
def test_split_outputs_keep_their_range(fmt, H, power):
    """Latent values far from 1, over several key splits: the same relative error."""
    import serving_memory_tier_amd as hs
    rs = np.random.default_rng(6)
    ctx, page = 1500, 64
    assert hs.hs_paged_mla_workspace_bytes(1, 1, H, ctx) > H * 1048      # more than one
    pool = make_pool(rs, 24 * page, fmt)
    if fmt == 400:
        pool[:, 256:272] += np.uint8(power % 256)
    else:
        s = np.ascontiguousarray(pool[:, 512:528]).view("<f4") * np.float32(2.0 ** power)
        pool[:, 512:528] = s.view(np.uint8)
    bt = table(rs, 1, 24, 24)
    q = bits(rs, 1, 1, H, 576)
    if power > 0:                                  # scores of order 1
        q[..., :512] = ol.to_bf16(sm.bf16_to_float(q[..., :512]) * 2.0 ** -power)
    out, lse = run_paged(pool, bt, [ctx], q, page, 0.05)
    ref, refl = ol.paged_mla_decode(pool, bt, [ctx], q, page, 0.05)
    ids = ol.table_rows(bt[0], ctx, page, pool.shape[0])
    tol, toll = bound(sm.bf16_to_float(q[0, 0]), ids, pool, np.ones((H, ctx), bool), 0.05, ref[0, 0],
                      refl[0, 0])
    compare(out[0, 0], lse[0, 0], ref[0, 0], refl[0, 0],
            tol - 2.0 ** -30 + 2.0 ** (power - 30), toll, power)


def test_values_past_the_range_of_a_later_token():
    """A 4-bit row whose values overflow, in tokens that earlier positions do not
    see: no part in theirs."""
    rs = np.random.default_rng(7)
    for H in (16, 128):
        pool = make_pool(rs, 64, 400)
        bt, q = np.array([[0]], np.int32), bits(rs, 1, 3, H, 576)
        clean = run_paged(pool, bt, [50], q, 64, 0.1)
        for row, scale, code in ((49, 254, 0x44), (48, 253, 0x66)):
            pool[row, 256:272], pool[row, :256] = scale, code
        pool[50, 256:272], pool[50, :256] = 254, 0x77        # past the context
        out, lse = run_paged(pool, bt, [50], q, 64, 0.1)
        assert (out[0, 0] == clean[0][0, 0]).all() and (lse[0, 0] == clean[1][0, 0]).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H", [16, 32, 64, 128])
def test_scales_of_any_sign(fmt, H):
    """Negative scales, and zero: the average of the values seen."""
    rs = np.random.default_rng(H)
    pool, ctx = make_pool(rs, 40 * 16, fmt), [300, 90]
    bt, q = table(rs, 2, 19, 40), bits(rs, 2, 1, H, 576)
    check_paged(pool, bt, ctx, q, 16, -0.07)
    check_paged(pool, bt, ctx, q, 16, 0.0)


@pytest.mark.parametrize("fmt", FORMATS)
def test_offsets_past_32_bits(fmt):
    """Rows past the fourth gibibyte of a layer."""
    import serving_memory_tier_amd as hs
    rs = np.random.default_rng(5)
    page, H = 4096, 16
    blocks = (5 << 30) // (page * fmt)
    rows = blocks * page
    pool = torch.zeros((rows, fmt), dtype=torch.uint8, device="cuda")
    bt = np.array([[blocks - 1, blocks - 2]], np.int32)
    some = make_pool(rs, 2 * page, fmt)
    pool[-2 * page:] = dev(some)
    small = np.array([[1, 0]], np.int32)
    ctx, q = [5000], bits(rs, 1, 1, H, 576)
    gb, gc, gq = dev(bt), dev(np.asarray(ctx, np.int32)), dev(q)
    lay = hs.layout_of(page, fmt, 1, page, rows, 0)
    batch = hs.batch_of(1, 2, pool, None, gb, None, gc, None, None, None)
    out = torch.empty((1, 1, H, 512), dtype=torch.int16, device="cuda")
    lse = torch.empty((1, 1, H), device="cuda")
    ws = torch.empty(max(16, hs.hs_paged_mla_workspace_bytes(1, 1, H, 5000)), dtype=torch.uint8,
                     device="cuda")
    hs.hs_paged_mla_decode(lay, batch, 0, gq, 1, H, 5000, 0.1, out, lse, ws)
    got = f64(out), lse.cpu().numpy().astype(np.float64)
    check_paged(some, small, ctx, q, page, 0.1, got=got)
    if fmt == 400:
        ids = rs.integers(rows - 2 * page, rows, (1, 300)).astype(np.int32)
        o = torch.empty((1, H, 512), dtype=torch.int16, device="cuda")
        gi = dev(ids)
        ws = torch.empty(max(16, hs.hs_sparse_mla_fp4_workspace_bytes(1, H, 300)),
                         dtype=torch.uint8, device="cuda")
        hs.hs_sparse_mla_decode_fp4(lay, pool, gi, 1, 300, gq, H, 0.1, o, lse, ws)
        near = ids - (rows - 2 * page)
        want, wantl = ol.sparse_mla_decode(some, near, q[0], 0.1)
        tol, toll = bound(sm.bf16_to_float(q[0, 0]), near[0], some, np.ones((H, 300), bool), 0.1,
                          want[0], wantl[0])
        compare(f64(o)[0], lse.cpu().numpy()[0, 0].astype(np.float64), want[0], wantl[0], tol, toll,
                "sparse")
