"""GPU parity of hs_mla_prefill with the float64 oracle, within a bound the
arithmetic fixes.  Per (query, head), with p the probabilities, k and v the
expanded keys and values, A = sum_t p_t |v_t| and C_t = |W^V| |c_t|:
  - a key value is off by 2^-8 of itself (its rounding) plus 2^-8 |W^K| |c_t|
    where the latent values were rounded too, and by 600 * 2^-24 of that from
    float32 sums; a score by the scaled sum of |q| times those, plus 200 * 2^-24
    of the sum of |q| |k|: e at most over the keys seen; the probabilities then
    by a factor of exp(+-2 e);
  - the probabilities are rounded to bfloat16, 2^-8, the values likewise and,
    through the latent values, by 2^-8 C_t;
  - a key split's output is rounded to half precision, scaled so that its largest
    value is in [1, 2): 2^-11 A and 2^-25 max A; the output to bfloat16.
|d out| <= (exp(2 e) - 1 + 2 * 2^-8 + 2^-11) A + 2^-25 max A + (r 2^-8 + 2^-14) sum_t p_t C_t + 2^-8 |out| +
2^-30, r = 1 where scales are no powers of two, else 0.  This is the worst case;
the errors average over the keys, so the relative error of a whole output is
held to the root-sum-square of the five roundings to bfloat16 as well: 3^-0.5 *
2^-8 (the root mean square of a half step) * sqrt(5) * 1.5."""

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


def make_pool(rs, rows, fmt, odd_scales=False):
    pool = ol.encode_rows(bits(rs, rows, 512), bits(rs, rows, 64), fmt)
    if odd_scales and fmt == 656:
        s = np.ascontiguousarray(pool[:, 512:528]).view("<f4") * rs.uniform(0.6, 1.4, (rows, 4))
        pool[:, 512:528] = s.astype("<f4").view(np.uint8)
    return pool


def table(rs, R, pages, blocks, holes=0.0):
    bt = rs.permutation(blocks)[:R * pages].reshape(R, pages).astype(np.int32)
    gone = rs.random(bt.shape) < holes
    bt[gone] = rs.choice(np.array([-1, -5, blocks, 2 ** 31 - 1], np.int32), gone.sum())
    return bt


def run(pool, bt, ctx, start, q, w, page, scale, num_kv=None, layers=1, layer=0, stream=None,
        fill=0x1234):
    import serving_memory_tier_amd as hs
    N, H = q.shape[:2]
    R = len(ctx)
    num_kv = int(sum(max(c, 0) for c in ctx)) if num_kv is None else num_kv
    lay = hs.layout_of(page, pool.shape[-1], layers, page, pool.shape[-2], 0)
    keep = [dev(pool), dev(bt), dev(np.asarray(ctx, np.int32)), dev(np.asarray(start, np.int32)),
            dev(q), dev(w)]
    batch = hs.batch_of(R, bt.shape[1], keep[0], None, keep[1], None, keep[2], None, None, None)
    out = torch.full((N, H, 128), fill, dtype=torch.int16, device="cuda")
    need = hs.hs_mla_prefill_workspace_bytes(R, N, num_kv, H)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")     # NaN everywhere
    print(f"[prefill] fmt={pool.shape[-1]} R={R} N={N} H={H} num_kv={num_kv} ws={need}", flush=True)
    hs.hs_mla_prefill(lay, batch, layer, keep[3], N, num_kv, keep[4], H, keep[5], scale, out, ws,
                      stream)
    torch.cuda.synchronize()
    return sm.bf16_to_float(out.cpu().numpy().view(np.uint16))


def check(got, pool, bt, ctx, start, q, w, page, scale, rounded=False, floor=2.0 ** -30):
    ref = ol.mla_prefill(pool, bt, ctx, start, q, w, page, scale)
    wf, aw = sm.bf16_to_float(w), np.abs(sm.bf16_to_float(w))
    r8 = 2.0 ** -8 if rounded else 0.0
    mark = sm.bf16_to_float(np.array([0x1234], np.uint16))[0]
    free = np.ones(len(q), bool)
    for r in range(len(ctx)):
        lo, hi = int(start[r]), int(start[r + 1])
        free[lo:hi] = False
        ids = ol.table_rows(bt[r], int(ctx[r]), page, pool.shape[0])
        t = np.arange(len(ids))
        k, v = ol.decode_rows(pool[np.maximum(ids, 0)])
        seen = (ids >= 0)[None] & (t[None] <= (int(ctx[r]) - (hi - lo) + np.arange(hi - lo))[:, None])
        for h in range(q.shape[1]):
            qa = np.abs(sm.bf16_to_float(q[lo:hi, h]))
            c = np.abs(v)
            ck = np.concatenate([c @ aw[h, :128].T, np.zeros((len(ids), 64))], 1)
            kh = np.abs(np.concatenate([v @ wf[h, :128].T, k[:, 512:]], 1))
            e = abs(scale) * (qa[:, :128] @ (2.0 ** -8 * kh + (r8 + 600 * 2.0 ** -24) * ck)[:, :128].T
                         + 200 * 2.0 ** -24 * (qa @ kh.T))
            e = np.where(seen, e, 0).max(1, initial=0)[:, None]
            kk = np.concatenate([v @ wf[h, :128].T, k[:, 512:]], 1)
            vv = np.abs(v @ wf[h, 128:].T)
            both, _ = ol.attend(sm.bf16_to_float(q[lo:hi, h]), kk,
                                np.concatenate([vv, c @ aw[h, 128:].T], 1), seen, scale)
            tol = ((np.expm1(2 * e) + 2.0 ** -7 + 2.0 ** -11) * both[:, :128]
                   + 2.0 ** -25 * both[:, :128].max(1, keepdims=True)
                   + (r8 + 2.0 ** -14) * both[:, 128:] + 2.0 ** -8 * np.abs(ref[lo:hi, h])
                   + floor)
            err = np.abs(got[lo:hi, h] - ref[lo:hi, h])
            assert (err <= tol).all(), (r, h, err.max(), tol[err > tol].min())
        if hi > lo and seen.any():
            x, y = got[lo:hi], ref[lo:hi]
            assert np.linalg.norm(x - y) <= 3 ** -0.5 * 2.0 ** -8 * 5 ** 0.5 * 1.5 * np.linalg.norm(y)
    assert (got[free] == mark).all()


CASES = {  # (contexts, new tokens, heads, page, share of pages without a block)
    "one": ([1], [1], 1, 64, 0.0), "no_context": ([0, 5], [3, 2], 2, 64, 0.0),
    "more_new_than_context": ([3, 10], [7, 10], 3, 16, 0.0),
    "some_without_queries": ([40, 0, 100, 7, 64], [0, 0, 33, 0, 64], 2, 16, 0.0),
    "tile_edges": ([64, 65, 128, 129, 63], [64, 65, 128, 129, 63], 2, 64, 0.0),
    "chunk": ([700], [300], 3, 64, 0.0), "chunk_aligned": ([1024], [512], 2, 128, 0.0),
    "holes": ([500, 333], [100, 333], 3, 8, 0.3), "page1": ([90, 70], [90, 20], 2, 1, 0.1),
    "nothing_resident": ([100], [40], 2, 64, 1.0), "short_on_long": ([2500], [3], 5, 4096, 0.0),
    "heads9": ([150, 200], [150, 200], 9, 64, 0.0), "many": ([5 * i for i in range(70)],
                                                             [i % 7 for i in range(70)], 2, 16, 0.0),
    "reqs64": ([(11 * i) % 90 for i in range(64)], [i % 5 for i in range(64)], 1, 16, 0.0),
    "reqs65": ([(11 * i) % 90 for i in range(65)], [i % 5 for i in range(65)], 1, 16, 0.0),
    # tiles of 256 queries and of 256 tokens: many heads, more queries
    "heads128": ([700], [300], 128, 64, 0.0), "heads64_holes": ([600, 900], [600, 520], 64, 64, 0.1),
}


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", sorted(CASES))
def test_prefill(name, fmt):
    ctx, new, H, page, holes = CASES[name]
    rs = np.random.default_rng(zlib.crc32(name.encode()))
    R, pages = len(ctx), max(1, -(-max(ctx) // page))
    blocks = R * pages + 2
    pool = make_pool(rs, blocks * page, fmt)
    bt = table(rs, R, pages, blocks, holes)
    start = np.concatenate([[0], np.cumsum(new)])
    q, w = bits(rs, sum(new) + 3, H, 192), bits(rs, H, 256, 512, mult=512 ** -0.5)
    args = pool, bt, ctx, start, q, w, page, 192 ** -0.5
    check(run(*args), *args)


@pytest.mark.parametrize("fmt", FORMATS)
def test_peaky_scales_layers_and_loose_bounds(fmt):
    """Scores of many units, scales that are no powers of two, another layer, a loose
    num_kv, queries that start past row 0, a second stream."""
    rs = np.random.default_rng(9)
    page, ctx = 32, [300, 280]
    pool = make_pool(rs, 24 * page, fmt, odd_scales=True)
    bt = table(rs, 2, 11, 24)
    q, w = bits(rs, 100, 3, 192, mult=3.0), bits(rs, 3, 256, 512, mult=512 ** -0.5)
    start = [5, 60, 90]
    args = bt, ctx, start, q, w, page, 192 ** -0.5
    two = np.stack([pool[::-1], pool])
    got = run(two, *args, num_kv=1000, layers=2, layer=1, stream=torch.cuda.Stream())
    check(got, pool, *args, rounded=True)


def test_short_bounds_cut_instead_of_overrunning():
    """num_kv below the contexts' sum: earlier requests are whole, later ones cut;
    q_start outside its range reads and writes nothing outside."""
    rs = np.random.default_rng(10)
    page = 16
    pool = make_pool(rs, 20 * page, 400)
    bt = table(rs, 2, 9, 20)
    q, w = bits(rs, 40, 2, 192), bits(rs, 2, 256, 512, mult=512 ** -0.5)
    args = bt, [100, 140], [0, 20, 40], q, w, page, 192 ** -0.5
    full, cut = run(pool, *args), run(pool, *args, num_kv=130)
    assert (full[:20] == cut[:20]).all() and not (full[20:] == cut[20:]).all()
    assert np.isfinite(cut).all()
    for start in ([0, 20, 10 ** 9], [-7, 20, 40], [40, 20, 0], [0, 40, 40]):
        run(pool, bt, [100, 140], start, q, w, page, 192 ** -0.5)


@pytest.mark.parametrize("fmt", FORMATS)
def test_nan_rows_reach_only_who_sees_them(fmt):
    rs = np.random.default_rng(11)
    page, ctx, start = 16, [200, 190], [0, 150, 190]
    pool = make_pool(rs, 32 * page, fmt)
    bt = table(rs, 2, 13, 30)
    q, w = bits(rs, 190, 3, 192), bits(rs, 3, 256, 512, mult=512 ** -0.5)
    args = bt, ctx, start, q, w, page, 0.07
    clean = run(pool, *args)

    def poison(row):
        if fmt == 656:
            pool[row, 516:520] = np.array([np.nan], "<f4").view(np.uint8)
        else:
            pool[row, 256 + 3] = 255

    for row in range(30 * page, 32 * page):
        poison(row)
    poison(bt[0, 12] * page + 8)                           # token 200: past the context
    same = run(pool, *args)
    assert (same == clean).all()
    poison(bt[0, 120 // page] * page + 120 % page)         # token 120: queries 70 and on
    got = run(pool, *args)
    assert np.isnan(got[70:150]).all()
    assert (got[:70] == clean[:70]).all() and (got[150:] == clean[150:]).all()
    pool[bt[1, 189 // page] * page + 189 % page, -2:] = [0x80, 0x7F]     # rope infinity, last token
    got = run(pool, *args)
    assert np.isnan(got[189]).all() and (got[150:189] == clean[150:189]).all()


@pytest.mark.parametrize("power", [-60, 40])
@pytest.mark.parametrize("fmt", FORMATS)
def test_split_outputs_keep_their_range(fmt, power):
    """Latent values far from 1, over several key splits: the same relative error."""
    import serving_memory_tier_amd as hs
    rs = np.random.default_rng(8)
    page, ctx, new, H = 64, [1500], [20], 4
    size = hs.hs_mla_prefill_workspace_bytes(1, 20, 1500, H)
    assert size > 1500 * (1024 + 128 + 512 * H) + 2 * 20 * H * 128 * 2       # more than one
    rows = 24 * page
    pool = ol.encode_rows(ol.to_bf16(rs.standard_normal((rows, 512)) * 2.0 ** power),
                          bits(rs, rows, 64), fmt)
    q = bits(rs, 20, H, 192)
    if power > 0:                                  # scores of order 1
        q[..., :128] = ol.to_bf16(sm.bf16_to_float(q[..., :128]) * 2.0 ** -power)
    w, start = bits(rs, H, 256, 512, mult=0.05), [0, 20]
    bt = table(rs, 1, 24, 24)
    got = run(pool, bt, ctx, start, q, w, page, 0.05)
    check(got, pool, bt, ctx, start, q, w, page, 0.05, floor=2.0 ** (power - 30))


@pytest.mark.parametrize("fmt", FORMATS)
def test_scales_of_any_sign(fmt):
    """Negative scales, and zero: the average of the values seen."""
    rs = np.random.default_rng(9)
    page, ctx, start, H = 16, [300, 90], [0, 150, 240], 3
    pool = make_pool(rs, 40 * page, fmt)
    bt = table(rs, 2, 19, 40, holes=0.1)
    q, w = bits(rs, 240, H, 192), bits(rs, H, 256, 512, mult=0.05)
    for scale in (-0.07, 0.0):
        got = run(pool, bt, ctx, start, q, w, page, scale)
        check(got, pool, bt, ctx, start, q, w, page, scale)
