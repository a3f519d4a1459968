"""CPU oracle for the latent-cache operators: row formats, rows appended with the
position rotation, attention over 4-bit rows, through the block table, and in
the expanded form.

TEST INFRASTRUCTURE ONLY.  Plain numpy in float64; it shares nothing with the
HIP library.  The FP8 row format is that of ``oracle.sparse_mla``; the 4-bit
row is 256 bytes of OCP E2M1 pairs (value 2 i in byte i's low half), 16 E8M0
scales, one per 32 values, then 64 bfloat16 rope values.
"""

from __future__ import annotations

import numpy as np

from . import sparse_mla as sm

FP8, FP4 = 656, 400
LATENT, ROPE = 512, 64
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
E2M1_16 = np.concatenate([E2M1, -E2M1])


def to_bf16(x: np.ndarray) -> np.ndarray:
    """float64 to bfloat16 bits: rounded to float32, then to bfloat16, each to
    nearest even."""
    b = np.asarray(x, np.float64).astype(np.float32).view(np.uint32)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def _nearest(x: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Index of the nearest value of an ascending grid, ties to the even index."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def scale_exponent(most: np.ndarray, limit: float) -> np.ndarray:
    """The smallest e >= -126 with most <= limit * 2^e, by stepping; 0 for 0."""
    e = np.full(most.shape, -126)
    while True:
        up = most > limit * 2.0 ** e
        if not up.any():
            return np.where(most == 0, 0, e)
        e = np.where(up, e + 1, e)


def encode_rows(latent_bits: np.ndarray, rope_bits: np.ndarray, row_bytes: int) -> np.ndarray:
    """bfloat16 bits [n, 512] and [n, 64] to rows uint8 [n, row_bytes]."""
    n = latent_bits.shape[0]
    x = sm.bf16_to_float(latent_bits)
    fp4 = row_bytes == FP4
    group = 32 if fp4 else 128
    g = x.reshape(n, -1, group)
    with np.errstate(invalid="ignore"):
        bad = ~np.isfinite(g).all(-1)
        most = np.where(bad, 0, np.abs(np.where(np.isfinite(g), g, 0)).max(-1))
        e = scale_exponent(most, 7.0 if fp4 else 448.0)
        y = np.where(bad[..., None], 0, g) * 2.0 ** -e[..., None].astype(np.float64)
    sign = (np.signbit(y) & ~bad[..., None]).reshape(n, LATENT)
    rows = np.zeros((n, row_bytes), np.uint8)
    if fp4:
        c = _nearest(np.minimum(np.abs(y), 6), E2M1).reshape(n, LATENT) | (sign << 3)
        rows[:, :256] = c[:, 0::2] | (c[:, 1::2] << 4)
        rows[:, 256:272] = np.where(bad, 255, e + 127)
        rows[:, 272:] = np.ascontiguousarray(rope_bits).view(np.uint8).reshape(n, 128)
    else:
        grid = np.array([sm.fp8_e4m3_value(b) for b in range(127)])
        c = _nearest(np.abs(y), grid).reshape(n, LATENT) | (sign << 7)
        rows[:, :512] = c
        s = np.where(bad, np.nan, 2.0 ** e.astype(np.float64)).astype("<f4")
        rows[:, 512:528] = np.ascontiguousarray(s).view(np.uint8).reshape(n, 16)
        rows[:, 528:] = np.ascontiguousarray(rope_bits).view(np.uint8).reshape(n, 128)
    return rows


def decode_rows(rows: np.ndarray):
    """uint8 [n, 656 or 400] -> (keys float64 [n, 576], values float64 [n, 512])."""
    rows = np.ascontiguousarray(rows, np.uint8)
    if rows.shape[1] == FP8:
        return sm.decode_rows(rows)
    n = rows.shape[0]
    b = rows[:, :256]
    lat = E2M1_16[np.stack([b & 15, b >> 4], -1).reshape(n, LATENT)]
    e = rows[:, 256:272].astype(np.float64)
    scale = np.where(e == 255, np.nan, 2.0 ** (e - 127))
    lat = lat * np.repeat(scale, 32, axis=1)
    rope = sm.bf16_to_float(rows[:, 272:].copy().view("<u2"))
    return np.concatenate([lat, rope], 1), lat


def rotate(x: np.ndarray, positions: np.ndarray, freq: np.ndarray, interleaved: bool):
    """float64 [n, ..., 64] rotated by positions [n] times freq [32], as complex products."""
    t = positions.astype(np.float64)[:, None] * freq
    t = t.reshape(t.shape[0], *(1,) * (x.ndim - 2), 32)
    z = x[..., 0::2] + 1j * x[..., 1::2] if interleaved else x[..., :32] + 1j * x[..., 32:]
    with np.errstate(invalid="ignore"):
        z = z * (np.cos(t) + 1j * np.sin(t))
    out = np.empty_like(x)
    if interleaved:
        out[..., 0::2], out[..., 1::2] = z.real, z.imag
    else:
        out[..., :32], out[..., 32:] = z.real, z.imag
    return out


def append_rows(block_table, page, pool_rows, token_req, positions):
    """The row of each token: -1 padding, -3 none."""
    R, pages = block_table.shape
    out = np.empty(len(token_req), np.int32)
    for i, (r, n) in enumerate(zip(token_req, positions)):
        out[i] = -1 if r < 0 else -3
        if 0 <= r < R and n >= 0 and n // page < pages:
            b = block_table[r, n // page]
            if 0 <= b < pool_rows // page:
                out[i] = b * page + n % page
    return out


def attend(q, k, v, seen, scale):
    """q [m, d], k [n, d], v [n, e], seen [m, n]: (out [m, e], lse [m]); a row
    that sees nothing gives 0 and -inf."""
    with np.errstate(all="ignore"):
        s = np.where(seen, scale * (q @ k.T), -np.inf)
        m = s.max(1, initial=-np.inf)
        w = np.where(seen, np.exp(s - np.where(np.isneginf(m), 0, m)[:, None]), 0)
        z = w.sum(1)
        v = np.where(seen.any(0)[:, None], v, 0)     # a row nobody sees says nothing
        return (w @ v) / np.where(z == 0, 1, z)[:, None], m + np.log(z)


def table_rows(block_table_row, ctx, page, pool_rows):
    """Row ids of tokens 0..ctx-1 of a request, -1 where there is none."""
    t = np.arange(min(ctx, len(block_table_row) * page))
    b = block_table_row[t // page].astype(np.int64)
    return np.where((b >= 0) & (b < pool_rows // page), b * page + t % page, -1)


def sparse_mla_decode(pool, row_ids, q_bits, scale):
    """As oracle.sparse_mla.sparse_mla_decode, for either row format."""
    T, H = q_bits.shape[:2]
    out, lse = np.zeros((T, H, LATENT)), np.full((T, H), -np.inf)
    for t in range(T):
        ids = row_ids[t].astype(np.int64)
        ids = ids[(ids >= 0) & (ids < pool.shape[0])]
        k, v = decode_rows(pool[ids])
        out[t], lse[t] = attend(sm.bf16_to_float(q_bits[t]), k, v,
                                np.ones((H, len(ids)), bool), scale)
    return out, lse


def paged_mla_decode(pool, block_table, ctx, q_bits, page, scale):
    """q_bits [R, P, H, 576]: position p of request r sees tokens t <= ctx - P + p."""
    R, P, H = q_bits.shape[:3]
    out, lse = np.zeros((R, P, H, LATENT)), np.full((R, P, H), -np.inf)
    for r in range(R):
        ids = table_rows(block_table[r], int(ctx[r]), page, pool.shape[0])
        t = np.arange(len(ids))
        k, v = decode_rows(pool[np.maximum(ids, 0)])
        for p in range(P):
            seen = np.broadcast_to((ids >= 0) & (t <= int(ctx[r]) - P + p), (H, len(ids)))
            out[r, p], lse[r, p] = attend(sm.bf16_to_float(q_bits[r, p]), k, v, seen, scale)
    return out, lse


def mla_prefill(pool, block_table, ctx, q_start, q_bits, w_bits, page, scale):
    """q_bits [N, H, 192], w_bits [H, 256, 512]: request r's queries q_start[r]..
    are its last tokens; out float64 [N, H, 128] (NaN where no request has the row)."""
    N, H = q_bits.shape[:2]
    out = np.full((N, H, 128), np.nan)
    w = sm.bf16_to_float(w_bits)
    for r in range(len(ctx)):
        lo, hi = int(q_start[r]), int(q_start[r + 1])
        ids = table_rows(block_table[r], int(ctx[r]), page, pool.shape[0])
        t = np.arange(len(ids))
        k, v = decode_rows(pool[np.maximum(ids, 0)])
        last = int(ctx[r]) - (hi - lo) + np.arange(hi - lo)
        seen = (ids >= 0)[None] & (t[None] <= last[:, None])
        for h in range(H):
            kh = np.concatenate([v @ w[h, :128].T, k[:, LATENT:]], 1)
            out[lo:hi, h] = attend(sm.bf16_to_float(q_bits[lo:hi, h]), kh, v @ w[h, 128:].T,
                                   seen, scale)[0]
    return out
