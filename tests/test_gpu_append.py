"""GPU parity of hs_mla_append with the oracle.  Rows are compared byte for byte
(scales are powers of two, so a code's rounding is the only one; the keys are
rotated in float64 and rounded to float32, then bfloat16).  A rotated query value is off by half a
bfloat16 step, 2^-8 |v| at most, and by float32: the sine and cosine, two
products and a sum, 2^-24 each of (|a| + |b|) at most, 4 * 2^-24 * sqrt(2) of
the pair's length -- 2^-21 of it is allowed."""

from __future__ import annotations

import os

import numpy as np
import pytest
import torch

from oracle import latent as ol
from oracle import sparse_mla as sm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import serving_memory_tier_amd as hs
    if not os.path.exists(hs.LIB_PATH):
        from serving_memory_tier_amd import build
        build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    hs.lib()


def bits(rs, *shape, mult=1.0):
    return ol.to_bf16(rs.standard_normal(shape) * mult)


def dev(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


FREQ = 10000.0 ** (-np.arange(32) / 32)


def tables(rs, R, pages, blocks):
    bt = np.full((R, pages), -1, np.int32)
    order = rs.permutation(blocks)[:R * pages]
    bt.reshape(-1)[:len(order)] = order
    return bt


def run(rs, fmt, interleaved, T, H, page=64, R=3, pages=5, longest=None, layers=1, layer=0,
        latent=None, stride=512, with_values=True, in_place=False, bt=None, req=None, pos=None,
        stream=None):
    """One call on random tokens at distinct positions against the oracle, every
    byte of the pool, the queries and the values compared."""
    import serving_memory_tier_amd as hs
    blocks = R * pages + 2
    bt = tables(rs, R, pages, blocks) if bt is None else bt
    if req is None:
        flat = rs.permutation(R * pages * page)[:T]
        req, pos = (flat // (pages * page)).astype(np.int32), (flat % (pages * page)).astype(np.int32)
    T = len(req)
    rows = blocks * page
    lat = bits(rs, T, stride)
    if latent is not None:
        lat[:, :512] = latent
    kv, q = bits(rs, T, 576), bits(rs, T, H, 192)
    pool = rs.integers(0, 256, (layers, rows, fmt)).astype(np.uint8)
    lay = hs.layout_of(page, fmt, layers, page, rows, 0)
    gp, gb = dev(pool), dev(bt)
    batch = hs.batch_of(R, pages, gp, None, gb, None, None, None, None, None)
    glat, gkv, gq = dev(lat), dev(kv), dev(q)
    mark = np.full((T, H, 576), 0x1234, np.uint16)
    gout = dev(mark) if not in_place else None
    qo = None if H == 0 else gq[:, :, 128:] if in_place else gout[:, :, 512:]
    call = hs.append_of(T, dev(req), dev(pos), glat[:, :512], gkv[:, 512:], dev(FREQ),
                        interleaved, gq[:, :, 128:] if H else None, qo)
    ids = torch.full((T,), 77, dtype=torch.int32, device="cuda")
    vals = dev(np.full((T, 576), 0x4321, np.uint16)) if with_values else None
    print(f"[append] fmt={fmt} T={T} H={H} page={page} il={interleaved}", flush=True)
    hs.hs_mla_append(lay, batch, layer, call, ids, vals, stream)
    torch.cuda.synchronize()
    want_ids = ol.append_rows(bt, page, rows, req, pos)
    assert (ids.cpu().numpy() == want_ids).all()
    ok = want_ids >= 0
    turned = ol.rotate(sm.bf16_to_float(kv[:, 512:]), pos, FREQ, interleaved)
    enc = ol.encode_rows(lat[:, :512], ol.to_bf16(turned), fmt)
    want = pool.copy()
    want[layer, want_ids[ok]] = enc[ok]
    got = gp.cpu().numpy()
    k, v = ol.decode_rows(enc)
    plain = ~np.isnan(k).any(1)
    # NaN scales have many bit patterns: those rows are compared as values
    check = np.ones((layers, rows), bool)
    check[layer, want_ids[ok & ~plain]] = False
    assert (got[check] == want[check]).all()
    for i in np.flatnonzero(ok & ~plain):
        gk, _ = ol.decode_rows(got[layer, want_ids[i]][None])
        assert np.array_equal(gk[0], k[i], equal_nan=True)
    if with_values:
        gv = vals.cpu().numpy().view(np.uint16)
        assert (gv[~ok] == 0x4321).all()
        x = sm.bf16_to_float(gv[ok])
        assert np.array_equal(x, sm.bf16_to_float(ol.to_bf16(k[ok])), equal_nan=True)
    if H:
        x = sm.bf16_to_float(q[:, :, 128:])
        ref = ol.rotate(x, pos, FREQ, interleaved)
        a, b = (ref[..., 0::2], ref[..., 1::2]) if interleaved else (ref[..., :32], ref[..., 32:])
        length = np.hypot(a, b)
        length = np.repeat(length, 2, -1) if interleaved else np.concatenate([length] * 2, -1)
        full = (gq if in_place else gout).cpu().numpy().view(np.uint16)
        part = full[:, :, 128:] if in_place else full[:, :, 512:]
        rest = full[:, :, :128] if in_place else full[:, :, :512]
        err = np.abs(sm.bf16_to_float(part[ok]) - ref[ok])
        assert (err <= 2.0 ** -8 * np.abs(ref[ok]) + 2.0 ** -21 * length[ok]).all()
        assert (part[~ok] == (q[:, :, 128:][~ok] if in_place else 0x1234)).all()
        assert (rest == (q[:, :, :128] if in_place else 0x1234)).all()


@pytest.mark.parametrize("fmt", [656, 400])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("T,H,page", [(1, 1, 64), (1, 0, 1), (7, 16, 16), (33, 128, 64),
                                      (5, 129, 4096), (300, 3, 64), (2, 300, 128)])
def test_shapes(fmt, interleaved, T, H, page):
    rs = np.random.default_rng(T * 1000 + H)
    run(rs, fmt, interleaved, T, H, page=page, pages=max(2, 700 // page))


@pytest.mark.parametrize("fmt", [656, 400])
def test_far_positions(fmt):
    """Positions up to two billion: the angles are reduced in float64."""
    rs = np.random.default_rng(5)
    pages = 1 << 19                     # 2^31 tokens of pages of 4,096
    bt = np.full((1, pages), -1, np.int32)
    pos = np.array([0, 1, 4095, 999999, 142000, 2 ** 31 - 1, 2 ** 31 - 4097, 1 << 24], np.int32)
    for i, n in enumerate(pos):
        bt[0, n // 4096] = n // 4096 % 5
    keep = [i for i in range(len(pos))]
    got = ol.append_rows(bt, 4096, 7 * 4096, np.zeros(len(pos), int), pos)
    seen = set()
    keep = [i for i in keep if not (got[i] in seen or seen.add(got[i]))]
    import serving_memory_tier_amd as hs
    lat, kv, q = bits(rs, len(keep), 512), bits(rs, len(keep), 64), bits(rs, len(keep), 4, 64)
    lay = hs.layout_of(4096, fmt, 1, 4096, 7 * 4096, 0)
    pool = torch.zeros((7 * 4096, fmt), dtype=torch.uint8, device="cuda")
    batch = hs.batch_of(1, pages, pool, None, dev(bt), None, None, None, None, None)
    gbt = dev(bt)
    batch.block_table = gbt.data_ptr()
    qo = torch.zeros((len(keep), 4, 64), dtype=torch.int16, device="cuda")
    call = hs.append_of(len(keep), dev(np.zeros(len(keep), np.int32)), dev(pos[keep]), dev(lat),
                        dev(kv), dev(FREQ), True, dev(q), qo)
    hs.hs_mla_append(lay, batch, 0, call)
    turned = ol.rotate(sm.bf16_to_float(kv), pos[keep], FREQ, True)
    rows = pool.cpu().numpy()[got[keep]]
    assert (rows == ol.encode_rows(lat, ol.to_bf16(turned), fmt)).all()
    ref = ol.rotate(sm.bf16_to_float(q), pos[keep], FREQ, True)
    err = np.abs(sm.bf16_to_float(qo.cpu().numpy().view(np.uint16)) - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -19).all()   # lengths below 4


@pytest.mark.parametrize("fmt", [656, 400])
def test_padding_and_tokens_without_a_row(fmt):
    rs = np.random.default_rng(6)
    R, pages, page = 3, 4, 16
    bt = tables(rs, R, pages, R * pages + 2)
    bt[0, 1], bt[1, 2], bt[2, 0] = -1, R * pages + 2, 2 ** 31 - 1    # null, outside, far outside
    req = np.array([0, 0, -1, 1, 1, 2, 2, 3, -7, 0, 1, 2 ** 31 - 1, 0], np.int32)
    pos = np.array([3, 20, 5, 40, 47, 2, 63, 1, -3, -1, 64, 0, 2 ** 31 - 1], np.int32)
    run(rs, fmt, True, 0, 5, page=page, R=R, pages=pages, bt=bt, req=req, pos=pos)


@pytest.mark.parametrize("fmt", [656, 400])
def test_value_extremes(fmt):
    """Zero groups, negative zeros, the largest and smallest bfloat16 values, ties,
    NaN and infinities: one group each, others beside them unharmed."""
    rs = np.random.default_rng(7)
    T, g = 24, 128 if fmt == 656 else 32
    lat = bits(rs, T, 512)
    lat[0] = 0
    lat[1] = 0x8000
    lat[2, :g] = 0x7F80                      # inf
    lat[3, g + 3] = 0x7FC0                   # NaN
    lat[4, 511] = 0xFF80                     # -inf, last group
    lat[5] = 0x7F7F                          # largest finite
    lat[6] = rs.integers(0, 128, 512)        # subnormals
    lat[7] = 0x0001
    lat[8] = bits(rs, 512, mult=2.0 ** -120)
    lat[9] = bits(rs, 512, mult=2.0 ** 120)
    lat[10] = ol.to_bf16(rs.integers(-56, 57, 512) / 8.0)      # E2M1 ties under scale 1
    lat[10, ::g] = ol.to_bf16(7.0)
    lat[11] = ol.to_bf16(rs.integers(-127, 128, 512) * 2.0 ** rs.integers(-8, 3, 512))
    lat[11, ::g] = ol.to_bf16(448.0)
    lat[12] = bits(rs, 512, mult=1.0)
    lat[12, 5] = ol.to_bf16(3e38)            # one value dwarfs its group
    for i in range(13, T):
        lat[i] = rs.integers(0, 0x7F80, 512) | (rs.integers(0, 2, 512) << 15)
    run(rs, fmt, False, T, 2, latent=lat)


def test_layers_strides_and_options():
    rs = np.random.default_rng(8)
    run(rs, 400, True, 40, 8, layers=3, layer=2)
    run(rs, 656, False, 40, 8, layers=2, layer=0, stride=520)
    run(rs, 400, True, 40, 8, with_values=False)
    run(rs, 656, True, 40, 130, in_place=True)
    run(rs, 400, False, 40, 16, in_place=True)
    run(rs, 656, True, 2000, 16, R=4, pages=20, stream=torch.cuda.Stream())


def test_no_tokens():
    import serving_memory_tier_amd as hs
    lay = hs.layout_of(64, 656, 1, 64, 64, 0)
    batch = hs.batch_of(0, 1, None, None, None, None, None, None, None, None)
    hs.hs_mla_append(lay, batch, 0, hs.HsAppend())
