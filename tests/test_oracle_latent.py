"""Pins of the latent-cache oracle: values the formats fix, a hand-built 4-bit
row, the rounding rules, and the rotation's group property."""

from __future__ import annotations

import numpy as np

from oracle import latent as ol
from oracle import sparse_mla as sm


def bf(x):
    return ol.to_bf16(np.asarray(x, np.float64))


def test_hand_built_fp4_row():
    row = np.zeros((1, 400), np.uint8)
    row[0, 0] = 0x7A          # values 0 and 1: code 10 = -1, code 7 = 6
    row[0, 17] = 0x05         # values 34, 35: code 5 = 3, 0
    row[0, 256], row[0, 257] = 127, 130
    row[0, 258] = 255
    row[0, 272:274] = bf(1.5).reshape(1).view(np.uint8)
    k, v = ol.decode_rows(row)
    assert v[0, 0] == -1 and v[0, 1] == 6 and v[0, 34] == 24 and v[0, 35] == 0
    assert np.isnan(v[0, 64:96]).all() and not np.isnan(v[0, 96:]).any()
    assert k[0, 512] == 1.5 and (k[0, :64] == v[0, :64]).all()


def test_rounding_to_codes():
    # a group whose largest value is 7 keeps scale 1 and rounds 7 to 6; just above, scale 2
    for most, e in ((7.0, 0), (7.0625, 1), (6.0, 0), (3.5, -1), (0.0, 0), (2.0 ** -133, -126)):
        assert ol.scale_exponent(np.array([most]), 7.0)[0] == e, most
    assert ol.scale_exponent(np.array([448.0]), 448.0)[0] == 0
    assert ol.scale_exponent(np.array([450.0]), 448.0)[0] == 1
    x = np.zeros((1, 512))
    x[0, :12] = [7, 0.25, 0.26, 0.75, -1.25, 1.75, 2.5, -3.5, 5, 5.03125, -0.2, 6]
    rows = ol.encode_rows(bf(x), np.zeros((1, 64), np.uint16), 400)
    _, v = ol.decode_rows(rows)
    assert v[0, :12].tolist() == [6, 0, 0.5, 1, -1, 2, 2, -4, 4, 6, 0, 6]
    assert np.signbit(v[0, 10])
    x[0, 0] = np.inf
    _, v = ol.decode_rows(ol.encode_rows(bf(x), np.zeros((1, 64), np.uint16), 400))
    assert np.isnan(v[0, :32]).all() and (v[0, 32:] == 0).all()


def test_encode_is_idempotent_and_within_half_a_step():
    rs = np.random.default_rng(1)
    x = rs.standard_normal((20, 512)) * np.exp2(rs.integers(-20, 20, (20, 1)))
    for fmt, half in ((656, 2.0 ** -4), (400, 2.0 ** -2)):
        rows = ol.encode_rows(bf(x), np.zeros((20, 64), np.uint16), fmt)
        _, v = ol.decode_rows(rows)
        xb = sm.bf16_to_float(bf(x))
        g = 128 if fmt == 656 else 32
        most = np.repeat(np.abs(xb).reshape(20, -1, g).max(-1), g, 1)
        small = 2.0 ** -9 if fmt == 656 else 2.0 ** -2      # half the smallest step, unscaled
        top = 224 if fmt == 656 else 3.5                     # the scaled maximum is above this
        assert (np.abs(v - xb) <= half * np.abs(xb) + small * most / top).all()
        again = ol.encode_rows(bf(v), np.zeros((20, 64), np.uint16), fmt)
        assert (ol.decode_rows(again)[1] == v).all()


def test_rotation():
    rs = np.random.default_rng(2)
    x = rs.standard_normal((5, 3, 64))
    f = 10000.0 ** (-np.arange(32) / 32)
    n = np.array([0, 1, 5, 1000, 999999])
    for il in (True, False):
        y = ol.rotate(x, n, f, il)
        assert (y[0] == x[0]).all()
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        assert np.allclose(ol.rotate(ol.rotate(x, n, f, il), 2 * n, f, il),
                           ol.rotate(x, 3 * n, f, il), atol=1e-8)
    # position 1, frequency pi / 2: (a, b) -> (-b, a)
    q = ol.rotate(x[:1], np.array([1]), np.full(32, np.pi / 2), True)
    assert np.allclose(q[..., 0::2], -x[:1, :, 1::2]) and np.allclose(q[..., 1::2], x[:1, :, 0::2])


def test_attention_forms_agree():
    """The paged form over a request equals the sparse form over its rows, and the
    expanded form equals the absorbed one with the weights moved over."""
    rs = np.random.default_rng(3)
    page, n = 4, 21
    pool = ol.encode_rows(bf(rs.standard_normal((40, 512))), bf(rs.standard_normal((40, 64))), 400)
    bt = np.array([[3, 1, 9, 0, 5, 2]], np.int32)
    q = bf(rs.standard_normal((1, 2, 3, 576)))
    out, lse = ol.paged_mla_decode(pool, bt, [n], q, page, 0.1)
    ids = ol.table_rows(bt[0], n, page, 40)
    o, l = ol.sparse_mla_decode(pool, np.stack([np.append(ids[:-1], -1), ids]), q[0], 0.1)
    assert np.allclose(out[0], o) and np.allclose(lse[0], l)
    w = bf(rs.standard_normal((2, 256, 512)) / 20)
    qe = bf(rs.standard_normal((2, 2, 192)))
    e = ol.mla_prefill(pool, bt, [n], [0, 2], qe, w, page, 0.1)
    wf, qf = sm.bf16_to_float(w), sm.bf16_to_float(qe)
    k, v = ol.decode_rows(pool[ids])
    for i in range(2):
        for h in range(2):
            qa = np.concatenate([qf[i, h, :128] @ wf[h, :128], qf[i, h, 128:]])
            seen = np.arange(n)[None] <= n - 2 + i
            a, _ = ol.attend(qa[None], k, v, seen, 0.1)
            assert np.allclose(a[0] @ wf[h, 128:].T, e[i, h])
    # a context shorter than its positions: nothing seen
    out, lse = ol.paged_mla_decode(pool, bt, [1], q, page, 0.1)
    assert (out[0, 0] == 0).all() and np.isneginf(lse[0, 0]).all() and np.isfinite(lse[0, 1]).all()
