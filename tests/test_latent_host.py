"""Host-side checks of the latent-cache operators (no GPU): the struct mirror, and
every refusal before anything is enqueued."""

from __future__ import annotations

import ctypes
import os
import subprocess

import pytest
import torch

import serving_memory_tier_amd as hs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x1000      # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(hs.LIB_PATH):
        from serving_memory_tier_amd import build
        build.build()
    return hs.lib()


def layout(**kw):
    d = dict(page_size=64, row_bytes=656, num_layers=2, hot_capacity=64, pool_rows=6400,
             host_rows=0)
    d.update(kw)
    return hs.layout_of(**d)


def batch(**kw):
    b = hs.batch_of(2, 16, FAKE, None, FAKE, None, FAKE, None, None, None)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def test_append_struct_mirrors_header(tmp_path):
    names = [n for n, _ in hs.HsAppend._fields_]
    src = ('#include <stddef.h>\n#include <stdio.h>\n#include "hisparse.h"\nint main(void) {\n'
           '  printf("%zu %d %d", sizeof(hs_append), HS_ROW_FP8, HS_ROW_FP4);\n'
           + "".join(f'  printf(" %zu", offsetof(hs_append, {n}));\n' for n in names)
           + "  return 0;\n}\n")
    c = tmp_path / "s.c"
    c.write_text(src)
    subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I",
                    "/opt/rocm/include", str(c), "-o", str(tmp_path / "s")], check=True,
                   capture_output=True)
    out = [int(x) for x in subprocess.run([str(tmp_path / "s")], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert out == [ctypes.sizeof(hs.HsAppend), hs.HS_ROW_FP8, hs.HS_ROW_FP4] + [
        getattr(hs.HsAppend, n).offset for n in names]


def append(**kw):
    a = hs.HsAppend(4, 2, FAKE, FAKE, FAKE, 512, FAKE, 64, FAKE, FAKE, 128, 64, FAKE, 128, 64, 1, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("lay,bat,layer,app,row_ids,values,code", [
    (dict(page_size=48), {}, 0, {}, FAKE, FAKE, 1),
    (dict(row_bytes=640), {}, 0, {}, FAKE, FAKE, 2),
    ({}, {}, -1, {}, FAKE, FAKE, 1), ({}, {}, 2, {}, FAKE, FAKE, 1),
    ({}, dict(num_reqs=-1), 0, {}, FAKE, FAKE, 1), ({}, dict(max_pages=0), 0, {}, FAKE, FAKE, 1),
    ({}, dict(kv_pool=None), 0, {}, FAKE, FAKE, 1), ({}, dict(kv_pool=0x1008), 0, {}, FAKE, FAKE, 1),
    ({}, dict(block_table=None), 0, {}, FAKE, FAKE, 1),
    ({}, {}, 0, dict(num_tokens=-1), FAKE, FAKE, 1), ({}, {}, 0, dict(num_heads=-1), FAKE, FAKE, 1),
    ({}, {}, 0, dict(num_heads=(1 << 20) + 1), FAKE, FAKE, 2),
    ({}, {}, 0, dict(token_req=None), FAKE, FAKE, 1), ({}, {}, 0, dict(positions=None), FAKE, FAKE, 1),
    ({}, {}, 0, dict(latent=None), FAKE, FAKE, 1), ({}, {}, 0, dict(latent=0x1008), FAKE, FAKE, 1),
    ({}, {}, 0, dict(latent_stride=516), FAKE, FAKE, 1),
    ({}, {}, 0, dict(latent_stride=-512), FAKE, FAKE, 1),
    ({}, {}, 0, dict(rope=None), FAKE, FAKE, 1), ({}, {}, 0, dict(rope_stride=-1), FAKE, FAKE, 1),
    ({}, {}, 0, dict(rope_freq=None), FAKE, FAKE, 1),
    ({}, {}, 0, dict(q_rope=None), FAKE, FAKE, 1), ({}, {}, 0, dict(q_out=None), FAKE, FAKE, 1),
    ({}, {}, 0, dict(q_rope=0x1002), FAKE, FAKE, 1), ({}, {}, 0, dict(q_out=0x1002), FAKE, FAKE, 1),
    ({}, {}, 0, dict(q_head_stride=68), FAKE, FAKE, 1),
    ({}, {}, 0, dict(q_out_token_stride=130), FAKE, FAKE, 1),
    ({}, {}, 0, dict(q_out_token_stride=56), FAKE, FAKE, 1),
    ({}, {}, 0, dict(q_out_head_stride=0), FAKE, FAKE, 1),
    ({}, {}, 0, dict(rope_interleaved=2), FAKE, FAKE, 1), ({}, {}, 0, dict(reserved=1), FAKE, FAKE, 1),
    ({}, {}, 0, {}, FAKE, 0x1008, 1),
])
def test_append_refusals(lib, lay, bat, layer, app, row_ids, values, code):
    lay, bat, app = layout(**lay), batch(**bat), append(**app)
    assert lib.hs_mla_append(ctypes.byref(lay), ctypes.byref(bat), layer, ctypes.byref(app),
                             row_ids, values, None) == code


def test_append_null_structs(lib):
    lay, bat, app = layout(), batch(), append()
    r = ctypes.byref
    assert lib.hs_mla_append(None, r(bat), 0, r(app), FAKE, FAKE, None) == 1
    assert lib.hs_mla_append(r(lay), None, 0, r(app), FAKE, FAKE, None) == 1
    assert lib.hs_mla_append(r(lay), r(bat), 0, None, FAKE, FAKE, None) == 1
    assert lib.hs_mla_append(r(lay), r(bat), 0, r(append(num_tokens=0)), None, None, None) == 0


def test_append_binding_refuses_wrong_tensors():
    t = torch.zeros
    i32, bf, f64 = torch.int32, torch.bfloat16, torch.float64
    args = lambda **kw: {**dict(num_tokens=2, token_req=t(2, dtype=i32), positions=t(2, dtype=i32),
                                latent=t(2, 512, dtype=bf), rope=t(2, 64, dtype=bf),
                                rope_freq=t(32, dtype=f64), rope_interleaved=True), **kw}
    with pytest.raises(ValueError, match="shape"):
        hs.append_of(**args(latent=t(2, 576, dtype=bf)))
    with pytest.raises(ValueError, match="go together"):
        hs.append_of(**args(q_rope=t(2, 4, 64, dtype=bf)))
    with pytest.raises(ValueError, match="last dimension"):
        hs.append_of(**args(rope=t(64, 2, dtype=bf).t()))
    with pytest.raises(TypeError, match="token_req"):
        hs.append_of(**args(token_req=t(2, dtype=torch.int64)))
    with pytest.raises(ValueError, match="current CUDA device"):
        hs.append_of(**args())              # host tensors


def test_append_too_many_tokens(lib):
    r = ctypes.byref
    assert lib.hs_mla_append(r(layout()), r(batch()), 0, r(append(num_tokens=2 ** 31 - 1)), FAKE,
                             FAKE, None) == 2


BIG = 1 << 40      # a workspace's stated size


@pytest.mark.parametrize("lay,kw,code", [
    (dict(page_size=48), {}, 1), ({}, {}, 2), (dict(row_bytes=656), {}, 2),
    (dict(row_bytes=416), {}, 2),
] + [(dict(row_bytes=400), kw, code) for kw, code in [
    (dict(tokens=-1), 1), (dict(k=-1), 1), (dict(heads=0), 1), (dict(heads=-3), 1),
    (dict(tokens=(1 << 20) + 1), 2), (dict(k=(1 << 20) + 1), 2), (dict(heads=(1 << 20) + 1), 2),
    (dict(kv=None), 1), (dict(kv=0x1008), 1), (dict(ids=None), 1), (dict(q=None), 1),
    (dict(q=0x1008), 1), (dict(out=None), 1), (dict(out=0x1002), 1), (dict(lse=None), 1),
    (dict(lse=0x1002), 1), (dict(ws=None), 1), (dict(ws=0x1008), 1), (dict(size=0), 1),
    (dict(size="short"), 1), (dict(tokens=1 << 20, heads=1 << 20), 2), (dict(tokens=0), 0),
    (dict(tokens=0, kv=None, ids=None, q=None, out=None, lse=None, ws=None), 0),
]])
def test_sparse_refusals(lib, lay, kw, code):
    a = dict(kv=FAKE, ids=FAKE, tokens=2, k=5000, q=FAKE, heads=16, out=FAKE, lse=FAKE, ws=FAKE,
             size=BIG)
    a.update(kw)
    need = lib.hs_sparse_mla_fp4_workspace_bytes(a["tokens"], a["heads"], a["k"])
    if a["size"] == "short":
        a["size"] = need - 1
    l = layout(**lay)
    assert lib.hs_sparse_mla_decode_fp4(ctypes.byref(l), a["kv"], a["ids"], a["tokens"], a["k"],
                                        a["q"], a["heads"], 1.0, a["out"], a["lse"], a["ws"],
                                        a["size"], None) == code
    assert lib.hs_sparse_mla_decode_fp4(None, FAKE, FAKE, 1, 1, FAKE, 1, 1.0, FAKE, FAKE, None, 0,
                                        None) == 1


@pytest.mark.parametrize("lay,bat,kw,code", [
    (dict(page_size=0), {}, {}, 1), (dict(row_bytes=640), {}, {}, 2),
    ({}, {}, dict(layer=-1), 1), ({}, {}, dict(layer=2), 1),
    ({}, dict(num_reqs=-1), {}, 1), ({}, dict(max_pages=0), {}, 1), ({}, dict(kv_pool=None), {}, 1),
    ({}, dict(kv_pool=0x1008), {}, 1), ({}, dict(block_table=None), {}, 1),
    ({}, dict(ctx_len=None), {}, 1), ({}, {}, dict(pos=0), 1), ({}, {}, dict(heads=0), 1),
    ({}, {}, dict(ctx=-1), 1), ({}, {}, dict(pos=1 << 11, heads=1 << 10), 2),
    ({}, {}, dict(pos=2 ** 31 - 1, heads=2 ** 31 - 1), 2),
    ({}, {}, dict(q=None), 1), ({}, {}, dict(q=0x1008), 1), ({}, {}, dict(out=None), 1),
    ({}, {}, dict(out=0x1008), 1), ({}, {}, dict(lse=None), 1), ({}, {}, dict(lse=0x1001), 1),
    ({}, {}, dict(ws=None), 1),
    ({}, {}, dict(ws=0x1008), 1), ({}, {}, dict(size="short"), 1),
    ({}, dict(num_reqs=2 ** 31 - 1), dict(size=1 << 62), 2),
    ({}, dict(num_reqs=0), dict(q=None, out=None, ws=None), 0),
])
def test_paged_refusals(lib, lay, bat, kw, code):
    a = dict(layer=1, q=FAKE, pos=1, heads=16, ctx=5000, out=FAKE, lse=FAKE, ws=FAKE, size=BIG)
    a.update(kw)
    l, b = layout(**lay), batch(**{**dict(ctx_len=FAKE), **bat})
    if a["size"] == "short":
        a["size"] = lib.hs_paged_mla_workspace_bytes(b.num_reqs, a["pos"], a["heads"], a["ctx"]) - 1
    f = lib.hs_paged_mla_decode
    assert f(ctypes.byref(l), ctypes.byref(b), a["layer"], a["q"], a["pos"], a["heads"], a["ctx"],
             1.0, a["out"], a["lse"], a["ws"], a["size"], None) == code
    assert f(ctypes.byref(l), None, 0, FAKE, 1, 1, 1, 1.0, FAKE, FAKE, None, 0, None) == 1
    assert f(None, ctypes.byref(b), 0, FAKE, 1, 1, 1, 1.0, FAKE, FAKE, None, 0, None) == 1


@pytest.mark.parametrize("lay,bat,kw,code", [
    (dict(page_size=0), {}, {}, 1), (dict(row_bytes=640), {}, {}, 2),
    ({}, {}, dict(layer=-1), 1), ({}, {}, dict(layer=2), 1),
    ({}, dict(num_reqs=-1), {}, 1), ({}, dict(max_pages=0), {}, 1), ({}, dict(kv_pool=None), {}, 1),
    ({}, dict(kv_pool=0x1008), {}, 1), ({}, dict(block_table=None), {}, 1),
    ({}, dict(ctx_len=None), {}, 1), ({}, {}, dict(start=None), 1), ({}, {}, dict(num_q=-1), 1),
    ({}, {}, dict(start=0x1002), 1),
    ({}, {}, dict(num_kv=-1), 1), ({}, {}, dict(heads=0), 1), ({}, {}, dict(heads=(1 << 20) + 1), 2),
    ({}, dict(num_reqs=(1 << 20) + 1), {}, 2), ({}, {}, dict(q=None), 1), ({}, {}, dict(q=0x1008), 1),
    ({}, {}, dict(w=None), 1), ({}, {}, dict(w=0x1008), 1), ({}, {}, dict(out=None), 1),
    ({}, {}, dict(out=0x1008), 1), ({}, {}, dict(ws=None), 1), ({}, {}, dict(ws=0x1008), 1),
    ({}, {}, dict(size="short"), 1), ({}, {}, dict(num_q=2 ** 31 - 1, size=1 << 62), 2),
    ({}, {}, dict(num_kv=2 ** 31 - 1, size=1 << 62), 2),
    ({}, {}, dict(num_kv=65535 * 128 + 1, size=1 << 62), 2),
    ({}, {}, dict(num_q=0, q=None, out=None, ws=None), 0),
    ({}, dict(num_reqs=0), dict(q=None, out=None, ws=None), 0),
])
def test_prefill_refusals(lib, lay, bat, kw, code):
    a = dict(layer=0, start=FAKE, num_q=100, num_kv=300, q=FAKE, heads=4, w=FAKE, out=FAKE, ws=FAKE,
             size=BIG)
    a.update(kw)
    l, b = layout(**lay), batch(**{**dict(ctx_len=FAKE), **bat})
    if a["size"] == "short":
        a["size"] = lib.hs_mla_prefill_workspace_bytes(b.num_reqs, a["num_q"], a["num_kv"],
                                                       a["heads"]) - 1
    f = lib.hs_mla_prefill
    assert f(ctypes.byref(l), ctypes.byref(b), a["layer"], a["start"], a["num_q"], a["num_kv"],
             a["q"], a["heads"], a["w"], 1.0, a["out"], a["ws"], a["size"], None) == code
    assert f(ctypes.byref(l), None, 0, FAKE, 1, 1, FAKE, 1, FAKE, 1.0, FAKE, FAKE, BIG, None) == 1
    assert f(None, ctypes.byref(b), 0, FAKE, 1, 1, FAKE, 1, FAKE, 1.0, FAKE, FAKE, BIG, None) == 1


def test_workspace_sizes(lib):
    assert hs.hs_sparse_mla_fp4_workspace_bytes(0, 16, 100) == 0
    assert hs.hs_sparse_mla_fp4_workspace_bytes(4, 16, -1) == 0
    assert hs.hs_paged_mla_workspace_bytes(4, 0, 16, 100) == 0
    assert hs.hs_paged_mla_workspace_bytes(4, 1, 16, -1) == 0
    assert hs.hs_mla_prefill_workspace_bytes(1, 0, 100, 4) == 0
    assert hs.hs_mla_prefill_workspace_bytes(1, 10, -1, 4) == 0
    # a split's row: 512 halves and six floats
    for n, heads, k in ((1, 16, 4096), (32, 128, 2048), (3, 129, 70000)):
        assert hs.hs_sparse_mla_fp4_workspace_bytes(n, heads, k) % (n * heads * 1048) == 0
    # the expanded keys and values at least, whatever the requests
    assert hs.hs_mla_prefill_workspace_bytes(3, 100, 1000, 8) >= 1000 * 8 * 512
    # sizes beyond 32 bits
    assert hs.hs_mla_prefill_workspace_bytes(1, 4096, 1 << 17, 128) > 1 << 33


def test_bindings_refuse_wrong_tensors():
    t = torch.zeros
    i32, bf, f32, u8 = torch.int32, torch.bfloat16, torch.float32, torch.uint8
    lay = layout(row_bytes=400)
    sparse = lambda **kw: hs.hs_sparse_mla_decode_fp4(lay, **{**dict(
        kv_layer=t(64, 400, dtype=u8), row_ids=t(2, 8, dtype=i32), num_tokens=2, top_k=8,
        q=t(2, 4, 576, dtype=bf), num_heads=4, sm_scale=1.0, out=t(2, 4, 512, dtype=bf),
        lse=t(2, 4)), **kw})
    with pytest.raises(ValueError, match="row_ids"):
        sparse(row_ids=t(2, 7, dtype=i32))
    with pytest.raises(ValueError, match="q has"):
        sparse(q=t(2, 4, 512, dtype=bf))
    with pytest.raises(TypeError, match="kv_layer"):
        sparse(kv_layer=t(64, 400, dtype=i32))
    with pytest.raises(ValueError, match="current CUDA device"):
        sparse()
    with pytest.raises(TypeError, match="cannot pass"):
        sparse(kv_layer=[1])
    b = batch(ctx_len=FAKE)
    paged = lambda **kw: hs.hs_paged_mla_decode(lay, b, 0, **{**dict(
        q=FAKE, num_pos=1, num_heads=4, max_ctx=9, sm_scale=1.0, out=FAKE, lse=FAKE), **kw})
    with pytest.raises(ValueError, match="out has"):
        paged(out=t(2, 4, 576, dtype=bf))
    with pytest.raises(TypeError, match="lse"):
        paged(lse=t(2, 4, dtype=bf))
    with pytest.raises(ValueError, match="lse has"):
        paged(lse=t(3, 4))
    with pytest.raises(TypeError, match="out is"):
        paged(out=t(2, 4, 512, dtype=f32))
    prefill = lambda **kw: hs.hs_mla_prefill(lay, b, 0, **{**dict(
        q_start=FAKE, num_q=5, num_kv=9, q=FAKE, num_heads=4, w_kv=FAKE, sm_scale=1.0, out=FAKE,
        workspace=None), **kw})
    with pytest.raises(ValueError, match="q_start"):
        prefill(q_start=t(2, dtype=i32))
    with pytest.raises(TypeError, match="q_start"):
        prefill(q_start=t(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="w_kv"):
        prefill(w_kv=t(4, 256, 576, dtype=bf))
    with pytest.raises(ValueError, match="current CUDA device"):
        prefill(workspace=t(64, dtype=u8))
    with pytest.raises(hs.HsError):
        prefill(stream=0)


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), float("-inf")])
def test_scales_that_are_not_finite(lib, scale):
    r = ctypes.byref
    l8, l4, b = layout(), layout(row_bytes=400), batch(ctx_len=FAKE)
    assert lib.hs_sparse_mla_decode_fp4(r(l4), FAKE, FAKE, 1, 8, FAKE, 1, scale, FAKE, FAKE, FAKE,
                                        BIG, None) == 1
    assert lib.hs_paged_mla_decode(r(l8), r(b), 0, FAKE, 1, 1, 8, scale, FAKE, FAKE, FAKE, BIG,
                                   None) == 1
    assert lib.hs_mla_prefill(r(l8), r(b), 0, FAKE, 1, 8, FAKE, 1, FAKE, scale, FAKE, FAKE, BIG,
                              None) == 1
