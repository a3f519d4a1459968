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
