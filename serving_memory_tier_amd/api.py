"""Thin wrappers with the C names: torch tensors in, raw pointers to the C ABI.

Every function checks the status the library returns and raises HsError on
anything but HS_OK.  Streams default to torch's current stream, so the calls
order with surrounding torch work exactly as the C calls would.
"""

from __future__ import annotations

import ctypes

import numpy as np
import torch

from ._lib import HS_OK, HsAppend, HsBatch, HsError, HsLayout, lib


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, torch.Tensor):
        if not t.is_contiguous():
            raise ValueError("tensors passed to the library must be contiguous")
        return t.data_ptr()
    raise TypeError(f"cannot pass {type(t)} as a pointer")


def _stream(stream) -> int:
    if stream is None:                   # torch.cuda.current_stream().cuda_stream, without its object
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int, what: str) -> None:
    if status != HS_OK:
        detail = lib().hs_last_error().decode() if status in (3, 4) else ""
        raise HsError(status, f"{what} failed ({hs_status_string(status)}"
                              f"{'; ' + detail if detail else ''})")


def hs_status_string(status: int) -> str:
    return lib().hs_status_string(status).decode()


def layout_of(page_size: int, row_bytes: int, num_layers: int, hot_capacity: int,
              pool_rows: int, host_rows: int, pool_layer_stride: int | None = None,
              host_layer_stride: int | None = None) -> HsLayout:
    return HsLayout(page_size, row_bytes, num_layers, hot_capacity, pool_rows, host_rows,
                    pool_layer_stride if pool_layer_stride is not None else pool_rows * row_bytes,
                    host_layer_stride if host_layer_stride is not None else host_rows * row_bytes)


def batch_of(num_reqs: int, max_pages: int, kv_pool, host_pool, block_table, host_block_table,
             ctx_len, hot_blocks, slot_token, slot_stamp, fill_sync=None,
             fill_sync_words: int | None = None) -> HsBatch:
    """kv_pool and the tables are CUDA tensors; host_pool is a HostPool, a
    device-visible address (int), or None when host_rows is 0; fill_sync is
    None or zeroed int32 device words (at least HS_FILL_SYNC_WORDS): a CUDA
    tensor, whose length is the word count unless fill_sync_words says
    otherwise, or an address with fill_sync_words."""
    hp = host_pool.device_ptr if isinstance(host_pool, HostPool) else _ptr(host_pool)
    if isinstance(fill_sync, torch.Tensor) and fill_sync.dtype != torch.int32:
        raise TypeError(f"fill_sync must be int32, not {fill_sync.dtype}")
    if fill_sync_words is None:
        fill_sync_words = fill_sync.numel() if isinstance(fill_sync, torch.Tensor) else 0
    return HsBatch(num_reqs, max_pages, _ptr(kv_pool), hp, _ptr(block_table),
                   _ptr(host_block_table), _ptr(ctx_len), _ptr(hot_blocks), _ptr(slot_token),
                   _ptr(slot_stamp), _ptr(fill_sync), fill_sync_words)


def hs_resolve(layout: HsLayout, batch: HsBatch, topk, top_k: int, stamp: int, row_ids,
               gather_out, stats, stream=None) -> None:
    _check(lib().hs_resolve(ctypes.byref(layout), ctypes.byref(batch), _ptr(topk), top_k,
                            ctypes.c_uint32(stamp), _ptr(row_ids), _ptr(gather_out), _ptr(stats),
                            _stream(stream)), "hs_resolve")


def hs_plan_replay(layout: HsLayout, batch: HsBatch, topk, num_pos: int, top_k: int, stamp: int,
                   row_ids, gather_out, stats, offload_pairs=None, n_offload: int = 0,
                   stream=None) -> None:
    _check(lib().hs_plan_replay(ctypes.byref(layout), ctypes.byref(batch), _ptr(topk), num_pos,
                                top_k, ctypes.c_uint32(stamp), _ptr(row_ids), _ptr(gather_out),
                                _ptr(stats), _ptr(offload_pairs), n_offload, _stream(stream)),
           "hs_plan_replay")


def hs_resolve_grouped(layout: HsLayout, batch: HsBatch, group_layers: int, topk, num_pos: int,
                       top_k: int, stamp: int, row_ids, gather_out, stats, offload_pairs=None,
                       n_offload: int = 0, stream=None) -> None:
    _check(lib().hs_resolve_grouped(ctypes.byref(layout), ctypes.byref(batch), group_layers,
                                    _ptr(topk), num_pos, top_k, ctypes.c_uint32(stamp),
                                    _ptr(row_ids), _ptr(gather_out), _ptr(stats),
                                    _ptr(offload_pairs), n_offload, _stream(stream)),
           "hs_resolve_grouped")


def hs_resolve_decide(layout: HsLayout, batch: HsBatch, topk, num_pos: int, top_k: int,
                      stamp: int, row_ids, gather_out, stats, stream=None) -> None:
    _check(lib().hs_resolve_decide(ctypes.byref(layout), ctypes.byref(batch), _ptr(topk), num_pos,
                                   top_k, ctypes.c_uint32(stamp), _ptr(row_ids), _ptr(gather_out),
                                   _ptr(stats), _stream(stream)), "hs_resolve_decide")


def hs_resolve_fetch(layout: HsLayout, batch: HsBatch, topk, num_pos: int, top_k: int,
                     gather_out, stream=None) -> None:
    _check(lib().hs_resolve_fetch(ctypes.byref(layout), ctypes.byref(batch), _ptr(topk), num_pos,
                                  top_k, _ptr(gather_out), _stream(stream)), "hs_resolve_fetch")


def hs_resolve_move(layout: HsLayout, batch: HsBatch, topk, num_pos: int, top_k: int, row_ids,
                    gather_out, stream=None) -> None:
    _check(lib().hs_resolve_move(ctypes.byref(layout), ctypes.byref(batch), _ptr(topk), num_pos,
                                 top_k, _ptr(row_ids), _ptr(gather_out), _stream(stream)),
           "hs_resolve_move")


def hs_resolve_commit(layout: HsLayout, batch: HsBatch, topk, num_pos: int, top_k: int, row_ids,
                      gather_out, stream=None) -> None:
    _check(lib().hs_resolve_commit(ctypes.byref(layout), ctypes.byref(batch), _ptr(topk),
                                   num_pos, top_k, _ptr(row_ids), _ptr(gather_out),
                                   _stream(stream)), "hs_resolve_commit")


def hs_gather(layout: HsLayout, kv_pool, row_ids, num_reqs: int, rows_per_req_layer: int, out,
              stream=None) -> None:
    _check(lib().hs_gather(ctypes.byref(layout), _ptr(kv_pool), _ptr(row_ids), num_reqs,
                           rows_per_req_layer, _ptr(out), _stream(stream)), "hs_gather")


def hs_offload_prefix_pages(layout: HsLayout, kv_pool, host_pool, pairs, n: int,
                            stream=None) -> None:
    hp = host_pool.device_ptr if isinstance(host_pool, HostPool) else _ptr(host_pool)
    _check(lib().hs_offload_prefix_pages(ctypes.byref(layout), _ptr(kv_pool), hp, _ptr(pairs), n,
                                         _stream(stream)), "hs_offload_prefix_pages")


def hs_page_touch(layout: HsLayout, batch: HsBatch, topk, entries_per_req: int, stamp: int,
                  page_use, stream=None) -> None:
    _check(lib().hs_page_touch(ctypes.byref(layout), ctypes.byref(batch), _ptr(topk),
                               entries_per_req, stamp, _ptr(page_use), _stream(stream)),
           "hs_page_touch")


def hs_resolve_in_place(layout: HsLayout, batch: HsBatch, topk, num_pos: int, top_k: int,
                        stamp: int, row_ids, staging, stats, offload_pairs=None, n_offload: int = 0,
                        stream=None) -> None:
    _check(lib().hs_resolve_in_place(ctypes.byref(layout), ctypes.byref(batch), _ptr(topk),
                                     num_pos, top_k, ctypes.c_uint32(stamp), _ptr(row_ids),
                                     _ptr(staging), _ptr(stats), _ptr(offload_pairs), n_offload,
                                     _stream(stream)), "hs_resolve_in_place")


def hs_sparse_mla_workspace_bytes(num_tokens: int, num_heads: int, top_k: int) -> int:
    return int(lib().hs_sparse_mla_workspace_bytes(num_tokens, num_heads, top_k))


def hs_sparse_mla_decode(layout: HsLayout, kv_layer, row_ids, num_tokens: int, top_k: int, q,
                         num_heads: int, sm_scale: float, out, lse, workspace=None,
                         workspace_bytes: int = 0, stream=None) -> None:
    """kv_layer: a uint8 device tensor (one layer of the pool) or a device
    address; workspace: a device tensor of hs_sparse_mla_workspace_bytes."""
    kv = kv_layer if isinstance(kv_layer, int) else _ptr(kv_layer)
    if workspace is not None and not workspace_bytes:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(lib().hs_sparse_mla_decode(ctypes.byref(layout), kv, _ptr(row_ids), num_tokens, top_k,
                                      _ptr(q), num_heads, sm_scale, _ptr(out), _ptr(lse),
                                      _ptr(workspace), workspace_bytes, _stream(stream)),
           "hs_sparse_mla_decode")


def hs_sparse_mla_decode_noalloc(layout: HsLayout, kv_layer, row_ids, num_tokens: int,
                                 top_k: int, q, num_heads: int, sm_scale: float, out, lse,
                                 stream=None) -> None:
    """hs_sparse_mla_decode with the library's per-device workspace."""
    kv = kv_layer if isinstance(kv_layer, int) else _ptr(kv_layer)
    _check(lib().hs_sparse_mla_decode_noalloc(ctypes.byref(layout), kv, _ptr(row_ids), num_tokens,
                                              top_k, _ptr(q), num_heads, sm_scale, _ptr(out),
                                              _ptr(lse), _stream(stream)),
           "hs_sparse_mla_decode_noalloc")


def hs_sparse_mla_noalloc_max_workspace() -> int:
    return int(lib().hs_sparse_mla_noalloc_max_workspace())


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)


def _operand(t, what: str, dtypes, device: int | None = None, contiguous: bool = True):
    """The address of an operand of the latent-cache calls: a CUDA tensor of one
    of ``dtypes`` on the current device (``device``, for who asked already), an
    address (int), or None."""
    if t is None or isinstance(t, int):
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"cannot pass {type(t)} as {what}")
    if t.dtype not in dtypes:
        raise TypeError(f"{what} is {t.dtype}, not {dtypes[0]}")
    at = t.get_device()                  # -1: not a CUDA tensor
    if at < 0 or at != (torch.cuda.current_device() if device is None else device):
        raise ValueError(f"{what} is on {t.device}, not on the current CUDA device")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _device(t) -> int | None:
    """The current device, asked for once a call; None where ``t`` tells already
    that the call will be refused, or is no tensor."""
    return torch.cuda.current_device() if isinstance(t, torch.Tensor) and t.is_cuda else None


def _shaped(t, what: str, shape: tuple) -> None:
    if isinstance(t, torch.Tensor) and t.shape != shape:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, not {shape}")


def _sized(t, what: str, n: int) -> None:
    if isinstance(t, torch.Tensor) and t.numel() != n:
        raise ValueError(f"{what} has {t.numel()} values, not {n}")


def append_of(num_tokens: int, token_req, positions, latent, rope, rope_freq,
              rope_interleaved: bool, q_rope=None, q_out=None) -> HsAppend:
    """The tokens of one hs_mla_append call.  token_req, positions: int32 [T];
    latent bf16 [T, 512]; rope bf16 [T, 64]; rope_freq float64 [32]; q_rope and
    q_out (both or neither): bf16 [T, H, 64].  latent, rope, q_rope and q_out
    may be strided views with their last dimension contiguous.  The struct keeps
    the tensors alive."""
    if (q_rope is None) != (q_out is None):
        raise ValueError("q_rope and q_out go together")
    T = num_tokens
    _shaped(token_req, "token_req", (T,))
    _shaped(positions, "positions", (T,))
    _shaped(latent, "latent", (T, 512))
    _shaped(rope, "rope", (T, 64))
    _shaped(rope_freq, "rope_freq", (32,))
    here, i32 = _device(latent), (torch.int32,)
    strides = [latent.stride(), rope.stride()]
    heads = 0
    if q_rope is not None:
        heads = q_rope.shape[1]
        _shaped(q_rope, "q_rope", (T, heads, 64))
        _shaped(q_out, "q_out", (T, heads, 64))
        strides += [q_rope.stride(), q_out.stride()]
    for s, what in zip(strides, ("latent", "rope", "q_rope", "q_out")):
        if s[-1] != 1:
            raise ValueError(f"{what}'s last dimension must be contiguous")
    q, o = strides[2:] if heads else ((0, 0), (0, 0))
    a = HsAppend(T, heads, _operand(token_req, "token_req", i32, here),
                 _operand(positions, "positions", i32, here),
                 _operand(latent, "latent", _BF16, here, False), strides[0][0],
                 _operand(rope, "rope", _BF16, here, False), strides[1][0],
                 _operand(rope_freq, "rope_freq", (torch.float64,), here),
                 _operand(q_rope, "q_rope", _BF16, here, False), q[0], q[1],
                 _operand(q_out, "q_out", _BF16, here, False), o[0], o[1],
                 1 if rope_interleaved else 0, 0)
    a.tensors = (token_req, positions, latent, rope, rope_freq, q_rope, q_out)
    return a


def hs_mla_append(layout: HsLayout, batch: HsBatch, layer: int, tokens: HsAppend, row_ids=None,
                  values=None, stream=None) -> None:
    """tokens: append_of(...); row_ids int32 [T] or None; values bf16 [T, 576] or
    None."""
    _shaped(row_ids, "row_ids", (tokens.num_tokens,))
    _shaped(values, "values", (tokens.num_tokens, 576))
    _check(lib().hs_mla_append(ctypes.byref(layout), ctypes.byref(batch), layer,
                               ctypes.byref(tokens), _operand(row_ids, "row_ids", (torch.int32,)),
                               _operand(values, "values", _BF16), _stream(stream)),
           "hs_mla_append")


def _workspace(ws) -> tuple:
    """Address and bytes of a workspace: a contiguous CUDA tensor or None."""
    if ws is None:
        return None, 0
    return _operand(ws, "workspace", (ws.dtype,)), ws.numel() * ws.element_size()


def hs_sparse_mla_fp4_workspace_bytes(num_tokens: int, num_heads: int, top_k: int) -> int:
    return int(lib().hs_sparse_mla_fp4_workspace_bytes(num_tokens, num_heads, top_k))


def hs_sparse_mla_decode_fp4(layout: HsLayout, kv_layer, row_ids, num_tokens: int, top_k: int, q,
                             num_heads: int, sm_scale: float, out, lse, workspace=None,
                             stream=None) -> None:
    """kv_layer: a uint8 tensor (one layer of the pool) or a device address; q bf16
    [T, H, 576]; out bf16 [T, H, 512]; lse float32 [T, H]; workspace: a tensor of
    hs_sparse_mla_fp4_workspace_bytes."""
    _sized(row_ids, "row_ids", num_tokens * top_k)
    _sized(q, "q", num_tokens * num_heads * 576)
    _sized(out, "out", num_tokens * num_heads * 512)
    _sized(lse, "lse", num_tokens * num_heads)
    ws, ws_bytes = _workspace(workspace)
    _check(lib().hs_sparse_mla_decode_fp4(
        ctypes.byref(layout), _operand(kv_layer, "kv_layer", (torch.uint8,)),
        _operand(row_ids, "row_ids", (torch.int32,)), num_tokens, top_k, _operand(q, "q", _BF16),
        num_heads, sm_scale, _operand(out, "out", _BF16), _operand(lse, "lse", (torch.float32,)),
        ws, ws_bytes, _stream(stream)), "hs_sparse_mla_decode_fp4")


def hs_paged_mla_workspace_bytes(num_reqs: int, num_pos: int, num_heads: int, max_ctx: int) -> int:
    return int(lib().hs_paged_mla_workspace_bytes(num_reqs, num_pos, num_heads, max_ctx))


def hs_paged_mla_decode(layout: HsLayout, batch: HsBatch, layer: int, q, num_pos: int,
                        num_heads: int, max_ctx: int, sm_scale: float, out, lse, workspace=None,
                        stream=None) -> None:
    """q bf16 [R, P, H, 576]; out bf16 [R, P, H, 512]; lse float32 [R, P, H];
    workspace: a tensor of hs_paged_mla_workspace_bytes."""
    rows = batch.num_reqs * num_pos * num_heads
    _sized(q, "q", rows * 576)
    _sized(out, "out", rows * 512)
    _sized(lse, "lse", rows)
    ws, ws_bytes = _workspace(workspace)
    _check(lib().hs_paged_mla_decode(
        ctypes.byref(layout), ctypes.byref(batch), layer, _operand(q, "q", _BF16), num_pos,
        num_heads, max_ctx, sm_scale, _operand(out, "out", _BF16),
        _operand(lse, "lse", (torch.float32,)), ws, ws_bytes, _stream(stream)),
        "hs_paged_mla_decode")


def hs_mla_prefill_workspace_bytes(num_reqs: int, num_q: int, num_kv: int, num_heads: int) -> int:
    return int(lib().hs_mla_prefill_workspace_bytes(num_reqs, num_q, num_kv, num_heads))


def hs_mla_prefill(layout: HsLayout, batch: HsBatch, layer: int, q_start, num_q: int, num_kv: int,
                   q, num_heads: int, w_kv, sm_scale: float, out, workspace, stream=None) -> None:
    """q_start int32 [R + 1]; q bf16 [num_q, H, 192]; w_kv bf16 [H, 256, 512]; out bf16
    [num_q, H, 128]; workspace: a tensor of hs_mla_prefill_workspace_bytes."""
    _sized(q_start, "q_start", batch.num_reqs + 1)
    _sized(q, "q", num_q * num_heads * 192)
    _sized(w_kv, "w_kv", num_heads * 256 * 512)
    _sized(out, "out", num_q * num_heads * 128)
    ws, ws_bytes = _workspace(workspace)
    _check(lib().hs_mla_prefill(
        ctypes.byref(layout), ctypes.byref(batch), layer,
        _operand(q_start, "q_start", (torch.int32,)), num_q, num_kv, _operand(q, "q", _BF16),
        num_heads, _operand(w_kv, "w_kv", _BF16), sm_scale, _operand(out, "out", _BF16), ws,
        ws_bytes, _stream(stream)), "hs_mla_prefill")


def hs_host_alloc(nbytes: int) -> int:
    p = ctypes.c_void_p()
    _check(lib().hs_host_alloc(nbytes, ctypes.byref(p)), "hs_host_alloc")
    return p.value


def hs_host_free(ptr: int) -> None:
    _check(lib().hs_host_free(ptr), "hs_host_free")


def hs_host_device_pointer(ptr: int) -> int:
    d = ctypes.c_void_p()
    _check(lib().hs_host_device_pointer(ptr, ctypes.byref(d)), "hs_host_device_pointer")
    return d.value


class HostPool:
    """Pinned, device-mapped host memory holding the host pool.

    ``array`` is a numpy uint8 view of the whole allocation (host side);
    ``tensor`` the same memory as a CPU torch tensor; ``device_ptr`` the
    address kernels read and write.
    """

    def __init__(self, nbytes: int):
        self.nbytes = int(nbytes)
        self.host_ptr = hs_host_alloc(self.nbytes)
        self.device_ptr = hs_host_device_pointer(self.host_ptr)
        buf = (ctypes.c_uint8 * self.nbytes).from_address(self.host_ptr)
        self.array = np.frombuffer(buf, dtype=np.uint8)
        self.tensor = torch.from_numpy(self.array)

    def close(self) -> None:
        if self.host_ptr:
            self.tensor = None
            self.array = None
            hs_host_free(self.host_ptr)
            self.host_ptr = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
