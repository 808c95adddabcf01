"""Python binding of the INT4-weight / Hadamard-rotated INT4-KV decode-block
library (``libft.so``, C ABI declared in ``include/ft.h``).

Argument marshalling only: every function here forwards to the C entry point of
the same name; all computation runs in the library's CUDA kernels.  PyTorch is
used for device memory and streams.  If the compiled library is missing the
calls raise instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import c_int, c_int32, c_int64, c_size_t, c_uint, c_void_p, c_float, c_char_p, POINTER

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libft.so")

FT_OK, FT_ERR_INVALID_ARG, FT_ERR_UNSUPPORTED, FT_ERR_WORKSPACE, FT_ERR_CAPACITY, FT_ERR_CUDA = 0, -1, -2, -3, -4, -5
FT_DEV_CAPACITY, FT_DEV_TIMEOUT, FT_DEV_RANGE = 1, 2, 4
FT_BF16, FT_F32 = 0, 1
FT_WFMT_INT4, FT_WFMT_E4M3 = 0, 1
FT_W_QKV, FT_W_O, FT_W_GATEUP, FT_W_DOWN = 0, 1, 2, 3
FT_STAGE_PREP, FT_STAGE_QKV, FT_STAGE_ATTN, FT_STAGE_O = 1, 2, 4, 8
FT_STAGE_MID, FT_STAGE_GU, FT_STAGE_DOWN, FT_STAGE_ALL = 16, 32, 64, 127
ROLES = (FT_W_QKV, FT_W_O, FT_W_GATEUP, FT_W_DOWN)


class BlockCfg(ctypes.Structure):
    _fields_ = [("hidden", c_int32), ("n_q", c_int32), ("n_kv", c_int32), ("head_dim", c_int32),
                ("inter", c_int32), ("w_group", c_int32), ("had_block", c_int32), ("kv_group", c_int32),
                ("rms_eps", c_float), ("rope_base", c_float), ("weight_format", c_int32)]


class LayerWeights(ctypes.Structure):
    _fields_ = [("qkv", c_void_p), ("o", c_void_p), ("gateup", c_void_p), ("down", c_void_p)]


class GemvInfo(ctypes.Structure):
    _fields_ = [(n, c_int32) for n in ("ctas", "row_tiles", "warps", "col_tiles", "whole", "tensor_core", "stages",
                                       "groups_per_stage", "smem_bytes")]


class WsLayout(ctypes.Structure):
    _fields_ = [("qkv", c_size_t), ("rho1", c_size_t), ("o", c_size_t), ("h1", c_size_t), ("a", c_size_t),
                ("n_split", c_int32)]


class FTError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {ft_status_string(status)} ({status})")


_lib = None

# name -> (restype, argtypes)
_SIGS = {
    "ft_status_string": (c_char_p, [c_int]),
    "ft_validate_cfg": (c_int, [POINTER(BlockCfg)]),
    "ft_weight_shape": (c_int, [POINTER(BlockCfg), c_int, POINTER(c_int32), POINTER(c_int32)]),
    "ft_packed_weight_bytes": (c_size_t, [POINTER(BlockCfg), c_int]),
    "ft_pack_weights_int4": (c_int, [POINTER(BlockCfg), c_int, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "ft_unpack_weights_int4": (c_int, [POINTER(BlockCfg), c_int, c_void_p, c_void_p, c_void_p, c_void_p]),
    "ft_pack_weights_e4m3": (c_int, [POINTER(BlockCfg), c_int, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "ft_unpack_weights_e4m3": (c_int, [POINTER(BlockCfg), c_int, c_void_p, c_void_p, c_void_p, c_void_p]),
    "ft_kv_cache_bytes": (c_size_t, [POINTER(BlockCfg), c_int, c_int]),
    "ft_kv_append_int4": (c_int, [POINTER(BlockCfg), c_void_p, c_int, c_int, c_void_p, c_void_p, c_void_p,
                                  c_int, c_int, c_void_p, c_void_p]),
    "ft_kv_append_ragged_int4": (c_int, [POINTER(BlockCfg), c_void_p, c_int, c_int, c_void_p, c_void_p, c_void_p,
                                         c_void_p, c_int, c_int, c_void_p, c_void_p]),
    "ft_kv_unpack_int4": (c_int, [POINTER(BlockCfg), c_void_p, c_int, c_int, c_int, c_int, c_void_p, c_void_p,
                                  c_void_p, c_void_p, c_void_p]),
    "ft_kv_pages_bytes": (c_size_t, [POINTER(BlockCfg), c_int, c_int]),
    "ft_kv_page_map": (c_int, [c_int, c_int, c_void_p, c_void_p, c_int, c_void_p, c_int, c_void_p, c_int, c_void_p,
                               c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_void_p, c_void_p]),
    "ft_kv_append_paged_int4": (c_int, [POINTER(BlockCfg), c_void_p, c_int, c_int, c_void_p, c_int64, c_void_p,
                                        c_int64, c_void_p, c_int, c_void_p, c_void_p]),
    "ft_kv_read_paged_int4": (c_int, [POINTER(BlockCfg), c_void_p, c_int, c_int, c_void_p, c_int, c_void_p, c_void_p,
                                      c_void_p, c_void_p]),
    "ft_attn_paged_workspace_bytes": (c_size_t, [POINTER(BlockCfg), c_int, c_int, c_int]),
    "ft_attn_paged_int4": (c_int, [POINTER(BlockCfg), c_void_p, c_int, c_int, c_void_p, c_int64, c_void_p, c_void_p,
                                   c_void_p, c_int, c_int, c_int, c_int, c_float, c_void_p, c_int64, c_void_p,
                                   c_size_t, c_void_p, c_void_p]),
    "ft_decode_workspace_bytes": (c_size_t, [POINTER(BlockCfg), c_int, c_int]),
    "ft_decode_block": (c_int, [POINTER(BlockCfg), POINTER(LayerWeights), c_void_p, c_int, c_int, c_void_p,
                                c_void_p, c_int, c_void_p, c_int, c_void_p, c_size_t, c_void_p, c_void_p]),
    "ft_decode_block_stages": (c_int, [POINTER(BlockCfg), POINTER(LayerWeights), c_void_p, c_int, c_int, c_void_p,
                                       c_void_p, c_int, c_void_p, c_int, c_void_p, c_size_t, c_void_p, c_uint,
                                       c_void_p]),
    "ft_decode_workspace_layout": (c_int, [POINTER(BlockCfg), c_int, c_int, POINTER(WsLayout)]),
    "ft_decode_block_static_ws": (c_int, [POINTER(BlockCfg), POINTER(LayerWeights), c_void_p, c_int, c_int,
                                          c_void_p, c_void_p, c_int, c_void_p, c_int, c_void_p, c_void_p]),
    "ft_embed_bf16": (c_int, [c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_void_p, c_void_p]),
    "ft_lm_head_bf16": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_float, c_void_p]),
    "ft_rmsnorm_bf16": (c_int, [c_void_p, c_void_p, c_void_p, c_int, c_int, c_float, c_void_p]),
    "ft_logprobs": (c_int, [c_void_p, c_int, c_int64, c_int, c_int, c_void_p, c_int, c_void_p, c_void_p, c_void_p,
                            c_void_p, c_void_p, c_void_p, c_void_p]),
    "ft_read_device_status": (c_int, [c_void_p, c_void_p, c_void_p]),
    "ft_decode_plan_info": (c_int, [c_void_p, c_int, c_int, c_int, c_void_p]),
    "ft_decode_block_launches": (c_int, [POINTER(BlockCfg), c_int]),
    "ft_set_pdl": (c_int, [c_int]),
}


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run int4_weight_kv_gb300.build.build() first")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def exported_symbols() -> list[str]:
    return list(_SIGS)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _current():
    """(current CUDA device, its current stream's handle).  The stream object that
    torch.cuda.current_stream() builds costs 3 us a call, its handle alone 0.1."""
    if _torch is None:
        _bind_torch()
    dev = _torch[0]()
    return dev, _torch[1](dev)


# (current device, its current stream's handle, then the types that pass as INT32, FP32, BF16 or its bits, bytes),
# once torch is there
_torch = None
_I32, _F32, _B16, _U8, _ANY = 2, 3, 4, 5, None
_KINDS = {_I32: "int32", _F32: "float32", _B16: "bfloat16 (or int16, uint16: its bits)", _U8: "uint8", _ANY: "any type"}


def _bind_torch():
    global _torch
    import torch
    torch.cuda.init()
    _torch = (getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
              getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream),
              (torch.int32,), (torch.float32,), (torch.bfloat16, torch.int16, torch.uint16), (torch.uint8, torch.int8))


def _stream(stream):
    if stream is None:
        return _current()[1]
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _on(t, dev: int) -> None:
    if t.get_device() != dev:
        raise ValueError(f"tensor on {t.device}, the current device is cuda:{dev}")


def _plain(t, kind: int, dev: int):
    """Pointer of a contiguous tensor of that kind on device `dev` (or None, or a raw pointer)."""
    if t is None or isinstance(t, int):
        return t
    if t.get_device() != dev or not t.is_contiguous() or (kind and t.dtype not in _torch[kind]):
        _on(t, dev)
        raise ValueError(f"need a contiguous tensor of {_KINDS[kind]}, got {t.dtype} with strides {t.stride()}")
    return t.data_ptr()


def _rows(t, inner: int, kind: int, dev: int) -> tuple[int, int]:
    """(pointer, elements between rows) of a tensor on device `dev` whose rows are `inner` contiguous elements of that
    kind."""
    shape = t.shape
    if t.get_device() != dev:
        _on(t, dev)
    good = t.dtype in _torch[kind] and len(shape) >= 2
    if good and t.is_contiguous() and t.numel() == shape[0] * inner:
        return t.data_ptr(), inner
    step = t.stride()
    want = 1
    for i in range(len(shape) - 1, 0, -1):
        good = good and (step[i] == want or shape[i] == 1)
        want *= shape[i]
    if not good or want != inner:
        raise ValueError(f"need rows of {inner} contiguous elements of {_KINDS[kind]}, got {t.dtype} {tuple(shape)} "
                         f"with strides {step}")
    return t.data_ptr(), step[0] if shape[0] > 1 else max(step[0], inner)


def make_cfg(hidden, n_q, n_kv, head_dim, inter, had_block=0, kv_group=0, rms_eps=1e-5, rope_base=500000.0,
             w_group=128, weight_format=0) -> BlockCfg:
    hb = had_block or head_dim
    return BlockCfg(hidden, n_q, n_kv, head_dim, inter, w_group, hb, kv_group or head_dim, rms_eps, rope_base,
                    weight_format)


def cfg_from_shape(shape) -> BlockCfg:
    """BlockCfg from any object with the BlockShape attribute names."""
    return make_cfg(shape.hidden, shape.n_q, shape.n_kv, shape.head_dim, shape.inter,
                    getattr(shape, "had_block", 0), getattr(shape, "kv_group", 0),
                    shape.rms_eps, shape.rope_base, weight_format=getattr(shape, "weight_format", 0))


def check(status: int, what: str = "ft") -> None:
    if status != FT_OK:
        raise FTError(status, what)


# ---------------------------------------------------------------- the C ABI, same names
def ft_status_string(status: int) -> str:
    return lib().ft_status_string(status).decode()


def ft_validate_cfg(cfg: BlockCfg) -> int:
    return lib().ft_validate_cfg(ctypes.byref(cfg))


def ft_weight_shape(cfg: BlockCfg, role: int) -> tuple[int, int]:
    n, k = c_int32(), c_int32()
    check(lib().ft_weight_shape(ctypes.byref(cfg), role, ctypes.byref(n), ctypes.byref(k)), "ft_weight_shape")
    return n.value, k.value


def ft_packed_weight_bytes(cfg: BlockCfg, role: int) -> int:
    return lib().ft_packed_weight_bytes(ctypes.byref(cfg), role)


def ft_pack_weights_int4(cfg, role, W, gamma, packed, stream=None) -> int:
    return lib().ft_pack_weights_int4(ctypes.byref(cfg), role, _ptr(W), _ptr(gamma), _ptr(packed),
                                      packed.numel() * packed.element_size(), _stream(stream))


def ft_unpack_weights_int4(cfg, role, packed, codes, scales, stream=None) -> int:
    return lib().ft_unpack_weights_int4(ctypes.byref(cfg), role, _ptr(packed), _ptr(codes), _ptr(scales),
                                        _stream(stream))


def ft_pack_weights_e4m3(cfg, role, W, gamma, packed, stream=None) -> int:
    return lib().ft_pack_weights_e4m3(ctypes.byref(cfg), role, _ptr(W), _ptr(gamma), _ptr(packed),
                                      packed.numel() * packed.element_size(), _stream(stream))


def ft_unpack_weights_e4m3(cfg, role, packed, codes, scales, stream=None) -> int:
    return lib().ft_unpack_weights_e4m3(ctypes.byref(cfg), role, _ptr(packed), _ptr(codes), _ptr(scales),
                                        _stream(stream))


def ft_kv_cache_bytes(cfg, max_batch: int, max_ctx: int) -> int:
    return lib().ft_kv_cache_bytes(ctypes.byref(cfg), max_batch, max_ctx)


def ft_kv_append_int4(cfg, cache, max_batch, max_ctx, k_bits, v_bits, pos, B, T, dev_status=None,
                      stream=None) -> int:
    return lib().ft_kv_append_int4(ctypes.byref(cfg), _ptr(cache), max_batch, max_ctx, _ptr(k_bits), _ptr(v_bits),
                                   _ptr(pos), B, T, _ptr(dev_status), _stream(stream))


def ft_kv_append_ragged_int4(cfg, cache, max_batch, max_ctx, k_bits, v_bits, cu_seqlens, pos, B, total,
                             dev_status=None, stream=None) -> int:
    return lib().ft_kv_append_ragged_int4(ctypes.byref(cfg), _ptr(cache), max_batch, max_ctx, _ptr(k_bits),
                                          _ptr(v_bits), _ptr(cu_seqlens), _ptr(pos), B, total, _ptr(dev_status),
                                          _stream(stream))


def ft_kv_unpack_int4(cfg, cache, max_batch, max_ctx, B, length, k_codes, v_codes, k_scales, v_scales,
                      stream=None) -> int:
    return lib().ft_kv_unpack_int4(ctypes.byref(cfg), _ptr(cache), max_batch, max_ctx, B, length, _ptr(k_codes),
                                   _ptr(v_codes), _ptr(k_scales), _ptr(v_scales), _stream(stream))


def ft_kv_pages_bytes(cfg, n_pages: int, page_size: int) -> int:
    return lib().ft_kv_pages_bytes(ctypes.byref(cfg), n_pages, page_size)


def ft_kv_page_map(page_size, n_pages, ctx_len, new_len, B, block_table, free_pages, free_head, free_head_out,
                   cu_seqlens, kv_len, slots, dev_status=None, stream=None) -> int:
    """block_table: int32 [B, >= pages of a request]; the other tensors int32, one-dimensional."""
    dev, here = _current()
    if min(ctx_len.numel(), new_len.numel(), kv_len.numel(), cu_seqlens.numel() - 1, block_table.shape[0]) < B:
        raise ValueError(f"lengths, prefix sums or block tables of fewer than {B} requests")
    table, stride = _rows(block_table, block_table.shape[1], _I32, dev)
    return lib().ft_kv_page_map(page_size, n_pages, _plain(ctx_len, _I32, dev), _plain(new_len, _I32, dev), B, table,
                                stride, _plain(free_pages, _I32, dev), free_pages.numel(),
                                _plain(free_head, _I32, dev), _plain(free_head_out, _I32, dev),
                                _plain(cu_seqlens, _I32, dev), _plain(kv_len, _I32, dev), _plain(slots, _I32, dev),
                                slots.numel(), _plain(dev_status, _I32, dev),
                                here if stream is None else _stream(stream))


def _check_pool(cfg, pages, n_pages, page_size) -> None:
    if not isinstance(pages, int) and pages.numel() < n_pages * cfg.n_kv * page_size * (cfg.head_dim + 4):
        raise ValueError(f"a pool of {pages.numel()} bytes does not hold {n_pages} pages")


def ft_kv_append_paged_int4(cfg, pages, n_pages, page_size, k, v, slots, total, dev_status=None, stream=None) -> int:
    """k, v: BF16 [>= total, n_kv, d], rows at any stride; slots: int32 [>= total]."""
    dev, here = _current()
    _check_pool(cfg, pages, n_pages, page_size)
    if min(k.shape[0], v.shape[0], slots.numel()) < total:
        raise ValueError(f"fewer than {total} rows or slots")
    row = cfg.n_kv * cfg.head_dim
    kp, ks = _rows(k, row, _B16, dev)
    vp, vs = _rows(v, row, _B16, dev)
    return lib().ft_kv_append_paged_int4(ctypes.byref(cfg), _plain(pages, _U8, dev), n_pages, page_size, kp, ks, vp, vs,
                                         _plain(slots, _I32, dev), total, _plain(dev_status, _I32, dev),
                                         here if stream is None else _stream(stream))


def ft_kv_read_paged_int4(cfg, pages, n_pages, page_size, slots, total, k_out, v_out, dev_status=None,
                          stream=None) -> int:
    """k_out, v_out: BF16 [>= total, n_kv, d], contiguous; slots: int32 [>= total]."""
    dev, here = _current()
    _check_pool(cfg, pages, n_pages, page_size)
    if min(k_out.numel(), v_out.numel()) < total * cfg.n_kv * cfg.head_dim or slots.numel() < total:
        raise ValueError(f"fewer than {total} rows or slots")
    return lib().ft_kv_read_paged_int4(ctypes.byref(cfg), _plain(pages, _U8, dev), n_pages, page_size,
                                       _plain(slots, _I32, dev), total, _plain(k_out, _B16, dev),
                                       _plain(v_out, _B16, dev), _plain(dev_status, _I32, dev),
                                       here if stream is None else _stream(stream))


def ft_attn_paged_workspace_bytes(cfg, B: int, total_q: int, max_q: int) -> int:
    return lib().ft_attn_paged_workspace_bytes(ctypes.byref(cfg), B, total_q, max_q)


def ft_attn_paged_int4(cfg, pages, n_pages, page_size, q, cu_seqlens, kv_len, block_table, B, total_q, max_q, scale, o,
                       workspace, dev_status=None, stream=None) -> int:
    """q, o: BF16 [>= total_q, n_q, d], rows at any stride; block_table: int32 [>= B, pages of a request]."""
    dev, here = _current()
    _check_pool(cfg, pages, n_pages, page_size)
    if min(q.shape[0], o.shape[0]) < total_q or min(cu_seqlens.numel() - 1, kv_len.numel(), block_table.shape[0]) < B:
        raise ValueError(f"fewer than {total_q} rows or {B} requests")
    row = cfg.n_q * cfg.head_dim
    qp, qs = _rows(q, row, _B16, dev)
    op, os_ = _rows(o, row, _B16, dev)
    table, stride = _rows(block_table, block_table.shape[1], _I32, dev)
    return lib().ft_attn_paged_int4(ctypes.byref(cfg), _plain(pages, _U8, dev), n_pages, page_size, qp, qs,
                                    _plain(cu_seqlens, _I32, dev), _plain(kv_len, _I32, dev), table, stride, B, total_q,
                                    max_q, scale, op, os_, _plain(workspace, _ANY, dev),
                                    workspace.numel() * workspace.element_size(),
                                    _plain(dev_status, _I32, dev), here if stream is None else _stream(stream))


def ft_decode_workspace_bytes(cfg, B: int, max_ctx: int) -> int:
    return lib().ft_decode_workspace_bytes(ctypes.byref(cfg), B, max_ctx)


def ft_decode_workspace_layout(cfg, B: int, max_ctx: int) -> WsLayout:
    out = WsLayout()
    check(lib().ft_decode_workspace_layout(ctypes.byref(cfg), B, max_ctx, ctypes.byref(out)),
          "ft_decode_workspace_layout")
    return out


def _layer(w) -> LayerWeights:
    if isinstance(w, LayerWeights):
        return w
    return LayerWeights(_ptr(w["qkv"]), _ptr(w["o"]), _ptr(w["gateup"]), _ptr(w["down"]))


def ft_decode_block(cfg, weights, cache, max_batch, max_ctx, x_in, x_out, act_dtype, pos, B, workspace,
                    dev_status=None, stream=None) -> int:
    lw = _layer(weights)
    return lib().ft_decode_block(ctypes.byref(cfg), ctypes.byref(lw), _ptr(cache), max_batch, max_ctx, _ptr(x_in),
                                 _ptr(x_out), act_dtype, _ptr(pos), B, _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _ptr(dev_status), _stream(stream))


def ft_decode_block_stages(cfg, weights, cache, max_batch, max_ctx, x_in, x_out, act_dtype, pos, B, workspace,
                           stage_mask, dev_status=None, stream=None) -> int:
    lw = _layer(weights)
    return lib().ft_decode_block_stages(ctypes.byref(cfg), ctypes.byref(lw), _ptr(cache), max_batch, max_ctx,
                                        _ptr(x_in), _ptr(x_out), act_dtype, _ptr(pos), B, _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _ptr(dev_status),
                                        stage_mask, _stream(stream))


def ft_decode_block_static_ws(cfg, weights, cache, max_batch, max_ctx, x_in, x_out, act_dtype, pos, B,
                              dev_status=None, stream=None) -> int:
    """ft_decode_block with the library's fixed device scratch instead of a workspace."""
    lw = _layer(weights)
    return lib().ft_decode_block_static_ws(ctypes.byref(cfg), ctypes.byref(lw), _ptr(cache), max_batch, max_ctx,
                                           _ptr(x_in), _ptr(x_out), act_dtype, _ptr(pos), B, _ptr(dev_status),
                                           _stream(stream))


def ft_embed_bf16(table, tokens, x_out, B, V, H, dev_status=None, stream=None) -> int:
    return lib().ft_embed_bf16(_ptr(table), _ptr(tokens), _ptr(x_out), B, V, H, _ptr(dev_status), _stream(stream))


def ft_lm_head_bf16(x, gamma, W, logits, B, V, H, eps, stream=None) -> int:
    return lib().ft_lm_head_bf16(_ptr(x), _ptr(gamma), _ptr(W), _ptr(logits), B, V, H, eps, _stream(stream))


def ft_rmsnorm_bf16(x, gamma, z, B, H, eps, stream=None) -> int:
    return lib().ft_rmsnorm_bf16(_ptr(x), _ptr(gamma), _ptr(z), B, H, eps, _stream(stream))


def ft_logprobs(logits, targets, logprob, entropy, rank, top_ids, top_logprobs, top_k, dev_status=None,
                stream=None) -> int:
    """logits: FP32 or BF16 [N, V], rows at any stride; targets: int32 [N] or None; outputs may be None."""
    dev, here = _current()
    n, v = logits.shape
    dtype = FT_F32 if logits.element_size() == 4 else FT_BF16
    x, stride = _rows(logits, v, _F32 if dtype == FT_F32 else _B16, dev)
    for t, size in ((targets, n), (logprob, n), (entropy, n), (rank, n), (top_ids, n * top_k), (top_logprobs, n * top_k)):
        if t is not None and t.numel() < size:
            raise ValueError(f"an argument holds {t.numel()} of {size} elements")
    return lib().ft_logprobs(x, dtype, stride, n, v, _plain(targets, _I32, dev), top_k, _plain(logprob, _F32, dev),
                             _plain(entropy, _F32, dev), _plain(rank, _I32, dev), _plain(top_ids, _I32, dev),
                             _plain(top_logprobs, _F32, dev), _plain(dev_status, _I32, dev),
                             here if stream is None else _stream(stream))


def ft_read_device_status(dev_status, stream=None) -> int:
    """Waits for `stream` and returns the device status word (raises on a CUDA error)."""
    out = ctypes.c_int32(0)
    check(lib().ft_read_device_status(_ptr(dev_status), ctypes.byref(out), _stream(stream)), "ft_read_device_status")
    return int(out.value)


def ft_decode_plan_info(cfg, B: int, max_ctx: int, role: int) -> GemvInfo:
    out = GemvInfo()
    check(lib().ft_decode_plan_info(ctypes.byref(cfg), int(B), int(max_ctx), int(role), ctypes.byref(out)),
          "ft_decode_plan_info")
    return out


def ft_decode_block_launches(cfg, B: int = 1) -> int:
    return lib().ft_decode_block_launches(ctypes.byref(cfg), int(B))


def ft_set_pdl(enabled: bool) -> bool:
    return bool(lib().ft_set_pdl(1 if enabled else 0))
