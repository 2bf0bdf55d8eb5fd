"""ctypes binding of libcconv.so (declared in include/cconv.h).

Argument marshalling only: each function takes torch CUDA tensors, checks
their dtypes and shapes, and passes raw device pointers, element strides and
the current CUDA stream to the C entry point of the same name. Every step of
the computation runs in the library's kernels; there is no other path. A
missing library raises instead of falling back to anything.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcconv.so")

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_LAUNCH, ERR_TOO_LARGE = 0, -1, -2, -3, -4
DTYPE_F32, DTYPE_BF16 = 0, 1
ACT_NONE, ACT_SILU = 0, 1
DERR_SLOT_RANGE, DERR_CU_SEQLENS, DERR_NUM_ACCEPTED, DERR_TIMEOUT = 1, 2, 4, 8
DERR_ROW_INDEX, DERR_CHECKPOINT = 16, 32
DERR_POSITION, DERR_PAGE, DERR_SEQ_LEN, DERR_GROUP = 64, 128, 256, 512

# of a cache in 8 bits (None on a PyTorch without them)
_F8, _F8_SCALE = (getattr(torch, t, None) for t in ("float8_e4m3fn", "float8_e8m0fnu"))

_lock = threading.Lock()
_lib = None
_fast = None    # csrc/fast.c: the mixer calls' marshalling in C, set by load()


class Epilogue(ctypes.Structure):
    """cconv_epilogue_t: residual rows updated in place, optional outer residual,
    optional logical -> physical row map."""
    _fields_ = [("residual", ctypes.c_void_p), ("residual_row_stride", ctypes.c_int64),
                ("outer_residual", ctypes.c_void_p), ("outer_row_stride", ctypes.c_int64),
                ("token_indices", ctypes.c_void_p), ("num_rows", ctypes.c_int32)]


class Pool(ctypes.Structure):
    """cconv_pool_t: [slot, channel, column] view of a conv-state pool."""
    _fields_ = [("p", ctypes.c_void_p), ("s_slot", ctypes.c_int64),
                ("s_chan", ctypes.c_int64), ("s_col", ctypes.c_int64),
                ("num_slots", ctypes.c_int32), ("cap", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class GdnState(ctypes.Structure):
    """gdn_state_t: [slot, value head, dk, dv] view of a gated-delta-rule state pool."""
    _fields_ = [("p", ctypes.c_void_p), ("s_slot", ctypes.c_int64), ("s_head", ctypes.c_int64),
                ("num_slots", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class KvCache(ctypes.Structure):
    """kv_cache_t: [page, token, kv head, head_dim] views of a paged k and v cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("s_page", ctypes.c_int64),
                ("s_token", ctypes.c_int64), ("s_head", ctypes.c_int64),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class KvCacheQ8(ctypes.Structure):
    """kv_cache_q8_t: a paged cache of e4m3 rows and the [page, token, kv head] views of their scales."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("s_page", ctypes.c_int64),
                ("s_token", ctypes.c_int64), ("s_head", ctypes.c_int64),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("c_page", ctypes.c_int64), ("c_token", ctypes.c_int64), ("c_head", ctypes.c_int64),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class CConvError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn}: status {status} ({status_string(status)})")
        self.status = status


def load():
    """Load libcconv.so (raises if it has not been built)."""
    global _lib, _fast
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "state_cached_causal_gb300.build.build()")
        lib = ctypes.CDLL(LIB_PATH)
        P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        lib.cconv_fwd_varlen.argtypes = [P, I64, P, P, Pool, P, P, P, I32, I32, I32, I32, I32,
                                         I32, I32, P, I64, P, P]
        lib.cconv_fwd_varlen.restype = ctypes.c_int
        lib.cconv_update.argtypes = [P, I64, Pool, P, P, P, I32, I32, P, P, I32, I32, I32, I32,
                                     I32, P, I64, P, P]
        lib.cconv_update.restype = ctypes.c_int
        lib.cconv_fwd_varlen_fused.argtypes = [P, I64, P, P, Pool, P, P, P, I32, I32, I32, I32,
                                               I32, I32, I32, Epilogue, P, P]
        lib.cconv_fwd_varlen_fused.restype = ctypes.c_int
        lib.cconv_update_fused.argtypes = [P, I64, Pool, P, P, P, I32, I32, P, P, I32, I32, I32,
                                           I32, I32, Epilogue, P, P]
        lib.cconv_update_fused.restype = ctypes.c_int
        lib.cconv_checkpoint_export.argtypes = [P, I64, Pool, P, P, P, I32, P, I32, I32, P, I32,
                                                I32, I32, I32, I32, P, P]
        lib.cconv_checkpoint_export.restype = ctypes.c_int
        lib.cca_qk_conv.argtypes = [P, I64, P, P, P, P, I32, I32, I32, P, I64, P, I32, Pool, P,
                                    I64, P, P, P, I32, I32, I32, I32, P, I64, P, I64, P, P]
        lib.cca_qk_conv.restype = ctypes.c_int
        lib.cca_qk_conv_noalloc.argtypes = lib.cca_qk_conv.argtypes
        lib.cca_qk_conv_noalloc.restype = ctypes.c_int
        lib.cca_qk_conv_fused.argtypes = [P, I64, P, P, P, P, I32, I32, I32, I32, P, I64, P, I32,
                                          P, I64, Pool, P, I64, P, P, P, I32, I32, I32, I32, P,
                                          I64, P, P]
        lib.cca_qk_conv_fused.restype = ctypes.c_int
        F32 = ctypes.c_float
        lib.gdn_fwd_varlen.argtypes = [P, I64, P, I64, P, I64, P, I64, P, I64, P, P, GdnState, P,
                                       P, P, I32, I32, I32, I32, I32, I32, F32, I32, I32, P,
                                       I64, P, P]
        lib.gdn_fwd_varlen.restype = ctypes.c_int
        lib.gdn_update.argtypes = [P, I64, P, I64, P, I64, P, I64, P, I64, P, P, GdnState, P, I32,
                                   I32, P, P, I32, I32, I32, I32, F32, I32, I32, P, I64, P, P]
        lib.gdn_update.restype = ctypes.c_int
        lib.attn_norm_rope_cache.argtypes = [P, I64, P, I64, P, I64, P, P, F32, P, I32, I32, I32,
                                             P, KvCache, P, I32, I32, I32, P, I64, P, P]
        lib.attn_norm_rope_cache.restype = ctypes.c_int
        lib.attn_decode.argtypes = [P, I64, KvCache, P, I64, I32, P, I32, I32, I32, F32, I32, P,
                                    I64, P, P, I64, P, P]
        lib.attn_decode.restype = ctypes.c_int
        lib.attn_decode_workspace_bytes.argtypes = [I32, I32, I32, I32, I32]
        lib.attn_decode_workspace_bytes.restype = I64
        lib.attn_decode_shared.argtypes = [P, I64, KvCache, P, I64, I32, P, I32, P, P, I32, I32, I32,
                                           F32, I32, P, I64, P, P, I64, P, P]
        lib.attn_decode_shared.restype = ctypes.c_int
        lib.attn_decode_shared_workspace_bytes.argtypes = [I32, I32, I32, I32, I32, I32]
        lib.attn_decode_shared_workspace_bytes.restype = I64
        for name in ("attn_norm_rope_cache", "attn_decode", "attn_decode_shared"):
            plain, q8 = getattr(lib, name), getattr(lib, name + "_q8")
            q8.argtypes = [KvCacheQ8 if t is KvCache else t for t in plain.argtypes]
            q8.restype = ctypes.c_int
        lib.kv_cache_read_q8.argtypes = [KvCacheQ8, P, I32, I32, P, I64, P, I64, P, P]
        lib.kv_cache_read_q8.restype = ctypes.c_int
        lib.cconv_status_string.argtypes = [ctypes.c_int]
        lib.cconv_status_string.restype = ctypes.c_char_p
        lib.cconv_abi_version.argtypes = []
        lib.cconv_abi_version.restype = ctypes.c_int
        _fast = _load_fast(lib)
        _lib = lib
        return lib


def _load_fast(lib):
    """The C module with the library's entry points, or None where a part it stands on is
    missing (the functions below then marshal by themselves)."""
    try:
        from . import _fast as mod
        raw, device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    except (ImportError, AttributeError):
        return None
    types = (torch.float32, torch.bfloat16, torch.int32, torch.uint8, torch.bool)
    if _F8 is not None and _F8_SCALE is not None:
        types += (_F8, _F8_SCALE)
    mod.init(lib._handle, types, raw, lambda beside, n: beside.new_empty(n, dtype=torch.uint8), device)
    return mod


def _served(fn, rc):
    """What the C module answered: True for a call made, False for one left to Python."""
    if rc is None:
        return False
    if rc != OK:
        raise CConvError(fn, rc)
    return True


def status_string(status: int) -> str:
    return load().cconv_status_string(int(status)).decode()


def abi_version() -> int:
    return int(load().cconv_abi_version())


# ---- marshalling helpers ---------------------------------------------------

def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return DTYPE_F32
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to libcconv must live on the GPU")
    return ctypes.c_void_p(t.data_ptr())


def _rows(t: torch.Tensor) -> int:
    if t.dim() != 2 or (t.shape[0] > 1 and t.stride(1) != 1):
        raise ValueError("expected a 2-D tensor with contiguous rows")
    return int(t.stride(0)) if t.shape[0] > 0 else int(t.shape[1])


def _pool(view: torch.Tensor) -> Pool:
    if view.dim() != 3:
        raise ValueError("pool view must be [slot, channel, column]")
    s = view.stride()
    return Pool(ctypes.c_void_p(view.data_ptr()), s[0], s[1], s[2], view.shape[0],
                view.shape[2], _dtype_code(view))


def _same_state_dtype(conv_state, delayed_state):
    if delayed_state.dtype != conv_state.dtype:
        raise TypeError("delayed_state must have the conv-state pool's dtype")


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _i32(t, name):
    if t is not None and t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    return t


def _u8(t, name):
    if t is not None and t.dtype not in (torch.uint8, torch.bool):
        raise TypeError(f"{name} must be uint8/bool")
    return t


def _check(fn, status):
    if status != OK:
        raise CConvError(fn, status)


# ---- entry points ----------------------------------------------------------

def cconv_fwd_varlen(x, w, bias, conv_states, state_idx, cu_seqlens, has_init, width,
                     dilation, act, out, dev_err=None, stream=None, num_tokens=None):
    """Varlen causal depthwise conv with state (see cconv_fwd_varlen in cconv.h).

    x, out: [T, C]; w: [C, width]; bias: [C] or None; conv_states: [slot, C, cap]
    view (fp32 or bf16, whatever x's dtype); state_idx/cu_seqlens: int32;
    has_init: uint8/bool or None.
    """
    _i32(state_idx, "state_idx")
    _i32(cu_seqlens, "cu_seqlens")
    _u8(has_init, "has_init")
    T = int(x.shape[0]) if num_tokens is None else int(num_tokens)
    rc = load().cconv_fwd_varlen(
        _ptr(x), _rows(x), _ptr(w), _ptr(bias), _pool(conv_states), _ptr(state_idx),
        _ptr(cu_seqlens), _ptr(has_init), int(state_idx.shape[0]), T, int(x.shape[1]),
        int(width), int(dilation), int(act), _dtype_code(x), _ptr(out), _rows(out),
        _ptr(dev_err), _stream(stream))
    _check("cconv_fwd_varlen", rc)


def cconv_update(x, conv_states, w, bias, state_idx, n_spec, num_accepted, has_init, width,
                 dilation, act, out, dev_err=None, stream=None):
    """Decode / speculative decode against the pool (see cconv_update in cconv.h).

    x, out: [B*(1+n_spec), C]; num_accepted: int32 [B] when n_spec > 0.
    """
    _i32(state_idx, "state_idx")
    _i32(num_accepted, "num_accepted")
    _u8(has_init, "has_init")
    rc = load().cconv_update(
        _ptr(x), _rows(x), _pool(conv_states), _ptr(w), _ptr(bias), _ptr(state_idx),
        int(state_idx.shape[0]), int(n_spec), _ptr(num_accepted), _ptr(has_init),
        int(x.shape[1]), int(width), int(dilation), int(act), _dtype_code(x), _ptr(out),
        _rows(out), _ptr(dev_err), _stream(stream))
    _check("cconv_update", rc)


def _epilogue(residual, outer, token_indices, x):
    _i32(token_indices, "token_indices")
    return Epilogue(_ptr(residual), _rows(residual), _ptr(outer),
                    _rows(outer) if outer is not None else 0, _ptr(token_indices),
                    int(x.shape[0]))


def cconv_fwd_varlen_fused(x, w, bias, conv_states, state_idx, cu_seqlens, has_init, width,
                           dilation, act, residual, outer=None, token_indices=None,
                           dev_err=None, stream=None, num_tokens=None):
    """cconv_fwd_varlen with the fused residual epilogue (see cconv_fwd_varlen_fused
    in cconv.h): residual[p] += act(conv)[i] (+ outer[p]), p = token_indices[i].

    x, residual, outer: [R, C] physical rows; num_tokens: logical rows (default
    len(token_indices), else R).
    """
    _i32(state_idx, "state_idx")
    _i32(cu_seqlens, "cu_seqlens")
    _u8(has_init, "has_init")
    if num_tokens is None:
        num_tokens = int(token_indices.shape[0]) if token_indices is not None else int(x.shape[0])
    rc = load().cconv_fwd_varlen_fused(
        _ptr(x), _rows(x), _ptr(w), _ptr(bias), _pool(conv_states), _ptr(state_idx),
        _ptr(cu_seqlens), _ptr(has_init), int(state_idx.shape[0]), int(num_tokens),
        int(x.shape[1]), int(width), int(dilation), int(act), _dtype_code(x),
        _epilogue(residual, outer, token_indices, x), _ptr(dev_err), _stream(stream))
    _check("cconv_fwd_varlen_fused", rc)


def cconv_update_fused(x, conv_states, w, bias, state_idx, n_spec, num_accepted, has_init,
                       width, dilation, act, residual, outer=None, token_indices=None,
                       dev_err=None, stream=None):
    """cconv_update with the fused residual epilogue (see cconv_update_fused in
    cconv.h); request s owns logical rows [s*q, s*q + q)."""
    _i32(state_idx, "state_idx")
    _i32(num_accepted, "num_accepted")
    _u8(has_init, "has_init")
    rc = load().cconv_update_fused(
        _ptr(x), _rows(x), _pool(conv_states), _ptr(w), _ptr(bias), _ptr(state_idx),
        int(state_idx.shape[0]), int(n_spec), _ptr(num_accepted), _ptr(has_init),
        int(x.shape[1]), int(width), int(dilation), int(act), _dtype_code(x),
        _epilogue(residual, outer, token_indices, x), _ptr(dev_err), _stream(stream))
    _check("cconv_update_fused", rc)


def cconv_checkpoint_export(x, conv_states, ckpt_seq, ckpt_offset, ckpt_slot, cu_seqlens,
                            width, dilation, token_indices=None, num_tokens=None,
                            dev_err=None, stream=None):
    """Prefill checkpoint export (see cconv_checkpoint_export in cconv.h): the conv
    window ending at ckpt_offset[k] of request ckpt_seq[k] into slot ckpt_slot[k].

    x: [R, C] physical rows; ckpt_*: int32 [K]; cu_seqlens: int32 [B+1] over
    num_tokens logical rows (default len(token_indices), else R).
    """
    for t, n in ((ckpt_seq, "ckpt_seq"), (ckpt_offset, "ckpt_offset"), (ckpt_slot, "ckpt_slot"),
                 (cu_seqlens, "cu_seqlens"), (token_indices, "token_indices")):
        _i32(t, n)
    if num_tokens is None:
        num_tokens = int(token_indices.shape[0]) if token_indices is not None else int(x.shape[0])
    rc = load().cconv_checkpoint_export(
        _ptr(x), _rows(x), _pool(conv_states), _ptr(ckpt_seq), _ptr(ckpt_offset),
        _ptr(ckpt_slot), int(ckpt_seq.shape[0]), _ptr(cu_seqlens), int(cu_seqlens.shape[0]) - 1,
        int(num_tokens), _ptr(token_indices), int(x.shape[0]), int(x.shape[1]), int(width),
        int(dilation), _dtype_code(x), _ptr(dev_err), _stream(stream))
    _check("cconv_checkpoint_export", rc)


def cca_qk_conv(qk, w_dw, b_dw, w_gr, b_gr, groups, t0, t1, delayed, delayed_init,
                conv_state, delayed_state, state_idx, cu_seqlens, has_init, out_qk,
                out_delayed_prev, dev_err=None, stream=None, num_tokens=None):
    """Zaya CCA two-stage q/k conv + delayed-v shift (see cca_qk_conv in cconv.h)."""
    _cca_call("cca_qk_conv", qk, w_dw, b_dw, w_gr, b_gr, groups, t0, t1, delayed,
              delayed_init, conv_state, delayed_state, state_idx, cu_seqlens, has_init, out_qk,
              out_delayed_prev, dev_err, stream, num_tokens)


def cca_qk_conv_noalloc(qk, w_dw, b_dw, w_gr, b_gr, groups, t0, t1, delayed, delayed_init,
                        conv_state, delayed_state, state_idx, cu_seqlens, has_init, out_qk,
                        out_delayed_prev, dev_err=None, stream=None, num_tokens=None):
    """cca_qk_conv whose kernel scratch lives in a fixed array inside the library,
    for callers that must not allocate (see cca_qk_conv_noalloc in cconv.h). Calls
    whose kernels overlap on the GPU share that scratch and race."""
    _cca_call("cca_qk_conv_noalloc", qk, w_dw, b_dw, w_gr, b_gr, groups, t0, t1, delayed,
              delayed_init, conv_state, delayed_state, state_idx, cu_seqlens, has_init, out_qk,
              out_delayed_prev, dev_err, stream, num_tokens)


def _cca_call(fn, qk, w_dw, b_dw, w_gr, b_gr, groups, t0, t1, delayed, delayed_init,
              conv_state, delayed_state, state_idx, cu_seqlens, has_init, out_qk,
              out_delayed_prev, dev_err, stream, num_tokens):
    _same_state_dtype(conv_state, delayed_state)
    _i32(state_idx, "state_idx")
    _i32(cu_seqlens, "cu_seqlens")
    _u8(has_init, "has_init")
    T = int(qk.shape[0]) if num_tokens is None else int(num_tokens)
    rc = getattr(load(), fn)(
        _ptr(qk), _rows(qk), _ptr(w_dw), _ptr(b_dw), _ptr(w_gr), _ptr(b_gr), int(groups),
        int(t0), int(t1), _ptr(delayed), _rows(delayed), _ptr(delayed_init),
        int(delayed.shape[1]), _pool(conv_state), _ptr(delayed_state), _rows(delayed_state),
        _ptr(state_idx), _ptr(cu_seqlens), _ptr(has_init), int(state_idx.shape[0]), T,
        int(qk.shape[1]), _dtype_code(qk), _ptr(out_qk), _rows(out_qk),
        _ptr(out_delayed_prev), _rows(out_delayed_prev), _ptr(dev_err), _stream(stream))
    _check(fn, rc)


def cca_qk_conv_fused(qk, w_dw, b_dw, w_gr, b_gr, groups, num_q_heads, t0, t1, delayed,
                      delayed_init, v_current, conv_state, delayed_state, state_idx, cu_seqlens,
                      has_init, out, dev_err=None, stream=None, num_tokens=None):
    """cca_qk_conv with ZayaCCA.project's residual mix and value assembly (see
    cca_qk_conv_fused in cconv.h); out: [T, Cqk + 2*Dv] = [query | key | value]."""
    _same_state_dtype(conv_state, delayed_state)
    _i32(state_idx, "state_idx")
    _i32(cu_seqlens, "cu_seqlens")
    _u8(has_init, "has_init")
    T = int(qk.shape[0]) if num_tokens is None else int(num_tokens)
    rc = load().cca_qk_conv_fused(
        _ptr(qk), _rows(qk), _ptr(w_dw), _ptr(b_dw), _ptr(w_gr), _ptr(b_gr), int(groups),
        int(num_q_heads), int(t0), int(t1), _ptr(delayed), _rows(delayed), _ptr(delayed_init),
        int(delayed.shape[1]), _ptr(v_current), _rows(v_current), _pool(conv_state),
        _ptr(delayed_state), _rows(delayed_state), _ptr(state_idx), _ptr(cu_seqlens),
        _ptr(has_init), int(state_idx.shape[0]), T, int(qk.shape[1]), _dtype_code(qk),
        _ptr(out), _rows(out), _ptr(dev_err), _stream(stream))
    _check("cca_qk_conv_fused", rc)



# ---- the mixers behind the convolutions --------------------------------------
# A decode step's calls are short, so their plain cases are marshalled in C (csrc/fast.c);
# what that leaves -- another stream, anything unusual, whatever is wrong -- is checked and
# marshalled here, where each tensor's sizes and strides are read once.

_CODES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}


def _raw(*tensors):
    """Device addresses (None for None) of tensors that all live on the current device, whose stream
    and SMs the library takes."""
    got, on = [], None
    for t in tensors:
        if t is None:
            got.append(None)
            continue
        if not t.is_cuda:
            raise ValueError("tensors passed to libcconv must live on the GPU")
        if on is None:
            on = torch.cuda.current_device()
        if t.get_device() != on:
            raise ValueError(f"tensors passed to libcconv must live on the current device ({on})")
        got.append(t.data_ptr())
    return got


def _raw_stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if stream.device.index != torch.cuda.current_device():
        raise ValueError("the stream must be one of the current device")
    return stream.cuda_stream


def _heads(t, name, dtype, rows, heads=None, dim=None):
    """(heads, dim, row stride) of a [rows, heads, dim] tensor whose rows are contiguous."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must have the call's dtype")
    s, st = t.shape, t.stride()
    if len(s) != 3 or st[2] != 1 or (st[1] != s[2] and s[1] > 1):
        raise ValueError(f"{name} must be [rows, heads, dim] with contiguous rows")
    n, h, d = s
    if n < rows or (heads is not None and (h != heads or d != dim)):
        raise ValueError(f"{name} has the wrong rows, heads or head size")
    return h, d, (st[0] if n > 1 else max(st[0], h * d))


def _vector(t, name, dtype, n):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n}")


def _entries(t, name, n, flags=False):
    """An index vector (or a vector of flags) whose first n entries the library reads side by side."""
    if t is None:
        return
    (_u8 if flags else _i32)(t, name)
    if t.dim() == 0 or t.numel() != t.shape[0] or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector")
    if t.numel() < n:
        raise ValueError(f"{name} must have {n} entries")


def _error_word(dev_err):
    if dev_err is not None and (_i32(dev_err, "dev_err").numel() < 1):
        raise ValueError("dev_err must have an entry")


def _gates(t, name, dtype, rows, hv):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must have the call's dtype")
    s, st = t.shape, t.stride()
    if len(s) != 2 or s[0] < rows or s[1] != hv or (hv > 1 and st[1] != 1):
        raise ValueError(f"{name} must be [rows, value heads] with contiguous rows")
    return st[0] if s[0] > 1 else max(st[0], hv)


def _gdn_call(fn, q, k, v, a, b, A_log, dt_bias, states, out, rows, scale, l2norm, stream, dev_err,
              index, middle):
    """index: the int32/uint8 tensors after the pool; middle(addresses) -> the C arguments between
    the pool and the head counts."""
    _error_word(dev_err)
    dtype = k.dtype
    hk, dk, ks = _heads(k, "k", dtype, rows)
    hv, dv, vs = _heads(v, "v", dtype, rows)
    qs = _heads(q, "q", dtype, rows, hk, dk)[2]
    os_ = _heads(out, "out", dtype, rows, hv, dv)[2]
    a_s, b_s = _gates(a, "a", dtype, rows, hv), _gates(b, "b", dtype, rows, hv)
    _vector(A_log, "A_log", torch.float32, hv)
    _vector(dt_bias, "dt_bias", torch.float32, hv)
    s, st = states.shape, states.stride()
    if len(s) != 4 or s[1] != hv or s[2] != dk or s[3] != dv or st[3] != 1 or st[2] != dv:
        raise ValueError("states must be [slots, value heads, dk, dv], the last two contiguous")
    code, st_code = _CODES.get(dtype), _CODES.get(states.dtype)
    if code is None or st_code is None:
        raise TypeError(f"unsupported dtype {dtype} or {states.dtype}")
    P = _raw(q, k, v, a, b, A_log, dt_bias, states, out, dev_err, *index)
    # a pool of one slot or one head may carry any stride there
    pool = GdnState(P[7], st[0] if s[0] > 1 else max(st[0], hv * dk * dv),
                    st[1] if hv > 1 else max(st[1], dk * dv), s[0], st_code)
    rc = getattr(load(), fn)(P[0], qs, P[1], ks, P[2], vs, P[3], a_s, P[4], b_s, P[5], P[6], pool,
                             *middle(P[10:]), hk, hv, dk, dv, scale, l2norm, code, P[8], os_, P[9],
                             _raw_stream(stream))
    if rc != OK:
        raise CConvError(fn, rc)


def gdn_fwd_varlen(q, k, v, a, b, A_log, dt_bias, states, state_idx, cu_seqlens, has_init, scale,
                   out, qk_l2norm=True, dev_err=None, stream=None, num_tokens=None):
    """Gated delta rule over a packed varlen batch (see gdn_fwd_varlen in cconv.h).

    q, k: [T, Hk, dk]; v, out: [T, Hv, dv]; a, b: [T, Hv] raw gate projections; A_log,
    dt_bias: fp32 [Hv]; states: [slots, Hv, dk, dv] fp32 or bf16, updated in place;
    state_idx/cu_seqlens: int32; has_init: uint8/bool or None.
    """
    if stream is None and (_lib or load()) and _fast is not None and _served(
            "gdn_fwd_varlen", _fast.gdn_fwd_varlen(
                q, k, v, a, b, A_log, dt_bias, states, state_idx, cu_seqlens, has_init, scale, out,
                qk_l2norm, dev_err, num_tokens)):
        return
    _entries(state_idx, "state_idx", 0)
    T = q.shape[0] if num_tokens is None else int(num_tokens)
    B = state_idx.shape[0]
    _entries(cu_seqlens, "cu_seqlens", B + 1)
    _entries(has_init, "has_init", B, flags=True)
    if cu_seqlens.shape[0] != B + 1:
        raise ValueError("cu_seqlens must have one entry more than state_idx")
    _gdn_call("gdn_fwd_varlen", q, k, v, a, b, A_log, dt_bias, states, out, T, scale,
              1 if qk_l2norm else 0, stream, dev_err, (state_idx, cu_seqlens, has_init),
              lambda P: (P[0], P[1], P[2], B, T))


def gdn_update(q, k, v, a, b, A_log, dt_bias, states, state_idx, n_spec, num_accepted, has_init,
               scale, out, qk_l2norm=True, dev_err=None, stream=None):
    """Gated delta rule for decode / speculative decode (see gdn_update in cconv.h).

    Rows [s*(1+n_spec), (s+1)*(1+n_spec)) belong to request s; state_idx: int32 [B, 1+n_spec]
    (or [B] when n_spec is 0), the slot of the state after each token; num_accepted: int32 [B]
    when n_spec > 0.
    """
    if stream is None and (_lib or load()) and _fast is not None and _served(
            "gdn_update", _fast.gdn_update(
                q, k, v, a, b, A_log, dt_bias, states, state_idx, n_spec, num_accepted, has_init,
                scale, out, qk_l2norm, dev_err)):
        return
    _i32(state_idx, "state_idx")
    _i32(num_accepted, "num_accepted")
    B = state_idx.shape[0]
    _entries(has_init, "has_init", B, flags=True)
    if n_spec > 0:                  # (else it is not read)
        _entries(num_accepted, "num_accepted", B)
    if state_idx.numel() != B * (1 + n_spec) or not state_idx.is_contiguous():
        raise ValueError("state_idx must be a contiguous [requests, 1 + n_spec]")
    _gdn_call("gdn_update", q, k, v, a, b, A_log, dt_bias, states, out, B * (1 + n_spec), scale,
              1 if qk_l2norm else 0, stream, dev_err, (state_idx, num_accepted, has_init),
              lambda P: (P[0], B, n_spec, P[1], P[2]))


def _cache(k_cache, v_cache, dtype):
    """(shape, strides, dtype code) of a paged cache's two views."""
    s, st = k_cache.shape, k_cache.stride()
    if len(s) != 4 or v_cache.shape != s or st[3] != 1:
        raise ValueError("caches must be [pages, page_size, kv heads, head_dim] of one shape")
    if v_cache.stride() != st:
        raise ValueError("k_cache and v_cache must have the same strides")
    if k_cache.dtype is not dtype or v_cache.dtype is not dtype:
        raise TypeError("the caches must have q's dtype")
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    # a dimension of one entry may carry any stride
    st = [x if n > 1 else max(x, s[3]) for x, n in zip(st, s)]
    return s, st, code


def _cache_q8(k_cache, v_cache, k_scale, v_scale):
    """(shape, strides, scale strides) of an 8-bit cache's four views."""
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.dtype is not _F8:          # (nothing is where there is no such type)
            raise TypeError(f"{name} must be float8_e4m3fn")
    for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if t.dtype not in (torch.uint8, _F8_SCALE):
            raise TypeError(f"{name} must be uint8 or float8_e8m0fnu")
    s, st = k_cache.shape, k_cache.stride()
    if len(s) != 4 or v_cache.shape != s or st[3] != 1:
        raise ValueError("caches must be [pages, page_size, kv heads, head_dim] of one shape")
    if v_cache.stride() != st:
        raise ValueError("k_cache and v_cache must have the same strides")
    if k_scale.shape != s[:3] or v_scale.shape != s[:3]:
        raise ValueError("scales must be [pages, page_size, kv heads], as the caches")
    ct = k_scale.stride()
    if v_scale.stride() != ct:
        raise ValueError("k_scale and v_scale must have the same strides")
    # a dimension of one entry may carry any stride
    st = [x if n > 1 else max(x, s[3]) for x, n in zip(st, s)]
    return s, st, [x if n > 1 else max(x, 1) for x, n in zip(ct, s)]


def _q8_struct(P, s, st, ct):
    return KvCacheQ8(P[0], P[1], st[0], st[1], st[2], P[2], P[3], ct[0], ct[1], ct[2], *s)


def _call_dtype(dtype):
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def attn_norm_rope_cache(q, k, v, q_weight, k_weight, eps, cos_sin, positions, interleaved,
                         k_cache, v_cache, slot_mapping, q_out, dev_err=None, stream=None):
    """Head norm, rotation and cache write (see attn_norm_rope_cache in cconv.h).

    q, q_out: [T, Hq, D]; k, v: [T, Hkv, D]; q_weight, k_weight: [D] or None; cos_sin: fp32
    [max_position, rot_dim], the cosines then the sines; caches: [pages, page_size, Hkv, D]
    views (any order of storage with contiguous D); positions, slot_mapping: int32 [T].
    """
    if stream is None and (_lib or load()) and _fast is not None and _served(
            "attn_norm_rope_cache", _fast.attn_norm_rope_cache(
                q, k, v, q_weight, k_weight, eps, cos_sin, positions, interleaved, k_cache,
                v_cache, slot_mapping, q_out, dev_err)):
        return
    (pages, page, hkv, dim), st, code = _cache(k_cache, v_cache, q.dtype)
    _norm_call("attn_norm_rope_cache", q, k, v, q_weight, k_weight, eps, cos_sin, positions,
               interleaved, slot_mapping, q_out, dev_err, stream, hkv, dim, (k_cache, v_cache),
               lambda P: KvCache(P[0], P[1], st[0], st[1], st[2], pages, page, hkv, dim, code))


def _norm_call(fn, q, k, v, q_weight, k_weight, eps, cos_sin, positions, interleaved, slot_mapping,
               q_out, dev_err, stream, hkv, dim, views, cache):
    """views: the cache's tensors; cache(addresses) -> its C struct."""
    _entries(positions, "positions", q.shape[0])
    _entries(slot_mapping, "slot_mapping", q.shape[0])
    _error_word(dev_err)
    dtype, code = q.dtype, _call_dtype(q.dtype)
    T, hq = q.shape[0], q.shape[1]
    qs = _heads(q, "q", dtype, T, hq, dim)[2]
    ks = _heads(k, "k", dtype, T, hkv, dim)[2]
    vs = _heads(v, "v", dtype, T, hkv, dim)[2]
    os_ = _heads(q_out, "q_out", dtype, T, hq, dim)[2]
    if q_weight is not None:
        _vector(q_weight, "q_weight", dtype, dim)
    if k_weight is not None:
        _vector(k_weight, "k_weight", dtype, dim)
    if cos_sin.dtype is not torch.float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
        raise TypeError("cos_sin must be contiguous float32 [max_position, rot_dim]")
    P = _raw(q, k, v, q_weight, k_weight, cos_sin, positions, slot_mapping, q_out, dev_err, *views)
    rc = getattr(load(), fn)(P[0], qs, P[1], ks, P[2], vs, P[3], P[4], eps, P[5], cos_sin.shape[0],
                             cos_sin.shape[1], 1 if interleaved else 0, P[6], cache(P[10:]), P[7],
                             T, hq, code, P[8], os_, P[9], _raw_stream(stream))
    if rc != OK:
        raise CConvError(fn, rc)


def attn_norm_rope_cache_q8(q, k, v, q_weight, k_weight, eps, cos_sin, positions, interleaved,
                            k_cache, v_cache, k_scale, v_scale, slot_mapping, q_out, dev_err=None,
                            stream=None):
    """attn_norm_rope_cache into a cache in 8 bits (see attn_norm_rope_cache_q8 in cconv.h).

    caches: float8_e4m3fn [pages, page_size, Hkv, D] views; k_scale, v_scale: uint8 (or
    float8_e8m0fnu) [pages, page_size, Hkv] views, the biased exponents of the rows' powers of two.
    """
    if stream is None and (_lib or load()) and _fast is not None and _served(
            "attn_norm_rope_cache_q8", _fast.attn_norm_rope_cache_q8(
                q, k, v, q_weight, k_weight, eps, cos_sin, positions, interleaved, k_cache,
                v_cache, k_scale, v_scale, slot_mapping, q_out, dev_err)):
        return
    s, st, ct = _cache_q8(k_cache, v_cache, k_scale, v_scale)
    _norm_call("attn_norm_rope_cache_q8", q, k, v, q_weight, k_weight, eps, cos_sin, positions,
               interleaved, slot_mapping, q_out, dev_err, stream, s[2], s[3],
               (k_cache, v_cache, k_scale, v_scale), lambda P: _q8_struct(P, s, st, ct))


def kv_cache_read_q8(k_cache, v_cache, k_scale, v_scale, slot_mapping, k_out, v_out, dev_err=None,
                     stream=None):
    """Rows of a cache in 8 bits as fp32 or bf16 (see kv_cache_read_q8 in cconv.h).

    caches and scales as attn_norm_rope_cache_q8; slot_mapping: int32 [T], negative to leave a row
    as it is; k_out, v_out: [T, Hkv, D].
    """
    if stream is None and (_lib or load()) and _fast is not None and _served(
            "kv_cache_read_q8", _fast.kv_cache_read_q8(
                k_cache, v_cache, k_scale, v_scale, slot_mapping, k_out, v_out, dev_err)):
        return
    _entries(slot_mapping, "slot_mapping", 0)
    _error_word(dev_err)
    s, st, ct = _cache_q8(k_cache, v_cache, k_scale, v_scale)
    T, dtype = slot_mapping.shape[0], k_out.dtype
    code = _call_dtype(dtype)
    ks = _heads(k_out, "k_out", dtype, T, s[2], s[3])[2]
    vs = _heads(v_out, "v_out", dtype, T, s[2], s[3])[2]
    P = _raw(k_cache, v_cache, k_scale, v_scale, slot_mapping, k_out, v_out, dev_err)
    rc = load().kv_cache_read_q8(_q8_struct(P, s, st, ct), P[4], T, code, P[5], ks,
                                 P[6], vs, P[7], _raw_stream(stream))
    if rc != OK:
        raise CConvError("kv_cache_read_q8", rc)


def attn_decode_workspace_bytes(num_seqs, n_spec, num_q_heads, num_kv_heads, head_dim):
    """Bytes of workspace of an attn_decode call of these sizes."""
    n = load().attn_decode_workspace_bytes(num_seqs, n_spec, num_q_heads, num_kv_heads, head_dim)
    if n < 0:
        raise CConvError("attn_decode_workspace_bytes", n)
    return n


def attn_decode(q, k_cache, v_cache, block_table, seq_lens, n_spec, scale, out, lse=None,
                workspace=None, dev_err=None, stream=None):
    """Attention of new tokens over a paged cache (see attn_decode in cconv.h).

    q, out: [B*(1+n_spec), Hq, D]; block_table: int32 [B, width]; seq_lens: int32 [B], the
    cached tokens with the new ones; lse: fp32 [B*(1+n_spec), Hq] or None; workspace: a uint8
    tensor of attn_decode_workspace_bytes() or None (allocated for the call).
    """
    if stream is None and (_lib or load()) and _fast is not None and _served(
            "attn_decode", _fast.attn_decode(
                q, k_cache, v_cache, block_table, seq_lens, n_spec, scale, out, lse, workspace,
                dev_err)):
        return
    (pages, page, hkv, dim), st, code = _cache(k_cache, v_cache, q.dtype)
    _decode_call("attn_decode", q, block_table, seq_lens, n_spec, scale, out, lse, workspace, dev_err,
                 stream, hkv, dim, (k_cache, v_cache),
                 lambda P: KvCache(P[0], P[1], st[0], st[1], st[2], pages, page, hkv, dim, code))


def _decode_call(fn, q, block_table, seq_lens, n_spec, scale, out, lse, workspace, dev_err, stream,
                 hkv, dim, views, cache, groups=None):
    """views: the cache's tensors; cache(addresses) -> its C struct; groups: (cu_groups, prefix_lens)
    of the shared form."""
    _i32(block_table, "block_table")
    _entries(seq_lens, "seq_lens", 0)
    _error_word(dev_err)
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    dtype, code = q.dtype, _call_dtype(q.dtype)
    B = seq_lens.shape[0]
    rows, hq = B * (1 + n_spec), q.shape[1]
    qs = _heads(q, "q", dtype, rows, hq, dim)[2]
    os_ = _heads(out, "out", dtype, rows, hq, dim)[2]
    ts, tst = block_table.shape, block_table.stride()
    if len(ts) != 2 or ts[0] < B or (ts[1] > 1 and tst[1] != 1):
        raise ValueError("block_table must be [requests, width] with contiguous rows")
    if lse is not None and (lse.dtype is not torch.float32 or not lse.is_contiguous()
                            or lse.shape[0] < rows or lse.shape[1:] != (hq,)):
        raise ValueError("lse must be contiguous float32 [rows, heads]")
    more, G = (), 0
    if groups is not None:
        _entries(groups[1], "prefix_lens", 0)
        G = groups[1].shape[0]
        _entries(groups[0], "cu_groups", G + 1)
        if groups[0].shape[0] != G + 1:
            raise ValueError("cu_groups must have one entry more than prefix_lens")
        more = groups
    P = _raw(q, block_table, seq_lens, out, lse, workspace, dev_err, *views, *more)
    if workspace is None:
        need = (attn_decode_workspace_bytes(B, n_spec, hq, hkv, dim) if groups is None else
                attn_decode_shared_workspace_bytes(B, G, n_spec, hq, hkv, dim))
        if stream is None:
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
        else:
            with torch.cuda.stream(stream):     # the call's stream owns it
                workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
        P[5] = workspace.data_ptr()
    rc = getattr(load(), fn)(P[0], qs, cache(P[7:]), P[1],
                             tst[0] if ts[0] > 1 else max(tst[0], ts[1]), ts[1], P[2], B,
                             *((P[-2], P[-1], G) if more else ()), n_spec, hq, scale, code, P[3],
                             os_, P[4], P[5], workspace.numel() * workspace.element_size(), P[6],
                             _raw_stream(stream))
    if rc != OK:
        raise CConvError(fn, rc)


def attn_decode_q8(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, n_spec, scale, out,
                   lse=None, workspace=None, dev_err=None, stream=None):
    """attn_decode over a cache in 8 bits (see attn_decode_q8 in cconv.h).

    caches and scales as attn_norm_rope_cache_q8; the rest, and the workspace, as attn_decode.
    """
    if stream is None and (_lib or load()) and _fast is not None and _served(
            "attn_decode_q8", _fast.attn_decode_q8(
                q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, n_spec, scale, out,
                lse, workspace, dev_err)):
        return
    s, st, ct = _cache_q8(k_cache, v_cache, k_scale, v_scale)
    _decode_call("attn_decode_q8", q, block_table, seq_lens, n_spec, scale, out, lse, workspace,
                 dev_err, stream, s[2], s[3], (k_cache, v_cache, k_scale, v_scale),
                 lambda P: _q8_struct(P, s, st, ct))


def attn_decode_shared_workspace_bytes(num_seqs, num_groups, n_spec, num_q_heads, num_kv_heads,
                                       head_dim):
    """Bytes of workspace of an attn_decode_shared (or .._q8) call of these sizes."""
    n = load().attn_decode_shared_workspace_bytes(num_seqs, num_groups, n_spec, num_q_heads,
                                                  num_kv_heads, head_dim)
    if n < 0:
        raise CConvError("attn_decode_shared_workspace_bytes", n)
    return n


def attn_decode_shared(q, k_cache, v_cache, block_table, seq_lens, cu_groups, prefix_lens, n_spec,
                       scale, out, lse=None, workspace=None, dev_err=None, stream=None):
    """Attention of new tokens of requests that share their first positions in groups (see
    attn_decode_shared in cconv.h).

    cu_groups: int32 [groups + 1], group g holds requests cu_groups[g] to cu_groups[g + 1] - 1;
    prefix_lens: int32 [groups], the positions that it shares, read through the block table of the
    first of its requests that sees all of them; workspace: attn_decode_shared_workspace_bytes() or None (allocated for the
    call). The rest as attn_decode, in bf16.
    """
    if stream is None and (_lib or load()) and _fast is not None and _served(
            "attn_decode_shared", _fast.attn_decode_shared(
                q, k_cache, v_cache, block_table, seq_lens, cu_groups, prefix_lens, n_spec, scale,
                out, lse, workspace, dev_err)):
        return
    (pages, page, hkv, dim), st, code = _cache(k_cache, v_cache, q.dtype)
    _decode_call("attn_decode_shared", q, block_table, seq_lens, n_spec, scale, out, lse, workspace,
                 dev_err, stream, hkv, dim, (k_cache, v_cache),
                 lambda P: KvCache(P[0], P[1], st[0], st[1], st[2], pages, page, hkv, dim, code),
                 (cu_groups, prefix_lens))


def attn_decode_shared_q8(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_groups,
                          prefix_lens, n_spec, scale, out, lse=None, workspace=None, dev_err=None,
                          stream=None):
    """attn_decode_shared over a cache in 8 bits (see attn_decode_shared_q8 in cconv.h).

    caches and scales as attn_norm_rope_cache_q8; the rest as attn_decode_shared.
    """
    if stream is None and (_lib or load()) and _fast is not None and _served(
            "attn_decode_shared_q8", _fast.attn_decode_shared_q8(
                q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_groups,
                prefix_lens, n_spec, scale, out, lse, workspace, dev_err)):
        return
    s, st, ct = _cache_q8(k_cache, v_cache, k_scale, v_scale)
    _decode_call("attn_decode_shared_q8", q, block_table, seq_lens, n_spec, scale, out, lse,
                 workspace, dev_err, stream, s[2], s[3], (k_cache, v_cache, k_scale, v_scale),
                 lambda P: _q8_struct(P, s, st, ct), (cu_groups, prefix_lens))
