"""Thin ctypes binding of libhsa.so: the same names as the C ABI in include/hsa.h.

Only argument marshalling happens here.  Tensors are passed by device
address (``tensor.data_ptr()``); every step of the HSA path runs in the
library's CUDA kernels.  There is no fallback: if libhsa.so is missing, or a
call fails, an exception is raised.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libhsa.so")

# Every symbol the header declares, in header order.
SYMBOLS = [
    "hsa_create", "hsa_destroy", "hsa_last_error", "hsa_set_stream", "hsa_sync_check",
    "hsa_selftest_timeout", "hsa_kernel_launches", "hsa_time_kernels", "hsa_kernel_times", "hsa_n_active", "hsa_schedule", "hsa_score", "hsa_select_from_score",
    "hsa_select_groups", "hsa_ln_gather", "hsa_qkv_project", "hsa_qkv_project_peers", "hsa_linear", "hsa_kv_scatter", "hsa_kv_scatter_packed",
    "hsa_attention", "hsa_attention_kv", "hsa_out_proj_residual", "hsa_mlp_residual",
    "hsa_ln_gather_mod", "hsa_out_proj_residual_gated", "hsa_mlp_residual_mod",
    "hsa_layer_forward", "hsa_layer_forward_cond", "hsa_quant_rows", "hsa_linear_quant",
    "hsa_ln_gather_quant", "hsa_rope_table", "hsa_rope", "hsa_qk_norm_rope", "hsa_cross_attention",
    "hsa_layer_forward_ext", "hsa_step_ext",
    "hsa_embed", "hsa_head", "hsa_euler_step", "hsa_euler_step_score", "hsa_step", "hsa_step_cond",
    "hsa_select_groups_static",
]

STATUS = {0: "HSA_OK", 1: "HSA_ERR_INVALID_ARG", 2: "HSA_ERR_BUDGET", 3: "HSA_ERR_SHAPE",
          4: "HSA_ERR_CUDA", 5: "HSA_ERR_OOM", 6: "HSA_ERR_TIMEOUT", 7: "HSA_ERR_DEVICE_CHECK",
          8: "HSA_ERR_SCRATCH_LIMIT"}

SELECT_STATIC_MAX_N = 131072  # HSA_SELECT_STATIC_MAX_N in include/hsa.h


class HsaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class hsa_model_cfg(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("C", ctypes.c_int), ("D", ctypes.c_int),
                ("H", ctypes.c_int), ("F", ctypes.c_int), ("L", ctypes.c_int)]


class hsa_layer_weights(ctypes.Structure):
    _fields_ = [("w_qkv", ctypes.c_void_p), ("w_o", ctypes.c_void_p),
                ("w_1", ctypes.c_void_p), ("w_2", ctypes.c_void_p)]


class hsa_cross_attn(ctypes.Structure):
    _fields_ = [("w_q", ctypes.c_void_p), ("w_o", ctypes.c_void_p), ("k_txt", ctypes.c_void_p),
                ("v_txt", ctypes.c_void_p), ("n_txt", ctypes.c_int)]


class hsa_cond(ctypes.Structure):
    _fields_ = [("mod", ctypes.POINTER(ctypes.c_void_p)), ("xa", ctypes.POINTER(hsa_cross_attn))]


class hsa_rope_cfg(ctypes.Structure):
    _fields_ = [("n_axes", ctypes.c_int), ("dims", ctypes.c_int * 3), ("base", ctypes.c_double),
                ("scaling", ctypes.c_int), ("factor", ctypes.c_double),
                ("orig_len", ctypes.c_double), ("fast", ctypes.c_double),
                ("slow", ctypes.c_double), ("amp", ctypes.c_double)]


class hsa_qk_rope(ctypes.Structure):
    _fields_ = [("norm", ctypes.c_int), ("w_q", ctypes.c_void_p), ("w_k", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("table", ctypes.c_void_p), ("P", ctypes.c_int),
                ("rot", ctypes.c_int), ("layout", ctypes.c_int)]


class hsa_cross_args(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_start", ctypes.c_void_p), ("n", ctypes.c_int),
                ("B", ctypes.c_int), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("ld_k", ctypes.c_int64), ("bs_k", ctypes.c_int64), ("ld_v", ctypes.c_int64),
                ("bs_v", ctypes.c_int64), ("S", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("kv_len", ctypes.c_void_p), ("kv_mask", ctypes.c_void_p),
                ("scale", ctypes.c_float), ("o", ctypes.c_void_p)]


class hsa_layer_weights_quant(ctypes.Structure):
    _fields_ = [(f, ctypes.c_void_p) for f in ("w_qkv", "w_o", "w_1", "w_2", "s_qkv", "s_o",
                                               "s_1", "s_2")]


class hsa_block_ext(ctypes.Structure):
    _fields_ = [("mod", ctypes.c_void_p), ("xa", ctypes.POINTER(hsa_cross_attn)),
                ("txt_len", ctypes.c_void_p), ("txt_mask", ctypes.c_void_p),
                ("qk", ctypes.POINTER(hsa_qk_rope)),
                ("wq", ctypes.POINTER(hsa_layer_weights_quant))]


ROPE_LAYOUT = {"interleaved": 0, "half": 1}
ROPE_SCALING = {"none": 0, "linear": 1, "base": 2, "parts": 3}
QK_NORM = {"none": 0, "head": 1, "row": 2}


class hsa_model_weights(ctypes.Structure):
    _fields_ = [("w_in", ctypes.c_void_p), ("w_head", ctypes.c_void_p),
                ("layers", ctypes.POINTER(hsa_layer_weights))]


class hsa_kernel_class_time(ctypes.Structure):
    _fields_ = [("calls", ctypes.c_uint64), ("ms", ctypes.c_double), ("work", ctypes.c_double)]


KERNEL_CLASSES = ("attention", "gemm", "rows", "tokens")


class hsa_state(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("v_hat", ctypes.c_void_p),
                ("v_hat_prev", ctypes.c_void_p), ("v_fresh", ctypes.c_void_p),
                ("score", ctypes.c_void_p), ("g", ctypes.c_void_p), ("mask", ctypes.c_void_p),
                ("active_idx", ctypes.c_void_p), ("h", ctypes.c_void_p),
                ("k_cache", ctypes.POINTER(ctypes.c_void_p)),
                ("v_cache", ctypes.POINTER(ctypes.c_void_p))]


_lib = None


def load() -> ctypes.CDLL:
    """Load libhsa.so (built in-tree by ``token_sparse_denoising_layer_b200.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing; build it with "
                           "`python -m token_sparse_denoising_layer_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    L = ctypes.c_int64
    sig = {
        "hsa_create": (I, [ctypes.POINTER(hsa_model_cfg), I, ctypes.POINTER(I), ctypes.POINTER(I),
                           I, I, P, ctypes.POINTER(P)]),
        "hsa_destroy": (None, [P]),
        "hsa_last_error": (ctypes.c_char_p, [P]),
        "hsa_set_stream": (I, [P, P]),
        "hsa_sync_check": (I, [P]),
        "hsa_selftest_timeout": (I, [P, I]),
        "hsa_kernel_launches": (ctypes.c_uint64, [P]),
        "hsa_time_kernels": (I, [P, I]),
        "hsa_kernel_times": (I, [P, ctypes.POINTER(hsa_kernel_class_time), I]),
        "hsa_n_active": (I, [P, I]),
        "hsa_schedule": (I, [P, I, P, P, P, P, ctypes.POINTER(I)]),
        "hsa_score": (I, [P, P, P, P]),
        "hsa_select_from_score": (I, [P, P, P]),
        "hsa_select_groups": (I, [P, P, P, P, P]),
        "hsa_ln_gather": (I, [P, P, P, I, P]),
        "hsa_qkv_project": (I, [P, P, P, P, I, P, P, P]),
        "hsa_qkv_project_peers": (I, [P, P, P, P, I, P, ctypes.POINTER(P), ctypes.POINTER(P), I]),
        "hsa_linear": (I, [P, P, I, I, P, I, P]),
        "hsa_kv_scatter": (I, [P, P, P, P, I, P, P]),
        "hsa_kv_scatter_packed": (I, [P, P, P, I, P, P]),
        "hsa_attention": (I, [P, P, I, P, P, P]),
        "hsa_attention_kv": (I, [P, P, I, P, P, I, P]),
        "hsa_out_proj_residual": (I, [P, P, P, P, I, P]),
        "hsa_mlp_residual": (I, [P, P, P, P, P, I]),
        "hsa_ln_gather_mod": (I, [P, P, P, I, P, P, P]),
        "hsa_out_proj_residual_gated": (I, [P, P, P, P, I, P, P]),
        "hsa_mlp_residual_mod": (I, [P, P, P, P, P, I, P, P, P]),
        "hsa_layer_forward": (I, [P, ctypes.POINTER(hsa_layer_weights), P, P, I, P, P]),
        "hsa_layer_forward_cond": (I, [P, ctypes.POINTER(hsa_layer_weights), P,
                                       ctypes.POINTER(hsa_cross_attn), P, P, I, P, P]),
        "hsa_quant_rows": (I, [P, P, I, I, I, L, P, L, P]),
        "hsa_linear_quant": (I, [P, P, L, P, I, I, P, L, P, I, P]),
        "hsa_ln_gather_quant": (I, [P, P, P, I, P, P, P, P]),
        "hsa_rope_table": (I, [P, ctypes.POINTER(hsa_rope_cfg), P, I, P]),
        "hsa_rope": (I, [P, P, L, I, I, I, P, I, I, P, I, I, P, L]),
        "hsa_qk_norm_rope": (I, [P, ctypes.POINTER(hsa_qk_rope), P, P, I, P, L, P, P, L, P, P, L,
                                 P]),
        "hsa_cross_attention": (I, [P, ctypes.POINTER(hsa_cross_args)]),
        "hsa_layer_forward_ext": (I, [P, ctypes.POINTER(hsa_layer_weights),
                                      ctypes.POINTER(hsa_block_ext), P, P, I, P, P]),
        "hsa_step_ext": (I, [P, ctypes.POINTER(hsa_model_weights), ctypes.POINTER(hsa_state),
                             ctypes.POINTER(hsa_block_ext), I, F, F, I]),
        "hsa_embed": (I, [P, P, P, P, I, P]),
        "hsa_head": (I, [P, P, P, P, I, P]),
        "hsa_euler_step": (I, [P, P, P, P, P, P, F, F]),
        "hsa_euler_step_score": (I, [P, P, P, P, P, P, F, F, P]),
        "hsa_step": (I, [P, ctypes.POINTER(hsa_model_weights), ctypes.POINTER(hsa_state), I, F, F, I]),
        "hsa_step_cond": (I, [P, ctypes.POINTER(hsa_model_weights), ctypes.POINTER(hsa_state),
                              ctypes.POINTER(hsa_cond), I, F, F, I]),
        "hsa_select_groups_static": (I, [P, P, I, ctypes.POINTER(I), I, P, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _p(t) -> Optional[int]:
    """Device address of a tensor (None passes NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libhsa takes CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("libhsa takes contiguous tensors")
    return t.data_ptr()


def _addr(t) -> Optional[int]:
    """Device address of a tensor, or an int taken as a device address as is."""
    if isinstance(t, int):
        return t
    return _p(t)


def _check(ctx, status: int) -> None:
    if status != 0:
        msg = load().hsa_last_error(ctx)
        raise HsaError(status, msg.decode() if msg else "")


class Context:
    """Owns an ``hsa_ctx*``; the handle is ``.ptr``.  Destroyed with ``close()`` or on GC."""

    def __init__(self, ptr: int, cfg: hsa_model_cfg, device: Optional[int] = None):
        self.ptr = ptr
        self.cfg = cfg
        self.device = device  # CUDA device that was current at hsa_create

    def close(self) -> None:
        if self.ptr:
            load().hsa_destroy(self.ptr)
            self.ptr = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _stream_ptr(stream) -> Optional[int]:
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return getattr(stream, "cuda_stream", stream) or None


def hsa_create(N: int, D: int, H: int, F: int, L: int, T: int, budgets: Sequence[int],
               counts: Sequence[int], m: int = 0, C: int = 16, stream=None) -> Context:
    lib = load()
    K = len(budgets)
    cfg = hsa_model_cfg(N, C, D, H, F, L)
    b = (ctypes.c_int * K)(*budgets)
    c = (ctypes.c_int * K)(*counts)
    out = ctypes.c_void_p()
    st = lib.hsa_create(ctypes.byref(cfg), T, b, c, K, m, _stream_ptr(stream), ctypes.byref(out))
    _check(None, st)
    try:
        import torch
        device = torch.cuda.current_device()
    except ImportError:  # a caller with raw addresses and streams only
        device = None
    return Context(out.value, cfg, device)


def hsa_destroy(ctx: Context) -> None:
    ctx.close()


def hsa_set_stream(ctx: Context, stream) -> None:
    _check(ctx.ptr, load().hsa_set_stream(ctx.ptr, _stream_ptr(stream)))


def hsa_sync_check(ctx: Context) -> None:
    _check(ctx.ptr, load().hsa_sync_check(ctx.ptr))


def hsa_selftest_timeout(ctx: Context, timeout_us: int) -> None:
    _check(ctx.ptr, load().hsa_selftest_timeout(ctx.ptr, timeout_us))


def hsa_kernel_launches(ctx: Context) -> int:
    return int(load().hsa_kernel_launches(ctx.ptr))


def hsa_time_kernels(ctx: Context, on: bool) -> None:
    _check(ctx.ptr, load().hsa_time_kernels(ctx.ptr, 1 if on else 0))


def hsa_kernel_times(ctx: Context) -> dict:
    """Per-class totals since timing was turned on or last read: {class:
    {"calls", "ms", "work"}} (work: FLOP for attention and GEMM, bytes for row
    kernels); reading clears them."""
    out = (hsa_kernel_class_time * len(KERNEL_CLASSES))()
    _check(ctx.ptr, load().hsa_kernel_times(ctx.ptr, out, len(KERNEL_CLASSES)))
    return {name: {"calls": int(out[k].calls), "ms": float(out[k].ms), "work": float(out[k].work)}
            for k, name in enumerate(KERNEL_CLASSES)}


def hsa_n_active(ctx: Context, i: int) -> int:
    return load().hsa_n_active(ctx.ptr, i)


def hsa_schedule(ctx: Context, i: int, g, mask, active_idx, n_active_dev=None) -> int:
    n = ctypes.c_int(0)
    _check(ctx.ptr, load().hsa_schedule(ctx.ptr, i, _p(g), _p(mask), _p(active_idx),
                                        _p(n_active_dev), ctypes.byref(n)))
    return n.value


def hsa_score(ctx: Context, v_prev, v_cur, score) -> None:
    _check(ctx.ptr, load().hsa_score(ctx.ptr, _p(v_prev), _p(v_cur), _p(score)))


def hsa_select_from_score(ctx: Context, score, g) -> None:
    _check(ctx.ptr, load().hsa_select_from_score(ctx.ptr, _p(score), _p(g)))


def hsa_select_groups(ctx: Context, v_prev, v_cur, score, g) -> None:
    _check(ctx.ptr, load().hsa_select_groups(ctx.ptr, _p(v_prev), _p(v_cur), _p(score), _p(g)))


def hsa_ln_gather(ctx: Context, x, idx, n: int, u) -> None:
    _check(ctx.ptr, load().hsa_ln_gather(ctx.ptr, _p(x), _p(idx), n, _p(u)))


def hsa_qkv_project(ctx: Context, w_qkv, u, idx, n: int, q, k_cache, v_cache) -> None:
    _check(ctx.ptr, load().hsa_qkv_project(ctx.ptr, _p(w_qkv), _p(u), _p(idx), n, _p(q),
                                           _p(k_cache), _p(v_cache)))


def hsa_qkv_project_peers(ctx: Context, w_qkv, u, idx, n: int, q, k_caches, v_caches) -> None:
    """hsa_qkv_project writing the fresh K/V rows into every cache of the lists.

    ``k_caches`` / ``v_caches`` are equal-length sequences of device buffers
    (tensors) or raw device addresses (ints, e.g. peers' caches mapped into this
    process by CUDA IPC)."""
    if len(k_caches) != len(v_caches):
        raise ValueError("k_caches and v_caches differ in length")
    G = len(k_caches)
    ks = (ctypes.c_void_p * max(G, 1))(*[_addr(t) for t in k_caches])
    vs = (ctypes.c_void_p * max(G, 1))(*[_addr(t) for t in v_caches])
    _check(ctx.ptr, load().hsa_qkv_project_peers(ctx.ptr, _p(w_qkv), _p(u), _p(idx), n, _p(q),
                                                 ks, vs, G))


def hsa_linear(ctx: Context, a, M: int, Kd: int, w, Ncols: int, out) -> None:
    _check(ctx.ptr, load().hsa_linear(ctx.ptr, _p(a), M, Kd, _p(w), Ncols, _p(out)))


def hsa_kv_scatter(ctx: Context, k_rows, v_rows, idx, n: int, k_cache, v_cache) -> None:
    _check(ctx.ptr, load().hsa_kv_scatter(ctx.ptr, _p(k_rows), _p(v_rows), _p(idx), n,
                                          _p(k_cache), _p(v_cache)))


def hsa_kv_scatter_packed(ctx: Context, kv_rows, idx, n: int, k_cache, v_cache) -> None:
    _check(ctx.ptr, load().hsa_kv_scatter_packed(ctx.ptr, _p(kv_rows), _p(idx), n, _p(k_cache),
                                                 _p(v_cache)))


def hsa_attention(ctx: Context, q, n: int, k_cache, v_cache, o) -> None:
    _check(ctx.ptr, load().hsa_attention(ctx.ptr, _p(q), n, _p(k_cache), _p(v_cache), _p(o)))


def hsa_attention_kv(ctx: Context, q, n: int, k, v, n_kv: int, o) -> None:
    _check(ctx.ptr, load().hsa_attention_kv(ctx.ptr, _p(q), n, _p(k), _p(v), n_kv, _p(o)))


def hsa_out_proj_residual(ctx: Context, w_o, o, idx, n: int, x) -> None:
    _check(ctx.ptr, load().hsa_out_proj_residual(ctx.ptr, _p(w_o), _p(o), _p(idx), n, _p(x)))


def hsa_mlp_residual(ctx: Context, w_1, w_2, x, idx, n: int) -> None:
    _check(ctx.ptr, load().hsa_mlp_residual(ctx.ptr, _p(w_1), _p(w_2), _p(x), _p(idx), n))


def _opt(t):
    return _p(t) if t is not None else None


def hsa_ln_gather_mod(ctx: Context, x, idx, n: int, u, shift=None, scale=None) -> None:
    _check(ctx.ptr, load().hsa_ln_gather_mod(ctx.ptr, _p(x), _p(idx), n, _p(u), _opt(shift),
                                             _opt(scale)))


def hsa_out_proj_residual_gated(ctx: Context, w_o, o, idx, n: int, x, gate=None) -> None:
    _check(ctx.ptr, load().hsa_out_proj_residual_gated(ctx.ptr, _p(w_o), _p(o), _p(idx), n,
                                                       _p(x), _opt(gate)))


def hsa_mlp_residual_mod(ctx: Context, w_1, w_2, x, idx, n: int, shift=None, scale=None,
                         gate=None) -> None:
    _check(ctx.ptr, load().hsa_mlp_residual_mod(ctx.ptr, _p(w_1), _p(w_2), _p(x), _p(idx), n,
                                                _opt(shift), _opt(scale), _opt(gate)))


def layer_weights(w_qkv, w_o, w_1, w_2) -> hsa_layer_weights:
    """The struct holds raw device addresses, so it also keeps the tensors alive."""
    s = hsa_layer_weights(_p(w_qkv), _p(w_o), _p(w_1), _p(w_2))
    s._keep = (w_qkv, w_o, w_1, w_2)
    return s


def hsa_layer_forward(ctx: Context, w: hsa_layer_weights, x, idx, n: int, k_cache, v_cache) -> None:
    _check(ctx.ptr, load().hsa_layer_forward(ctx.ptr, ctypes.byref(w), _p(x), _p(idx), n,
                                             _p(k_cache), _p(v_cache)))


def cross_attn(w_q, w_o, k_txt, v_txt, n_txt: int) -> hsa_cross_attn:
    """The struct holds raw device addresses, so it also keeps the tensors alive."""
    s = hsa_cross_attn(_p(w_q), _p(w_o), _p(k_txt), _p(v_txt), n_txt)
    s._keep = (w_q, w_o, k_txt, v_txt)
    return s


def hsa_layer_forward_cond(ctx: Context, w: hsa_layer_weights, mod, xa, x, idx, n: int, k_cache,
                           v_cache) -> None:
    """mod: device fp32 [6, D] or None;  xa: hsa_cross_attn or None."""
    _check(ctx.ptr, load().hsa_layer_forward_cond(
        ctx.ptr, ctypes.byref(w), _p(mod) if mod is not None else None,
        ctypes.byref(xa) if xa is not None else None, _p(x), _p(idx), n, _p(k_cache),
        _p(v_cache)))


def _choice(table: dict, name: str, what: str) -> int:
    if name not in table:
        raise ValueError(f"{what} must be one of {', '.join(table)}, got {name!r}")
    return table[name]


_dtype_names: dict = {}  # tensor types by name, and names by type, filled as types are met


def _dtype(t) -> str:
    """Name of a tensor's type ("bfloat16")."""
    name = _dtype_names.get(t.dtype)
    if name is None:
        name = _dtype_names[t.dtype] = str(t.dtype)[len("torch."):]
        _dtype_names[name] = t.dtype
    return name


def _on_device(ctx: "Optional[Context]", t, what: str) -> None:
    where = t.get_device()
    if where < 0:
        raise ValueError("libhsa takes CUDA tensors")
    if ctx is not None and ctx.device is not None and where != ctx.device:
        raise ValueError(f"{what} is on cuda:{where}, the context on cuda:{ctx.device}")


def _typed(ctx: Optional[Context], t, n: int, dtype: str, what: str, row: int = 0) -> Optional[int]:
    """Device address of a contiguous tensor of at least n elements of a type; with
    `row`, of one that is read as dense rows of that many."""
    if t is None:
        return None
    have = t.numel()
    if (ctx is not None and t.dtype is _dtype_names.get(dtype) and t.get_device() == ctx.device
            and (have == n or have > n and row == 0) and t.is_contiguous()):
        return t.data_ptr()  # (most calls: a call's checks are a good part of its host time)
    if _dtype(t) != dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if have < n:
        raise ValueError(f"{what} needs {n} elements, has {have}")
    _on_device(ctx, t, what)
    if not t.is_contiguous():
        raise ValueError("libhsa takes contiguous tensors")
    if row and have > n > row and t.dim() > 1:  # longer rows (a flat tensor's have any length)
        length = 1
        for x in reversed(t.shape):  # trailing axes that make up a row
            length *= x
            if length >= row:
                break
        if length != row:
            raise ValueError(f"{what} needs rows of {row}, has {tuple(t.shape)}")
    return t.data_ptr()


def _planes(table, rot: int) -> int:
    """Row length that a rotary table [P, rot/2, 2] has to have (one of fewer axes may have any)."""
    return rot if table is not None and table.dim() == 3 else 0


def _rows(ctx: Context, t, n: int, width: int, dtypes: Sequence[str], what: str):
    """(address, row distance in elements) of a 2-D tensor with dense rows."""
    if t is None:
        return None, 0
    shape, stride = t.shape, t.stride()
    if (len(shape) == 2 and shape[0] >= n and shape[1] >= width and stride[1] == 1
            and t.get_device() == ctx.device and _dtype_names.get(t.dtype) in dtypes):
        # a single row has no distance to the next: any legal one will do
        return t.data_ptr(), stride[0] if shape[0] > 1 else (width + 15) // 16 * 16
    if _dtype(t) not in dtypes:
        raise ValueError(f"{what} must be {' or '.join(dtypes)}, got {t.dtype}")
    _on_device(ctx, t, what)
    if len(shape) != 2 or shape[0] < n or shape[1] < width:
        raise ValueError(f"{what} must be [>= {n}, >= {width}], got {tuple(shape)}")
    if stride[1] != 1 and shape[1] > 1:
        raise ValueError(f"{what} must have dense rows")
    return t.data_ptr(), stride[0] if shape[0] > 1 else (width + 15) // 16 * 16


def hsa_quant_rows(ctx: Context, a, n: int, Kd: int, q, scale) -> None:
    """a [>= n, >= Kd] bf16 or fp32 (rows may be strided) -> q int8 rows, scale fp32 [n]."""
    pa, lda = _rows(ctx, a, n, Kd, ("bfloat16", "float32"), "a")
    pq, ldq = _rows(ctx, q, n, Kd, ("int8",), "q")
    kind = 1 if _dtype(a) == "float32" else 0
    _check(ctx.ptr, load().hsa_quant_rows(ctx.ptr, pa, kind, n, Kd, lda, pq, ldq,
                                          _typed(ctx, scale, n, "float32", "scale")))


def hsa_linear_quant(ctx: Context, a, a_scale, M: int, Kd: int, w, w_scale, Ncols: int,
                     out) -> None:
    """out bf16 [M, Ncols] = (a_scale w_scale) a w^T for int8 rows a [M, ..], w [Ncols, ..]
    whose rows are a multiple of 16 bytes apart."""
    pa, lda = _rows(ctx, a, M, Kd, ("int8",), "a")
    pw, ldw = _rows(ctx, w, Ncols, Kd, ("int8",), "w")
    _check(ctx.ptr, load().hsa_linear_quant(
        ctx.ptr, pa, lda, _typed(ctx, a_scale, M, "float32", "a_scale"), M, Kd, pw, ldw,
        _typed(ctx, w_scale, Ncols, "float32", "w_scale"), Ncols,
        _typed(ctx, out, M * Ncols, "bfloat16", "out")))


def hsa_ln_gather_quant(ctx: Context, x, idx, n: int, q, scale, shift=None, mscale=None) -> None:
    D = ctx.cfg.D
    _check(ctx.ptr, load().hsa_ln_gather_quant(
        ctx.ptr, _typed(ctx, x, ctx.cfg.N * D, "float32", "x"), _typed(ctx, idx, n, "int32", "idx"), n,
        _typed(ctx, q, n * D, "int8", "q"), _typed(ctx, scale, n, "float32", "scale"),
        _typed(ctx, shift, D, "float32", "shift"), _typed(ctx, mscale, D, "float32", "mscale")))


def rope_cfg(dims: Sequence[int], base: float = 10000.0, scaling: str = "none",
             factor: float = 1.0, orig_len: float = 0.0, fast: float = 32.0, slow: float = 1.0,
             amp: float = 1.0) -> hsa_rope_cfg:
    """Rotated places of each position axis and how frequencies are scaled (include/hsa.h)."""
    if not 1 <= len(dims) <= 3:
        raise ValueError("a rotary table has 1 to 3 axes")
    d3 = (ctypes.c_int * 3)(*dims)
    return hsa_rope_cfg(len(dims), d3, base, _choice(ROPE_SCALING, scaling, "scaling"), factor, orig_len, fast, slow,
                        amp)


def hsa_rope_table(ctx: Context, cfg: hsa_rope_cfg, pos, P: int, table) -> None:
    """pos int32 [P, n_axes] or None (one axis, positions 0..P-1); table fp32 [P, rot/2, 2]."""
    rot = sum(cfg.dims[:max(0, min(cfg.n_axes, 3))])
    _check(ctx.ptr, load().hsa_rope_table(ctx.ptr, ctypes.byref(cfg),
                                          _typed(ctx, pos, P * cfg.n_axes, "int32", "pos", cfg.n_axes), P,
                                          _typed(ctx, table, P * rot, "float32", "table")))


def hsa_rope(ctx: Context, x, n: int, heads: int, table, P: int, rot: int, out,
             layout: str = "half", pos=None, inverse: bool = False) -> None:
    """Rotate the first ``rot`` places of each of ``heads`` heads of n rows; out may be x."""
    width = heads * (ctx.cfg.D // ctx.cfg.H)
    px, ldx = _rows(ctx, x, n, width, ("bfloat16", "float32"), "x")
    po, ldo = _rows(ctx, out, n, width, (_dtype(x),), "out")
    kind = 1 if _dtype(x) == "float32" else 0
    _check(ctx.ptr, load().hsa_rope(ctx.ptr, px, ldx, kind, n, heads,
                                    _typed(ctx, table, P * rot, "float32", "table", _planes(table, rot)), P, rot,
                                    _typed(ctx, pos, n, "int32", "pos"), _choice(ROPE_LAYOUT, layout, "layout"),
                                    1 if inverse else 0, po, ldo))


def qk_rope(norm: str = "head", w_q=None, w_k=None, eps: float = 1e-6, table=None, P: int = 0,
            rot: int = 0, layout: str = "half") -> hsa_qk_rope:
    """The struct holds raw device addresses, so it also keeps the tensors alive."""
    s = hsa_qk_rope(_choice(QK_NORM, norm, "norm"), _typed(None, w_q, 1, "float32", "w_q"),
                    _typed(None, w_k, 1, "float32", "w_k"), eps,
                    _typed(None, table, P * rot, "float32", "table", _planes(table, rot)), P, rot,
                    _choice(ROPE_LAYOUT, layout, "layout"))
    s._keep = [t for t in (w_q, w_k, table) if t is not None]
    s._widths = [t.numel() for t in (w_q, w_k) if t is not None]
    s._devices = {t.get_device() for t in s._keep}
    return s


def _check_qk(ctx: Context, a: hsa_qk_rope) -> None:
    """The struct's tensors against the context that is to use them."""
    if a.norm:
        width = ctx.cfg.D if a.norm == 2 else ctx.cfg.D // ctx.cfg.H
        for have in getattr(a, "_widths", ()):
            if have != width:  # (weights of a row given for heads would be read as the first head's)
                raise ValueError(f"norm weights need {width} elements, have {have}")
    for where in getattr(a, "_devices", ()):
        if ctx.device is not None and where != ctx.device:
            raise ValueError(f"norm weights or table on cuda:{where}, the context on cuda:{ctx.device}")


def hsa_qk_norm_rope(ctx: Context, a: hsa_qk_rope, idx, n: int, q, k_cache=None, v_cache=None,
                     q_in=None, k_in=None, v_in=None, pos=None) -> None:
    """Norm and rotation of n fresh query and key rows, and the cache write
    (include/hsa.h).  q_in / k_in / v_in may be strided rows, e.g. column
    blocks of a packed [n, 3 D] product; without q_in (k_in) the queries (the
    cache rows idx) change in place."""
    D, N = ctx.cfg.D, ctx.cfg.N
    _check_qk(ctx, a)
    pq, ldq = _rows(ctx, q_in, n, D, ("bfloat16",), "q_in")
    pk, ldk = _rows(ctx, k_in, n, D, ("bfloat16",), "k_in")
    pv, ldv = _rows(ctx, v_in, n, D, ("bfloat16",), "v_in")
    _check(ctx.ptr, load().hsa_qk_norm_rope(
        ctx.ptr, ctypes.byref(a), _typed(ctx, idx, n, "int32", "idx"), _typed(ctx, pos, n, "int32", "pos"),
        n, pq, ldq, _typed(ctx, q, n * D, "bfloat16", "q", D), pk, ldk,
        _typed(ctx, k_cache, N * D, "bfloat16", "k_cache", D), pv, ldv,
        _typed(ctx, v_cache, N * D, "bfloat16", "v_cache", D)))


def _padded(ctx: Context, t, B: int, S: int, width: int, what: str):
    """(address, row distance, sequence distance) of encoder states [B, S, width]."""
    if _dtype(t) != "bfloat16":
        raise ValueError(f"{what} must be bfloat16, got {t.dtype}")
    _on_device(ctx, t, what)
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[0] < B or shape[1] < S or shape[2] < width:
        raise ValueError(f"{what} must be [>= {B}, >= {S}, >= {width}], got {tuple(shape)}")
    if stride[2] != 1 and shape[2] > 1:
        raise ValueError(f"{what} must have dense rows")
    ld = stride[1] if shape[1] > 1 else width
    return t.data_ptr(), ld, stride[0] if shape[0] > 1 else ld * S


def hsa_cross_attention(ctx: Context, q, q_start, n: int, B: int, k, v, S: int, o, kv_len=None,
                        kv_mask=None, kv_heads: Optional[int] = None, scale: float = 0.0) -> None:
    """q, o bf16 [n, D]; q_start int32 [B + 1] or None (n / B rows each); k, v bf16 [B, S, kv_heads * D/H] (rows and
    sequences may be strided, a sequence distance of 0 shares one); kv_len int32 [B];
    kv_mask uint8 or bool [B, S] (or flat), non-zero = seen (include/hsa.h)."""
    D, H = ctx.cfg.D, ctx.cfg.H
    kvh = H if kv_heads is None else kv_heads
    width = kvh * (D // H)
    pk, ldk, bsk = _padded(ctx, k, B, S, width, "k")
    pv, ldv, bsv = _padded(ctx, v, B, S, width, "v")
    if kv_mask is not None:
        if B > 1 and kv_mask.dim() > 1 and kv_mask.shape[-1] != S:  # its rows are read S bytes apart
            raise ValueError(f"kv_mask needs rows of S = {S}, has {tuple(kv_mask.shape)}")
        if _dtype(kv_mask) == "bool":
            import torch
            kv_mask = kv_mask.view(torch.uint8)
    args = hsa_cross_args(_typed(ctx, q, n * D, "bfloat16", "q", D),
                          _typed(ctx, q_start, B + 1, "int32", "q_start"), n, B, pk, pv, ldk, bsk, ldv,
                          bsv, S, kvh, _typed(ctx, kv_len, B, "int32", "kv_len"),
                          _typed(ctx, kv_mask, B * S, "uint8", "kv_mask"), scale,
                          _typed(ctx, o, n * D, "bfloat16", "o"))
    _check(ctx.ptr, load().hsa_cross_attention(ctx.ptr, ctypes.byref(args)))


def quantize_weight(ctx: Context, w):
    """(int8, scale) of a weight [out, in] (bf16 or fp32), one scale per output channel, rows
    padded to a multiple of 16 bytes (hsa_quant_rows)."""
    import torch
    n, K = w.shape
    q = torch.zeros((n, (K + 15) // 16 * 16), dtype=torch.int8, device=w.device)
    scale = torch.empty((n,), dtype=torch.float32, device=w.device)
    hsa_quant_rows(ctx, w, n, K, q, scale)
    return q, scale


def layer_weights_quant(ctx: Context, w_qkv, w_o, w_1, w_2) -> hsa_layer_weights_quant:
    """A block's bf16 weights quantised to 8 bits; the struct keeps its tensors alive."""
    pairs = [quantize_weight(ctx, w) for w in (w_qkv, w_o, w_1, w_2)]
    s = hsa_layer_weights_quant(*[q.data_ptr() for q, _ in pairs],
                                *[t.data_ptr() for _, t in pairs])
    s._keep = pairs
    return s


def block_ext(mod=None, xa: Optional[hsa_cross_attn] = None, txt_len=None, txt_mask=None,
              qk: Optional[hsa_qk_rope] = None,
              wq: Optional[hsa_layer_weights_quant] = None) -> hsa_block_ext:
    """What a block has beyond hsa_layer_forward (include/hsa.h); keeps its parts alive.

    mod: device fp32 [6, D]; txt_len: device int32 [1]; txt_mask: device uint8 or bool [n_txt]."""
    n_txt = 0 if xa is None else xa.n_txt
    if txt_mask is not None and _dtype(txt_mask) == "bool":
        import torch
        txt_mask = txt_mask.view(torch.uint8)
    s = hsa_block_ext(_typed(None, mod, 1, "float32", "mod"),
                      ctypes.pointer(xa) if xa is not None else None,
                      _typed(None, txt_len, 1, "int32", "txt_len"),
                      _typed(None, txt_mask, n_txt, "uint8", "txt_mask"),
                      ctypes.pointer(qk) if qk is not None else None,
                      ctypes.pointer(wq) if wq is not None else None)
    s._keep = (mod, xa, txt_len, txt_mask, qk, wq)
    return s


def _check_ext(ctx: Context, ext: hsa_block_ext) -> None:
    """The struct's tensors against the context that is to use them (those that are
    known: a struct that the caller filled has addresses only)."""
    mod, xa, txt_len, txt_mask, qk, wq = getattr(ext, "_keep", (None,) * 6)
    D, F = ctx.cfg.D, ctx.cfg.F
    pairs = getattr(wq, "_keep", ())  # 8-bit weights and their scales
    for t, what in [(mod, "mod"), (txt_len, "txt_len"), (txt_mask, "txt_mask"),
                    *((t, "a cross-attention tensor") for t in getattr(xa, "_keep", ())),
                    *((t, "an 8-bit weight or scale") for pair in pairs for t in pair)]:
        if t is not None:
            _on_device(ctx, t, what)
    if mod is not None and (mod.numel() < 6 * D or mod.dim() > 1 and mod.shape[-1] != D):
        raise ValueError(f"mod needs rows [6, {D}], has {tuple(mod.shape)}")
    if qk is not None:
        _check_qk(ctx, qk)
        if qk.table is not None and qk.P < ctx.cfg.N:
            raise ValueError(f"a block's rotary table needs a row per token: {ctx.cfg.N}, has {qk.P}")
    for (q, _), shape in zip(pairs, ((3 * D, D), (D, D), (F, D), (D, F))):
        if tuple(q.shape) != shape:
            raise ValueError(f"8-bit block weights need shape {shape}, have {tuple(q.shape)}")


def hsa_layer_forward_ext(ctx: Context, w: Optional[hsa_layer_weights],
                          ext: Optional[hsa_block_ext], x, idx, n: int, k_cache, v_cache) -> None:
    if ext is not None:
        _check_ext(ctx, ext)
    _check(ctx.ptr, load().hsa_layer_forward_ext(
        ctx.ptr, ctypes.byref(w) if w is not None else None,
        ctypes.byref(ext) if ext is not None else None, _p(x), _p(idx), n, _p(k_cache),
        _p(v_cache)))


def hsa_embed(ctx: Context, w_in, x_lat, idx, n: int, h) -> None:
    _check(ctx.ptr, load().hsa_embed(ctx.ptr, _p(w_in), _p(x_lat), _p(idx), n, _p(h)))


def hsa_head(ctx: Context, w_head, h, idx, n: int, v_fresh) -> None:
    _check(ctx.ptr, load().hsa_head(ctx.ptr, _p(w_head), _p(h), _p(idx), n, _p(v_fresh)))


def hsa_euler_step(ctx: Context, x, v_hat, v_hat_prev, v_fresh, mask, sigma_i: float,
                   sigma_next: float) -> None:
    _check(ctx.ptr, load().hsa_euler_step(ctx.ptr, _p(x), _p(v_hat), _p(v_hat_prev), _p(v_fresh),
                                          _p(mask), float(sigma_i), float(sigma_next)))


def hsa_euler_step_score(ctx: Context, x, v_hat, v_hat_prev, v_fresh, mask, sigma_i: float,
                         sigma_next: float, score) -> None:
    _check(ctx.ptr, load().hsa_euler_step_score(ctx.ptr, _p(x), _p(v_hat), _p(v_hat_prev),
                                                _p(v_fresh), _p(mask), float(sigma_i),
                                                float(sigma_next), _p(score)))


class ModelBinding:
    """Keeps the ctypes structs of hsa_step (weights and state) alive."""

    def __init__(self, w_in, w_head, layers, x, v_hat, v_hat_prev, v_fresh, score, g, mask,
                 active_idx, h, k_caches, v_caches):
        L = len(layers)
        self._layers = (hsa_layer_weights * max(L, 1))(*[layer_weights(*lw) for lw in layers])
        self.weights = hsa_model_weights(_p(w_in), _p(w_head), self._layers)
        self._kc = (ctypes.c_void_p * max(L, 1))(*[_p(t) for t in k_caches])
        self._vc = (ctypes.c_void_p * max(L, 1))(*[_p(t) for t in v_caches])
        self.state = hsa_state(_p(x), _p(v_hat), _p(v_hat_prev), _p(v_fresh), _p(score), _p(g),
                               _p(mask), _p(active_idx), _p(h), self._kc, self._vc)
        self._keep = (w_in, w_head, layers, x, v_hat, v_hat_prev, v_fresh, score, g, mask,
                      active_idx, h, k_caches, v_caches)


def hsa_step(ctx: Context, model: ModelBinding, i: int, sigma_i: float, sigma_next: float,
             regroup: bool = True) -> None:
    _check(ctx.ptr, load().hsa_step(ctx.ptr, ctypes.byref(model.weights), ctypes.byref(model.state),
                                    i, float(sigma_i), float(sigma_next), 1 if regroup else 0))


class StepCond:
    """The ctypes arrays of one iteration's conditioning (keeps them alive).

    mods: a list of L device fp32 [6, D] tensors (None entries allowed) or
    None; cross: a list of L hsa_cross_attn structs (see cross_attn) or None."""

    def __init__(self, mods=None, cross=None):
        self._mods = None if mods is None else (ctypes.c_void_p * max(len(mods), 1))(
            *[None if m is None else _p(m) for m in mods])
        self._cross = None if cross is None else (hsa_cross_attn * max(len(cross), 1))(*cross)
        self.struct = hsa_cond(
            ctypes.cast(self._mods, ctypes.POINTER(ctypes.c_void_p)) if mods is not None else None,
            ctypes.cast(self._cross, ctypes.POINTER(hsa_cross_attn)) if cross is not None else None)
        self._keep = (mods, cross)


def hsa_step_cond(ctx: Context, model: ModelBinding, cond: Optional[StepCond], i: int,
                  sigma_i: float, sigma_next: float, regroup: bool = True) -> None:
    _check(ctx.ptr, load().hsa_step_cond(
        ctx.ptr, ctypes.byref(model.weights), ctypes.byref(model.state),
        ctypes.byref(cond.struct) if cond is not None else None, i, float(sigma_i),
        float(sigma_next), 1 if regroup else 0))


class StepExt:
    """The L block extensions of one iteration (keeps them alive)."""

    def __init__(self, exts: Sequence[hsa_block_ext]):
        self.array = (hsa_block_ext * max(len(exts), 1))(*exts)
        self._keep = list(exts)
        self._checked_for = None


def hsa_step_ext(ctx: Context, model: ModelBinding, ext: Optional[StepExt], i: int,
                 sigma_i: float, sigma_next: float, regroup: bool = True) -> None:
    if ext is not None:
        if len(ext._keep) != ctx.cfg.L:
            raise ValueError(f"{len(ext._keep)} block extensions for {ctx.cfg.L} layers")
        if ctx is not ext._checked_for:  # once per context: the structs do not change
            for e in ext._keep:
                _check_ext(ctx, e)
            ext._checked_for = ctx
    _check(ctx.ptr, load().hsa_step_ext(
        ctx.ptr, ctypes.byref(model.weights), ctypes.byref(model.state),
        ext.array if ext is not None else None, i, float(sigma_i), float(sigma_next),
        1 if regroup else 0))


def hsa_select_groups_static(v_prev, v_cur, N: int, counts: Sequence[int], g, stream=None) -> None:
    """Group selection without a context or any device allocation (see include/hsa.h).

    Its scratch is one static device array of the library, sized for at most
    SELECT_STATIC_MAX_N tokens; concurrent calls on the GPU race on it.
    """
    K = len(counts)
    c = (ctypes.c_int * K)(*counts)
    st = load().hsa_select_groups_static(_p(v_prev), _p(v_cur), N, c, K, _p(g), _stream_ptr(stream))
    if st != 0:
        why = {8: f"N = {N} exceeds the static scratch limit of {SELECT_STATIC_MAX_N} tokens"}
        raise HsaError(st, why.get(st, "hsa_select_groups_static rejected its arguments"))
