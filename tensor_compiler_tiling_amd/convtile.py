"""ctypes binding of libconvtile.so (include/convtile.h).

Argument marshalling only: every computation runs in the library's HIP
kernels.  The functions named like the C entry points take device pointers
(ints) or torch tensors and return the C status; the short helpers
(``conv2d``, ``broadcast``, ``tune``, ``query``) allocate outputs with torch
and raise ``ConvTileError`` on a non-zero status.  There is no fallback: if
the library is missing, loading it raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import List, Optional, Tuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libconvtile.so")

CT_OK = 0
CT_ERR_INVALID_ARG = -1
CT_ERR_UNSUPPORTED = -2
CT_ERR_HIP = -3
CT_ERR_NO_MEMORY = -4
CT_ERR_IO = -5
CT_ERR_TUNE_FAILED = -6

CT_F32, CT_F16, CT_BF16, CT_E4M3 = 0, 1, 2, 3
# bytes of the no-allocation entry point's fixed scratch (partials and filter copy)
CT_NOALLOC_SCRATCH_BYTES = 16 << 20
CT_EPI_NONE, CT_EPI_BIAS, CT_EPI_EXP_BIAS_RSQRT = 0, 1, 2
CT_ACT_NONE, CT_ACT_RELU, CT_ACT_GELU, CT_ACT_GELU_TANH, CT_ACT_SILU = 0, 1, 2, 3, 4
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
CT_BC_EXP = 0
CT_BC_AUTO, CT_BC_CHANNEL, CT_BC_FLAT = 0, 1, 2
CT_CHAIN_MAX_OPS = 8
CHAIN_OPS = {"set": 0, "add": 1, "sub": 2, "mul": 3, "div": 4, "rsub": 5, "rdiv": 6, "exp": 7, "rsqrt": 8,
             "sqrt": 9}
CHAIN_SRCS = {"imm": 0, "x": 1, "c0": 2, "c1": 3, "a0": 4, "a1": 5, "a2": 6, "a3": 7}
CT_TRIAL_OK, CT_TRIAL_ILLEGAL, CT_TRIAL_RUNTIME, CT_TRIAL_TIMEOUT = 0, 1, 4, 6


class ct_tile_config(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int), ("split_k", ctypes.c_int), ("stages", ctypes.c_int),
                ("kc", ctypes.c_int), ("index", ctypes.c_longlong), ("us", ctypes.c_float),
                ("error_no", ctypes.c_int)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class ct_chain_op(ctypes.Structure):
    _fields_ = [("op", ctypes.c_int), ("src", ctypes.c_int), ("imm", ctypes.c_float)]


class ct_bcast_program(ctypes.Structure):
    _fields_ = [("n_ops", ctypes.c_int * 3), ("ops", (ct_chain_op * CT_CHAIN_MAX_OPS) * 3)]


class ct_linear_epilogue(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int), ("bias", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("ldg", ctypes.c_longlong), ("residual", ctypes.c_void_p), ("ldr", ctypes.c_longlong)]


class ct_kv_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("dtype", ctypes.c_int), ("pages", ctypes.c_int),
                ("heads", ctypes.c_int), ("page", ctypes.c_int), ("dim", ctypes.c_int),
                ("ld_page", ctypes.c_longlong), ("ld_head", ctypes.c_longlong), ("ld_token", ctypes.c_longlong),
                ("lds_page", ctypes.c_longlong), ("lds_head", ctypes.c_longlong), ("lds_token", ctypes.c_longlong)]


class ct_kv_batch(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int), ("sequences", ctypes.c_int), ("lens", ctypes.c_void_p),
                ("starts", ctypes.c_void_p), ("table", ctypes.c_void_p), ("ldt", ctypes.c_longlong),
                ("width", ctypes.c_int)]


class ct_kv_mask(ctypes.Structure):
    _fields_ = [("window", ctypes.c_int), ("sinks", ctypes.c_int), ("tree", ctypes.c_void_p),
                ("words", ctypes.c_int)]


class ct_tvm_config(ctypes.Structure):
    _fields_ = [("tile_f", ctypes.c_int * 4), ("tile_y", ctypes.c_int * 4), ("tile_x", ctypes.c_int * 4),
                ("tile_rc", ctypes.c_int * 3), ("tile_ry", ctypes.c_int * 3), ("tile_rx", ctypes.c_int * 3),
                ("auto_unroll_max_step", ctypes.c_int), ("unroll_explicit", ctypes.c_int)]

    def as_dict(self):
        return {f: (list(getattr(self, f)) if f.startswith("tile_") else getattr(self, f))
                for f, _ in self._fields_}

    @classmethod
    def from_dict(cls, d):
        c = cls()
        for f, _ in cls._fields_:
            if f.startswith("tile_"):
                arr = getattr(c, f)
                for i, v in enumerate(d[f]):
                    arr[i] = v
            else:
                setattr(c, f, d[f])
        return c


CT_TVM_LIMITS_PAGE = 0
CT_TVM_LIMITS_GFX950 = 1


class ct_variant_desc(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("dtype", ctypes.c_int), ("kind", ctypes.c_int),
                ("mfma_m", ctypes.c_int), ("mfma_n", ctypes.c_int), ("mfma_k", ctypes.c_int),
                ("waves_m", ctypes.c_int), ("waves_n", ctypes.c_int), ("waves_k", ctypes.c_int),
                ("reps_m", ctypes.c_int), ("reps_n", ctypes.c_int), ("tile_m", ctypes.c_int),
                ("tile_n", ctypes.c_int), ("kc_max", ctypes.c_int), ("threads", ctypes.c_int)]

    def as_dict(self):
        d = {f: getattr(self, f) for f, _ in self._fields_}
        d["name"] = self.name.decode()
        return d


class ct_tune_record(ctypes.Structure):
    _fields_ = [("cfg", ct_tile_config), ("costs_us", ctypes.c_float * 3), ("n_costs", ctypes.c_int),
                ("error_no", ctypes.c_int), ("all_cost_s", ctypes.c_double),
                ("timestamp", ctypes.c_double)]


class ConvTileError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        lib = _load()
        msg = lib.ct_last_error().decode(errors="replace")
        super().__init__(f"{where}: {lib.ct_status_string(status).decode()} ({status}): {msg}")


_I, _LL, _F, _P = ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_void_p
_SHAPE = [_I] * 11  # N, CI, H, W, CO, KH, KW, stride, pad, dtype, epilogue

_SIGS = {
    "ct_conv2d_nchw_fwd": (_I, [_P, _P, _P] + [_I] * 11 + [_P, _P, _F, _P]),
    "ct_conv2d_nchw_fwd_noalloc": (_I, [_P, _P, _P] + [_I] * 11 + [_P, _P, _F, _P]),
    "ct_conv2d_nchw_fwd_prepared": (_I, [_P, _P, _P] + [_I] * 11 + [_P, _P, _F, _P]),
    "ct_conv2d_filter_prepared_bytes": (_LL, [_I] * 5),
    "ct_conv2d_prepare_filter": (_I, [_P, _P] + [_I] * 5 + [_P]),
    "ct_conv2d_nchw_fwd_config": (_I, [_P, _P, _P] + [_I] * 11 +
                                  [_P, _P, _F, ctypes.POINTER(ct_tile_config), _P]),
    "ct_conv2d_nchw_direct": (_I, [_P, _P, _P] + [_I] * 11 + [_P, _P, _F, _P]),
    "ct_conv2d_space_size": (_LL, _SHAPE),
    "ct_conv2d_space_entity": (_I, _SHAPE + [_LL, ctypes.POINTER(ct_tile_config),
                                             ctypes.POINTER(_I)]),
    "ct_conv2d_tune": (_I, _SHAPE + [_I, _F, _P, ctypes.POINTER(ct_tile_config),
                                     ctypes.POINTER(ct_tune_record), _I, ctypes.POINTER(_I)]),
    "ct_conv2d_query": (_I, _SHAPE + [ctypes.POINTER(ct_tile_config), ctypes.POINTER(_I)]),
    "ct_conv2d_tune_order": (_I, _SHAPE + [_I, ctypes.POINTER(_LL), _I, ctypes.POINTER(_I)]),
    "ct_conv2d_tune_guided": (_I, _SHAPE + [_I, _I, ctypes.c_ulonglong, _F, _P, ctypes.POINTER(ct_tile_config),
                                            ctypes.POINTER(ct_tune_record), _I, ctypes.POINTER(_I)]),
    "ct_ridge_fit": (_I, [_P, _P, _I, _I, ctypes.c_double, _P]),
    "ct_guided_search_table": (_I, [_P, _P, _I, _I, _I, _I, _I, ctypes.c_ulonglong, ctypes.c_double, _P, _P]),
    "ct_gemm_fwd": (_I, [_P, _P, _P] + [_I] * 5 + [_P, _P, _F, _P]),
    "ct_gemm_tune": (_I, [_I] * 5 + [_I, _F, _P, ctypes.POINTER(ct_tile_config),
                                   ctypes.POINTER(ct_tune_record), _I, ctypes.POINTER(_I)]),
    "ct_gemm_query": (_I, [_I] * 5 + [ctypes.POINTER(ct_tile_config), ctypes.POINTER(_I)]),
    "ct_conv2d_nchw_depthwise": (_I, [_P, _P, _P] + [_I] * 10 + [_P, _P, _F, _P]),
    "ct_broadcast_chain": (_I, [ctypes.POINTER(ct_bcast_program)] + [_P] * 6 + [_I, _LL, _I, _LL, _I, _P]),
    "ct_rmsnorm_fwd": (_I, [_P, _LL, _P, _LL, _P, _P, _LL, _P, _LL, _P, _I, _I, _I, _I, _F, _P]),
    "ct_quantize_rows": (_I, [_P, _LL, _P, _LL, _P, _I, _I, _I, _P]),
    "ct_linear_fwd": (_I, [_P, _LL, _P, _LL, _P, _LL] + [_I] * 5 + [_P, _P, _LL, _P]),
    "ct_linear_q8_fwd": (_I, [_P, _LL, _P, _P, _LL, _P, _P, _LL] + [_I] * 4 + [_P, _P, _LL, _P]),
    "ct_linear_workspace_bytes": (_LL, [_I] * 4),
    "ct_kv_write": (_I, [_P, _P, _P, _LL, _LL, _P, _LL, _LL, _I, _P]),
    "ct_kv_read": (_I, [_P, _P, _P, _LL, _LL, _P, _LL, _LL, _I, _P]),
    "ct_kv_attention_fwd": (_I, [_P, _P, _P, _P, _LL, _LL, _P, _LL, _LL, _I, _I, _F, _LL, _P, _LL, _P]),
    "ct_kv_attention_workspace_bytes": (_LL, [_I] * 5 + [_LL, _I, _I, _I]),
    "ct_variant_count": (_I, []),
    "ct_variant_info": (_I, [_I, ctypes.POINTER(ct_variant_desc)]),
    "ct_split_count": (_LL, [_LL, _I]),
    "ct_split_entity": (_I, [_LL, _I, _LL, ctypes.POINTER(_LL)]),
    "ct_tvm_space_size": (_LL, [_I] * 9),
    "ct_tvm_space_entity": (_I, [_I] * 9 + [_LL, ctypes.POINTER(ct_tvm_config)]),
    "ct_tvm_space_index": (_LL, [_I] * 9 + [ctypes.POINTER(ct_tvm_config)]),
    "ct_tvm_config_check": (_I, [ctypes.POINTER(ct_tvm_config), _I, _I, ctypes.POINTER(_LL),
                                 ctypes.POINTER(_I)]),
    "ct_broadcast_nchw": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _I, _P]),
    "ct_cache_load": (_I, [ctypes.c_char_p]),
    "ct_cache_save": (_I, [ctypes.c_char_p]),
    "ct_cache_clear": (_I, []),
    "ct_cache_size": (_I, []),
    "ct_release": (_I, []),
    "ct_init": (_I, [_I]),
    "ct_plan_misses": (_LL, []),
    "ct_status_string": (ctypes.c_char_p, [_I]),
    "ct_last_error": (ctypes.c_char_p, []),
    "ct_version": (ctypes.c_char_p, []),
}

_lib = None


def _load():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run "
                               "`python -m tensor_compiler_tiling_amd.build` (no CPU fallback exists)")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def library():
    """The loaded ctypes library (raises if it is not built)."""
    return _load()


def exported_names() -> List[str]:
    return list(_SIGS)


# ---------------------------------------------------------------- marshal --
def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"expected a torch tensor or a device pointer, got {type(t)}")
    if not t.is_cuda:
        raise ValueError("tensor must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(s) -> Optional[int]:
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def dtype_code(torch_dtype) -> int:
    import torch
    m = {torch.float32: CT_F32, torch.float16: CT_F16, torch.bfloat16: CT_BF16}
    if torch_dtype not in m:
        raise ValueError(f"unsupported dtype {torch_dtype}")
    return m[torch_dtype]


def out_extent(inp: int, k: int, stride: int, pad: int) -> int:
    return (inp + 2 * pad - k) // stride + 1


# ------------------------------------------------- entry points (same names) --
def ct_conv2d_nchw_fwd(x, w, y, N, CI, H, W, CO, KH, KW, stride, pad, dtype, epilogue,
                       bias=None, var=None, eps=1e-5, stream=None) -> int:
    return _load().ct_conv2d_nchw_fwd(_ptr(x), _ptr(w), _ptr(y), N, CI, H, W, CO, KH, KW, stride,
                                      pad, dtype, epilogue, _ptr(bias), _ptr(var), eps,
                                      _stream(stream))


def ct_conv2d_nchw_fwd_noalloc(x, w, y, N, CI, H, W, CO, KH, KW, stride, pad, dtype, epilogue,
                               bias=None, var=None, eps=1e-5, stream=None) -> int:
    return _load().ct_conv2d_nchw_fwd_noalloc(_ptr(x), _ptr(w), _ptr(y), N, CI, H, W, CO, KH, KW, stride,
                                              pad, dtype, epilogue, _ptr(bias), _ptr(var), eps,
                                              _stream(stream))


def ct_conv2d_nchw_fwd_prepared(x, wp, y, N, CI, H, W, CO, KH, KW, stride, pad, dtype, epilogue,
                                bias=None, var=None, eps=1e-5, stream=None) -> int:
    return _load().ct_conv2d_nchw_fwd_prepared(_ptr(x), _ptr(wp), _ptr(y), N, CI, H, W, CO, KH, KW, stride,
                                               pad, dtype, epilogue, _ptr(bias), _ptr(var), eps,
                                               _stream(stream))


def ct_conv2d_filter_prepared_bytes(CO, CI, KH, KW, dtype) -> int:
    return _load().ct_conv2d_filter_prepared_bytes(CO, CI, KH, KW, dtype)


def ct_conv2d_prepare_filter(w, wp, CO, CI, KH, KW, dtype, stream=None) -> int:
    return _load().ct_conv2d_prepare_filter(_ptr(w), _ptr(wp), CO, CI, KH, KW, dtype, _stream(stream))


def prepare_filter(w, stream=None):
    """The prepared (regrouped) copy of a half-precision filter w [CO, CI, KH, KW]
    as a flat torch tensor of the same dtype."""
    import torch
    _on_gpu(w=w)
    CO, CI, KH, KW = w.shape
    dt = dtype_code(w.dtype)
    nbytes = ct_conv2d_filter_prepared_bytes(CO, CI, KH, KW, dt)
    check(nbytes if nbytes < 0 else 0, "prepare_filter")
    wp = torch.empty(nbytes // 2, dtype=w.dtype, device=w.device)
    check(ct_conv2d_prepare_filter(w, wp, CO, CI, KH, KW, dt, stream), "prepare_filter")
    return wp


def ct_conv2d_nchw_fwd_config(x, w, y, N, CI, H, W, CO, KH, KW, stride, pad, dtype, epilogue,
                              bias, var, eps, cfg: ct_tile_config, stream=None) -> int:
    return _load().ct_conv2d_nchw_fwd_config(_ptr(x), _ptr(w), _ptr(y), N, CI, H, W, CO, KH, KW,
                                             stride, pad, dtype, epilogue, _ptr(bias), _ptr(var),
                                             eps, ctypes.byref(cfg), _stream(stream))


def ct_conv2d_nchw_direct(x, w, y, N, CI, H, W, CO, KH, KW, stride, pad, dtype, epilogue,
                          bias=None, var=None, eps=1e-5, stream=None) -> int:
    return _load().ct_conv2d_nchw_direct(_ptr(x), _ptr(w), _ptr(y), N, CI, H, W, CO, KH, KW,
                                         stride, pad, dtype, epilogue, _ptr(bias), _ptr(var), eps,
                                         _stream(stream))


def ct_conv2d_space_size(N, CI, H, W, CO, KH, KW, stride, pad, dtype, epilogue) -> int:
    return _load().ct_conv2d_space_size(N, CI, H, W, CO, KH, KW, stride, pad, dtype, epilogue)


def ct_conv2d_space_entity(N, CI, H, W, CO, KH, KW, stride, pad, dtype, epilogue,
                           index) -> Tuple[int, ct_tile_config, int]:
    cfg = ct_tile_config()
    legal = _I(0)
    st = _load().ct_conv2d_space_entity(N, CI, H, W, CO, KH, KW, stride, pad, dtype, epilogue,
                                        index, ctypes.byref(cfg), ctypes.byref(legal))
    return st, cfg, legal.value


def ct_conv2d_tune(N, CI, H, W, CO, KH, KW, stride, pad, dtype, epilogue, max_trials=0,
                   min_repeat_ms=100.0, stream=None, max_records=4096):
    best = ct_tile_config()
    recs = (ct_tune_record * max(max_records, 1))()
    n = _I(0)
    st = _load().ct_conv2d_tune(N, CI, H, W, CO, KH, KW, stride, pad, dtype, epilogue, max_trials,
                                min_repeat_ms, _stream(stream), ctypes.byref(best), recs,
                                max_records, ctypes.byref(n))
    return st, best, [recs[i] for i in range(n.value)]


def ct_conv2d_query(N, CI, H, W, CO, KH, KW, stride, pad, dtype, epilogue):
    cfg = ct_tile_config()
    fc = _I(0)
    st = _load().ct_conv2d_query(N, CI, H, W, CO, KH, KW, stride, pad, dtype, epilogue,
                                 ctypes.byref(cfg), ctypes.byref(fc))
    return st, cfg, fc.value


def ct_gemm_fwd(A, B, C, M, N, K, dtype, epilogue, bias=None, var=None, eps=1e-5, stream=None) -> int:
    return _load().ct_gemm_fwd(_ptr(A), _ptr(B), _ptr(C), M, N, K, dtype, epilogue, _ptr(bias),
                               _ptr(var), eps, _stream(stream))


def ct_conv2d_nchw_depthwise(x, w, y, N, C, H, W, KH, KW, stride, pad, dtype, epilogue, bias=None,
                             var=None, eps=1e-5, stream=None) -> int:
    return _load().ct_conv2d_nchw_depthwise(_ptr(x), _ptr(w), _ptr(y), N, C, H, W, KH, KW, stride, pad,
                                            dtype, epilogue, _ptr(bias), _ptr(var), eps,
                                            _stream(stream))


def ct_broadcast_chain(prog, a0, a1, a2, a3, x, out, out_dtype, outer, P, inner, mode=CT_BC_AUTO,
                       stream=None) -> int:
    return _load().ct_broadcast_chain(ctypes.byref(prog), _ptr(a0), _ptr(a1), _ptr(a2), _ptr(a3), _ptr(x),
                                      _ptr(out), out_dtype, outer, P, inner, mode, _stream(stream))


def _row_ptr(t) -> Optional[int]:
    """The address of a matrix whose rows may lie apart (or a device pointer)."""
    if t is None or isinstance(t, int):
        return t
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"expected a torch tensor or a device pointer, got {type(t)}")
    if not t.is_cuda:
        raise ValueError("tensor must be on the GPU")
    if t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("the elements of a row must be contiguous")
    return t.data_ptr()


def _counts(**sizes) -> None:
    """ctypes keeps the low 32 bits of an int: counts that need more are refused
    here, before the library would answer for others."""
    for name, n in sizes.items():
        if not -(1 << 31) <= n < 1 << 31:
            raise ValueError(f"{name} = {n} does not fit 32 bits")


def ct_rmsnorm_fwd(x, ldx, residual, ldr, gain, h, ldh, y, ldy, scale, M, D, dtype, out_dtype, eps=1e-6,
                   stream=None) -> int:
    _counts(M=M, D=D)
    return _load().ct_rmsnorm_fwd(_row_ptr(x), ldx, _row_ptr(residual), ldr, _ptr(gain), _row_ptr(h), ldh,
                                  _row_ptr(y), ldy, _ptr(scale), M, D, dtype, out_dtype, eps, _stream(stream))


def ct_quantize_rows(x, ldx, q, ldq, scale, M, D, dtype, stream=None) -> int:
    _counts(M=M, D=D)
    return _load().ct_quantize_rows(_row_ptr(x), ldx, _row_ptr(q), ldq, _ptr(scale), M, D, dtype, _stream(stream))


def ct_linear_fwd(x, ldx, w, ldw, y, ldy, M, N, K, dtype, out_dtype, epi: Optional[ct_linear_epilogue] = None,
                  workspace=None, workspace_bytes=0, stream=None) -> int:
    _counts(M=M, N=N, K=K)
    return _load().ct_linear_fwd(_row_ptr(x), ldx, _row_ptr(w), ldw, _row_ptr(y), ldy, M, N, K, dtype, out_dtype,
                                 ctypes.addressof(epi) if epi is not None else None, _ptr(workspace),
                                 workspace_bytes, _stream(stream))


def ct_linear_q8_fwd(x, ldx, xs, w, ldw, ws, y, ldy, M, N, K, out_dtype, epi: Optional[ct_linear_epilogue] = None,
                     workspace=None, workspace_bytes=0, stream=None) -> int:
    _counts(M=M, N=N, K=K)
    return _load().ct_linear_q8_fwd(_row_ptr(x), ldx, _ptr(xs), _row_ptr(w), ldw, _ptr(ws), _row_ptr(y), ldy, M, N,
                                    K, out_dtype, ctypes.addressof(epi) if epi is not None else None,
                                    _ptr(workspace), workspace_bytes, _stream(stream))


# The structs of these are kept alive by the caller for the call; the counts in
# them are held to 32 bits by KVCache and the helpers.
def _struct(t):
    return ctypes.addressof(t) if isinstance(t, ctypes.Structure) else t


def ct_kv_write(cache, batch, k, k_token, k_head, v, v_token, v_head, dtype, stream=None) -> int:
    return _load().ct_kv_write(_struct(cache), _struct(batch), _row_ptr(k), k_token, k_head, _row_ptr(v), v_token,
                               v_head, dtype, _stream(stream))


def ct_kv_read(cache, batch, k, k_token, k_head, v, v_token, v_head, dtype, stream=None) -> int:
    return _load().ct_kv_read(_struct(cache), _struct(batch), _row_ptr(k), k_token, k_head, _row_ptr(v), v_token,
                              v_head, dtype, _stream(stream))


def ct_kv_attention_fwd(cache, batch, mask, q, q_token, q_head, y, y_token, y_head, heads, dtype, scale, max_len=0,
                        workspace=None, workspace_bytes=0, stream=None) -> int:
    _counts(heads=heads)
    return _load().ct_kv_attention_fwd(_struct(cache), _struct(batch), _struct(mask), _row_ptr(q), q_token, q_head,
                                       _row_ptr(y), y_token, y_head, heads, dtype, scale, max_len, _ptr(workspace),
                                       workspace_bytes, _stream(stream))


def ct_kv_attention_workspace_bytes(tokens, sequences, heads, kv_heads, dim, max_len=0, window=0, sinks=0,
                                    cache_dtype=CT_BF16) -> int:
    _counts(tokens=tokens, sequences=sequences, heads=heads, kv_heads=kv_heads, dim=dim, window=window, sinks=sinks)
    return _load().ct_kv_attention_workspace_bytes(tokens, sequences, heads, kv_heads, dim, max_len, window, sinks,
                                                   cache_dtype)


def ct_linear_workspace_bytes(M, N, K, dtype) -> int:
    _counts(M=M, N=N, K=K)
    return _load().ct_linear_workspace_bytes(M, N, K, dtype)


def ct_conv2d_tune_guided(N, CI, H, W, CO, KH, KW, stride, pad, dtype, epilogue, max_trials=64, batch=8,
                          seed=0, min_repeat_ms=100.0, stream=None, max_records=4096):
    best = ct_tile_config()
    recs = (ct_tune_record * max(max_records, 1))()
    n = _I(0)
    st = _load().ct_conv2d_tune_guided(N, CI, H, W, CO, KH, KW, stride, pad, dtype, epilogue, max_trials, batch,
                                       seed, min_repeat_ms, _stream(stream), ctypes.byref(best), recs, max_records,
                                       ctypes.byref(n))
    return st, best, [recs[i] for i in range(n.value)]


def ct_ridge_fit(X, y, lam=0.0):
    """numpy in, numpy out: (status, w)."""
    import numpy as np
    X = np.ascontiguousarray(X, dtype=np.float64)
    y = np.ascontiguousarray(y, dtype=np.float64)
    n, d = X.shape
    w = np.zeros(d, np.float64)
    st = _load().ct_ridge_fit(X.ctypes.data, y.ctypes.data, n, d, float(lam), w.ctypes.data)
    return st, w


def ct_guided_search_table(feats, costs, max_trials, batch, n_explore, seed=0, lam=1e-3):
    """numpy in: (status, order of the points the search would time)."""
    import numpy as np
    F = np.ascontiguousarray(feats, dtype=np.float64)
    c = np.ascontiguousarray(costs, dtype=np.float64)
    n, d = F.shape
    order = np.zeros(max(max_trials, 1), np.int32)
    cnt = _I(0)
    st = _load().ct_guided_search_table(F.ctypes.data, c.ctypes.data, n, d, max_trials, batch, n_explore, seed,
                                        float(lam), order.ctypes.data, ctypes.addressof(cnt))
    return st, order[:cnt.value].tolist()


def ct_gemm_tune(M, N, K, dtype, epilogue, max_trials=0, min_repeat_ms=100.0, stream=None,
                 max_records=4096):
    best = ct_tile_config()
    recs = (ct_tune_record * max(max_records, 1))()
    n = _I(0)
    st = _load().ct_gemm_tune(M, N, K, dtype, epilogue, max_trials, min_repeat_ms, _stream(stream),
                              ctypes.byref(best), recs, max_records, ctypes.byref(n))
    return st, best, [recs[i] for i in range(n.value)]


def ct_gemm_query(M, N, K, dtype, epilogue):
    cfg = ct_tile_config()
    fc = _I(0)
    st = _load().ct_gemm_query(M, N, K, dtype, epilogue, ctypes.byref(cfg), ctypes.byref(fc))
    return st, cfg, fc.value


def ct_variant_count() -> int:
    return _load().ct_variant_count()


def ct_variant_info(v: int):
    d = ct_variant_desc()
    st = _load().ct_variant_info(v, ctypes.byref(d))
    return st, d


def ct_split_count(n: int, k: int) -> int:
    return _load().ct_split_count(n, k)


def ct_split_entity(n: int, k: int, i: int):
    out = (_LL * k)()
    st = _load().ct_split_entity(n, k, i, out)
    return st, list(out)


def ct_tvm_space_size(N, CI, H, W, CO, KH, KW, stride, pad) -> int:
    return _load().ct_tvm_space_size(N, CI, H, W, CO, KH, KW, stride, pad)


def ct_tvm_space_entity(N, CI, H, W, CO, KH, KW, stride, pad, index):
    """(status, config dict) of flat index `index` of the template's space."""
    out = ct_tvm_config()
    st = _load().ct_tvm_space_entity(N, CI, H, W, CO, KH, KW, stride, pad, index, ctypes.byref(out))
    return st, out.as_dict()


def ct_tvm_space_index(N, CI, H, W, CO, KH, KW, stride, pad, cfg: dict) -> int:
    c = ct_tvm_config.from_dict(cfg)
    return _load().ct_tvm_space_index(N, CI, H, W, CO, KH, KW, stride, pad, ctypes.byref(c))


def ct_tvm_config_check(cfg: dict, stride: int, mode: int = CT_TVM_LIMITS_PAGE):
    """(fits 1/0 or status < 0, shared bytes, threads per block)."""
    c = ct_tvm_config.from_dict(cfg)
    nb, nt = _LL(0), _I(0)
    r = _load().ct_tvm_config_check(ctypes.byref(c), stride, mode, ctypes.byref(nb), ctypes.byref(nt))
    return r, nb.value, nt.value


def ct_broadcast_nchw(var, out, N, C, H, W, out_dtype, op=CT_BC_EXP, mode=CT_BC_AUTO,
                      stream=None) -> int:
    return _load().ct_broadcast_nchw(_ptr(var), _ptr(out), N, C, H, W, out_dtype, op, mode,
                                     _stream(stream))


def ct_cache_load(path: str) -> int:
    return _load().ct_cache_load(path.encode())


def ct_cache_save(path: str) -> int:
    return _load().ct_cache_save(path.encode())


def ct_cache_clear() -> int:
    return _load().ct_cache_clear()


def ct_cache_size() -> int:
    return _load().ct_cache_size()


def ct_release() -> int:
    return _load().ct_release()


def ct_status_string(st: int) -> str:
    return _load().ct_status_string(st).decode()


def ct_last_error() -> str:
    return _load().ct_last_error().decode(errors="replace")


def ct_init(device: int = 0) -> int:
    return _load().ct_init(device)


def ct_plan_misses() -> int:
    return _load().ct_plan_misses()


def ct_conv2d_tune_order(N, CI, H, W, CO, KH, KW, stride, pad, dtype, epilogue, max_trials=0):
    """(status, [flat indices]) the exhaustive search would time, in order,
    skipping points already in the CT_CACHE_PATH log."""
    n = _I(0)
    st = _load().ct_conv2d_tune_order(N, CI, H, W, CO, KH, KW, stride, pad, dtype, epilogue, max_trials,
                                      None, 0, ctypes.byref(n))
    if st != 0:
        return st, []
    buf = (_LL * max(1, n.value))()
    st = _load().ct_conv2d_tune_order(N, CI, H, W, CO, KH, KW, stride, pad, dtype, epilogue, max_trials,
                                      buf, n.value, ctypes.byref(n))
    return st, list(buf[:n.value])


def ct_version() -> str:
    return _load().ct_version().decode()


def check(status: int, where: str = "convtile") -> None:
    if status != CT_OK:
        raise ConvTileError(status, where)


# ------------------------------------------------------------ helpers --------
def variants() -> List[dict]:
    out = []
    for v in range(ct_variant_count()):
        st, d = ct_variant_info(v)
        check(st, "ct_variant_info")
        out.append(dict(d.as_dict(), id=v))
    return out


def variant_id(name: str) -> int:
    for d in variants():
        if d["name"] == name:
            return d["id"]
    raise KeyError(name)


def _on_gpu(**tensors) -> None:
    """The C ABI takes raw device pointers: every tensor handed to it must live
    on a GPU and be contiguous (None is skipped)."""
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def conv2d(x, w, stride: int = 1, pad: int = 0, epilogue: int = CT_EPI_NONE, bias=None, var=None,
           eps: float = 1e-5, config: Optional[ct_tile_config] = None, out=None, stream=None,
           direct: bool = False):
    """y = conv2d_nchw(x, w) (+ epilogue), fp32 output allocated with torch."""
    import torch
    _on_gpu(x=x, w=w, bias=bias, var=var, out=out)
    N, CI, H, W = x.shape
    CO, CI2, KH, KW = w.shape
    if CI2 != CI or w.dtype != x.dtype:
        raise ValueError("x and w disagree in channels or dtype")
    OH, OW = out_extent(H, KH, stride, pad), out_extent(W, KW, stride, pad)
    y = out if out is not None else torch.empty((N, CO, OH, OW), dtype=torch.float32,
                                                device=x.device)
    dt = dtype_code(x.dtype)
    if direct:
        st = ct_conv2d_nchw_direct(x, w, y, N, CI, H, W, CO, KH, KW, stride, pad, dt, epilogue,
                                   bias, var, eps, stream)
    elif config is not None:
        st = ct_conv2d_nchw_fwd_config(x, w, y, N, CI, H, W, CO, KH, KW, stride, pad, dt,
                                       epilogue, bias, var, eps, config, stream)
    else:
        st = ct_conv2d_nchw_fwd(x, w, y, N, CI, H, W, CO, KH, KW, stride, pad, dt, epilogue, bias,
                                var, eps, stream)
    check(st, "conv2d")
    return y


def conv2d_prepared(x, wp, filter_shape, stride: int = 1, pad: int = 0, epilogue: int = CT_EPI_NONE,
                    bias=None, var=None, eps: float = 1e-5, out=None, stream=None):
    """conv2d with a half-precision filter already prepared by prepare_filter;
    filter_shape = (CO, CI, KH, KW) of the original filter."""
    import torch
    _on_gpu(x=x, wp=wp, bias=bias, var=var, out=out)
    N, CI, H, W = x.shape
    CO, CI2, KH, KW = filter_shape
    if CI2 != CI or wp.dtype != x.dtype:
        raise ValueError("x and the prepared filter disagree in channels or dtype")
    OH, OW = out_extent(H, KH, stride, pad), out_extent(W, KW, stride, pad)
    y = out if out is not None else torch.empty((N, CO, OH, OW), dtype=torch.float32, device=x.device)
    st = ct_conv2d_nchw_fwd_prepared(x, wp, y, N, CI, H, W, CO, KH, KW, stride, pad, dtype_code(x.dtype),
                                     epilogue, bias, var, eps, stream)
    check(st, "conv2d_prepared")
    return y


def gemm(A, B, epilogue: int = CT_EPI_NONE, bias=None, var=None, eps: float = 1e-5, out=None,
         stream=None):
    """C = A @ B (+ per-row epilogue), fp32 output allocated with torch: A [M, K], B [K, N],
    same dtype, contiguous."""
    import torch
    _on_gpu(A=A, B=B, bias=bias, var=var, out=out)
    M, K = A.shape
    K2, N = B.shape
    if K2 != K or A.dtype != B.dtype:
        raise ValueError("A and B disagree in the inner dimension or dtype")
    C = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=A.device)
    check(ct_gemm_fwd(A, B, C, M, N, K, dtype_code(A.dtype), epilogue, bias, var, eps, stream), "gemm")
    return C


def conv2d_depthwise(x, w, stride: int = 1, pad: int = 0, epilogue: int = CT_EPI_NONE, bias=None,
                     var=None, eps: float = 1e-5, out=None, stream=None):
    """Depthwise y[n][c] = conv2d(x[n][c], w[c][0]) (+ epilogue), fp32 output allocated with
    torch: x [N, C, H, W], w [C, 1, KH, KW], same dtype, contiguous."""
    import torch
    _on_gpu(x=x, w=w, bias=bias, var=var, out=out)
    N, C, H, W = x.shape
    C2, one, KH, KW = w.shape
    if C2 != C or one != 1 or w.dtype != x.dtype:
        raise ValueError("w must be [C, 1, KH, KW] of x's channels and dtype")
    OH, OW = out_extent(H, KH, stride, pad), out_extent(W, KW, stride, pad)
    y = out if out is not None else torch.empty((N, C, OH, OW), dtype=torch.float32,
                                                device=x.device)
    st = ct_conv2d_nchw_depthwise(x, w, y, N, C, H, W, KH, KW, stride, pad, dtype_code(x.dtype),
                                  epilogue, bias, var, eps, stream)
    check(st, "conv2d_depthwise")
    return y


# ---- transformer-block rows: matrices whose rows may lie apart -------------
# Forward only, like everything here: results carry no autograd history.
# The smallest calls take a few microseconds on the device, less than a careless
# wrapper takes on the host: what these helpers need of torch is looked up once,
# and a well-formed argument passes its checks in one comparison.
class _TorchSide:
    def __init__(self):
        import torch
        self.empty, self.Tensor = torch.empty_strided, torch.Tensor  # the form that parses fastest
        self.f32, self.bf16, self.e4m3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
        self.uint8, self.i32, self.i64 = torch.uint8, torch.int32, torch.int64
        self.codes = {torch.float32: CT_F32, torch.float16: CT_F16, torch.bfloat16: CT_BF16}
        self.current_device = torch.cuda.current_device
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.stream = raw or (lambda index: torch.cuda.current_stream(index).cuda_stream)


_torch_side: Optional[_TorchSide] = None


def _side() -> _TorchSide:
    global _torch_side
    if _torch_side is None:
        _torch_side = _TorchSide()
    return _torch_side


def _refuse_matrix(name: str, t, index: int, dtype, M, D):
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    if index < 0 or t.get_device() != index:
        raise ValueError(f"{name} must be a GPU tensor on the device of the others")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != (M, D):
        raise ValueError(f"{name} must be {[M, D]}, got {list(t.shape)}")
    if D > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    raise ValueError(f"{name}: rows must not overlap")


def _matrix(name: str, t, index: int, dtype, M: int, D: int) -> int:
    """Check a matrix argument; the distance between its rows, in elements."""
    if t.get_device() == index and t.dtype is dtype and t.shape == (M, D):
        ld, step = t.stride()
        if step == 1 or D <= 1:
            if M <= 1:
                return D  # a single row has no stride to speak of
            if ld >= D:
                return ld
    return _refuse_matrix(name, t, index, dtype, M, D)


def _vector(name: str, t, index: int, n: int) -> int:
    """Check an fp32 vector argument; its address."""
    if t.get_device() != index:
        raise ValueError(f"{name} must be a GPU tensor on the device of the others")
    if t.dtype is not _side().f32 or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous fp32 values")
    return t.data_ptr()


def _first(name: str, t):
    """Check a call's first matrix: (device index, rows, columns, row distance)."""
    index, shape = t.get_device(), t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must have two dimensions")
    M, D = shape
    if (M | D) >> 31:
        raise ValueError(f"{name}: {M} rows of {D} do not fit 32 bits")
    if index < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    ld, step = t.stride()
    if M <= 1:
        ld = D  # a single row has no stride to speak of
    if (step != 1 and D > 1) or ld < D:
        _refuse_matrix(name, t, index, t.dtype, M, D)
    return index, M, D, ld


def _code(dtype) -> int:
    code = _side().codes.get(dtype)
    return dtype_code(dtype) if code is None else code


def _elsewhere(device, stream):
    """A context that makes `device` current and, with an explicit stream, has
    torch allocate outputs and workspace for that stream."""
    import torch
    if stream is None:
        return torch.cuda.device(device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError("the stream belongs to another device than the tensors")
    return torch.cuda.stream(stream)


def rmsnorm(x, gain=None, residual=None, eps: float = 1e-6, out_dtype=None, h=True, out=None, scale=None,
            stream=None):
    """RMS norm of the rows of x + residual: (y, scale, h).

    y = s * rsqrt(mean(s^2) + eps) * gain, s = x + residual in fp32; y has
    out_dtype (x's by default), torch.float8_e4m3fn giving 8-bit rows with
    their scales (None otherwise).  h is s rounded to x's type (the new
    residual stream; None without a residual or with h=False; h may name the
    tensor to write, x and residual among them).  x, residual, h and out are
    [M, D] with contiguous rows; gain is fp32 [D]."""
    T = _side()
    index, M, D, ldx = _first("x", x)
    device = x.device
    if stream is not None or index != T.current_device():
        with _elsewhere(device, stream):
            return rmsnorm(x, gain, residual, eps, out_dtype, h, out, scale)
    xt = x.dtype
    dtype = _code(xt)
    gp = rp = hp = sp = None
    ldr = ldh = 0
    if gain is not None:
        gp = _vector("gain", gain, index, D)
    if out_dtype is None:
        out_dtype = xt if out is None else out.dtype
    q8 = out_dtype is T.e4m3
    code = CT_E4M3 if q8 else _code(out_dtype)
    if residual is not None:
        ldr = _matrix("residual", residual, index, xt, M, D)
        rp = residual.data_ptr()
        if h is True:
            h, ldh = T.empty((M, D), (D, 1), dtype=xt, device=device), D
        elif h is not False and h is not None:
            ldh = _matrix("h", h, index, xt, M, D)
        else:
            h = None
        hp = None if h is None else h.data_ptr()
    elif isinstance(h, T.Tensor):
        raise ValueError("h is the sum with a residual, and there is none")
    else:
        h = None
    if out is None:
        out, ldy = T.empty((M, D), (D, 1), dtype=out_dtype, device=device), D
    else:
        ldy = _matrix("out", out, index, out_dtype, M, D)
    if q8:
        if scale is None:
            scale = T.empty((M,), (1,), dtype=T.f32, device=device)
            sp = scale.data_ptr()
        else:
            sp = _vector("scale", scale, index, M)
    elif scale is not None:
        raise ValueError("scale belongs to 8-bit output")
    st = _load().ct_rmsnorm_fwd(x.data_ptr(), ldx, rp, ldr, gp, hp, ldh, out.data_ptr(), ldy, sp, M, D, dtype, code,
                                eps, T.stream(index))
    if st:
        check(st, "rmsnorm")
    return out, scale, h


def quantize_rows(x, out=None, scale=None, stream=None):
    """The rows of x [M, D] in 8 bits: (q float8_e4m3fn [M, D], scale fp32 [M]),
    x ~ scale[:, None] * q."""
    T = _side()
    index, M, D, ldx = _first("x", x)
    device = x.device
    if stream is not None or index != T.current_device():
        with _elsewhere(device, stream):
            return quantize_rows(x, out, scale)
    dtype = _code(x.dtype)
    if out is None:
        out, ldq = T.empty((M, D), (D, 1), dtype=T.e4m3, device=device), D
    else:
        ldq = _matrix("out", out, index, T.e4m3, M, D)
    if scale is None:
        scale = T.empty((M,), (1,), dtype=T.f32, device=device)
        sp = scale.data_ptr()
    else:
        sp = _vector("scale", scale, index, M)
    st = _load().ct_quantize_rows(x.data_ptr(), ldx, out.data_ptr(), ldq, sp, M, D, dtype, T.stream(index))
    if st:
        check(st, "quantize_rows")
    return out, scale


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(M: int, N: int, K: int, dtype: int) -> int:
    return max(0, _load().ct_linear_workspace_bytes(M, N, K, dtype))


def _product(x, xs, w, ws, bias, act, gate, residual, out_dtype, out, stream):
    T = _side()
    index, M, K, ldx = _first("x", x)
    device = x.device
    if stream is not None or index != T.current_device():
        with _elsewhere(device, stream):
            return _product(x, xs, w, ws, bias, act, gate, residual, out_dtype, out, None)
    N, K2 = w.shape if w.dim() == 2 else (0, 0)
    if K != K2:
        raise ValueError(f"x has rows of {K} and w of {K2}")
    if N >> 31:
        raise ValueError(f"w: {N} rows do not fit 32 bits")
    xt = x.dtype
    if xs is None:
        dtype = _code(xt)
    else:
        dtype = CT_E4M3
        xsp, wsp = _vector("xs", xs, index, M), _vector("ws", ws, index, N)
        xt = T.e4m3
    if x.dtype is not xt:
        raise ValueError(f"x must be {xt}, got {x.dtype}")
    ldw = _matrix("w", w, index, xt, N, K)
    a = ACTIVATIONS.get(act)
    if a is None:
        raise ValueError(f"unknown activation {act!r}: one of {', '.join(ACTIVATIONS)}")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else xt if xs is None else T.bf16
    code = _code(out_dtype)
    ep = None
    if a or bias is not None or gate is not None or residual is not None:
        bp = gp = rp = None
        ldg = ldr = 0
        if bias is not None:
            bp = _vector("bias", bias, index, N)
        if gate is not None:
            ldg = _matrix("gate", gate, index, out_dtype, M, N)
            gp = gate.data_ptr()
        if residual is not None:
            ldr = _matrix("residual", residual, index, out_dtype, M, N)
            rp = residual.data_ptr()
        epi = ct_linear_epilogue(a, bp, gp, ldg, rp, ldr)
        ep = ctypes.addressof(epi)
    if out is None:
        out, ldy = T.empty((M, N), (N, 1), dtype=out_dtype, device=device), N
    else:
        ldy = _matrix("out", out, index, out_dtype, M, N)
    need = _workspace_bytes(M, N, K, dtype)
    space = sp = None
    if need:
        space = T.empty((need,), (1,), dtype=T.uint8, device=device)
        sp = space.data_ptr()
    if xs is None:
        st = _load().ct_linear_fwd(x.data_ptr(), ldx, w.data_ptr(), ldw, out.data_ptr(), ldy, M, N, K, dtype, code, ep,
                                   sp, need, T.stream(index))
    else:
        st = _load().ct_linear_q8_fwd(x.data_ptr(), ldx, xsp, w.data_ptr(), ldw, wsp, out.data_ptr(), ldy, M, N, K,
                                      code, ep, sp, need, T.stream(index))
    if st:
        check(st, "linear" if xs is None else "linear_q8")
    return out


def linear(x, w, bias=None, act: str = "none", gate=None, residual=None, out_dtype=None, out=None, stream=None):
    """y = act(x @ w.T + bias) * gate + residual, rounded once.

    x [M, K] and w [N, K] of one type (fp32, fp16, bf16), rows contiguous; bias
    fp32 [N]; gate and residual [M, N] of y's type (out_dtype, x's by
    default); act one of ACTIVATIONS.  out may be gate or residual itself."""
    return _product(x, None, w, None, bias, act, gate, residual, out_dtype, out, stream)


def linear_q8(xq, xs, wq, ws, bias=None, act: str = "none", gate=None, residual=None, out_dtype=None, out=None,
              stream=None):
    """linear on 8-bit rows (float8_e4m3fn) with their fp32 scales xs [M] and
    ws [N]; y has out_dtype (bf16 by default)."""
    if xs is None or ws is None:
        raise ValueError("8-bit rows have scales")
    return _product(xq, xs, wq, ws, bias, act, gate, residual, out_dtype, out, stream)


# ---- key-value cache and attention: a transformer block between its projections
def _same_layout(a, b) -> bool:
    """One distance in every axis that has one."""
    return all(n <= 1 or x == y for n, x, y in zip(a.shape, a.stride(), b.stride()))


class KVCache:
    """A pool of pages for keys and values, k and v [pages, heads, page, dim].

    float16 and bfloat16 tensors hold values, torch.float8_e4m3fn ones codes
    with fp32 scales k_scale and v_scale [pages, heads, page] (powers of two:
    a row stands for scale * code).  Any order of the axes in memory will do
    (views of [pages, page, heads, dim], say), the same for k and v; rows are
    contiguous, 16-byte aligned, dim a multiple of 16 up to 256.  The tensors are
    the caller's: their contents may be copied, moved or cleared between calls."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "index", "device", "dtype", "pages", "heads", "page", "dim", "_c", "_at")

    def __init__(self, k, v, k_scale=None, v_scale=None):
        T = _side()
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or not _same_layout(k, v):
            raise ValueError("k and v must be [pages, heads, page, dim] of one shape, type and layout")
        q8 = k.dtype is T.e4m3
        if not q8 and (k.dtype is T.f32 or k.dtype not in T.codes):
            raise ValueError(f"a cache of {k.dtype}: float16, bfloat16 or float8_e4m3fn")
        if (k_scale is None) is q8 or (v_scale is None) is q8:
            raise ValueError("8-bit rows have scales, and others have none")
        self.index = k.get_device()
        if self.index < 0 or v.get_device() != self.index:
            raise ValueError("k and v must be GPU tensors on one device")
        if any(n >> 31 for n in k.shape):
            raise ValueError(f"{list(k.shape)} does not fit 32 bits")
        if k.shape[3] > 1 and k.stride(3) != 1:
            raise ValueError("the elements of a row must be contiguous")
        st = (0, 0, 0)
        if q8:
            for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
                if s.get_device() != self.index or s.dtype is not T.f32 or s.shape != k.shape[:3]:
                    raise ValueError(f"{name} must be fp32 {list(k.shape[:3])} on the device of k")
            st = k_scale.stride()
            if not _same_layout(k_scale, v_scale):
                raise ValueError("k_scale and v_scale must have one layout")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device, self.dtype = k.device, k.dtype
        self.pages, self.heads, self.page, self.dim = k.shape
        self._c = ct_kv_cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if q8 else None,
                              v_scale.data_ptr() if q8 else None, CT_E4M3 if q8 else T.codes[k.dtype], self.pages,
                              self.heads, self.page, self.dim, *k.stride()[:3], *st)
        self._at = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, pages: int, heads: int, page: int, dim: int, dtype=None, device="cuda"):
        """A cache of `pages` pages, uninitialised (bfloat16 by default)."""
        import torch
        dtype = dtype or torch.bfloat16
        k, v = (torch.empty((pages, heads, page, dim), dtype=dtype, device=device) for _ in range(2))
        if dtype != torch.float8_e4m3fn:
            return cls(k, v)
        return cls(k, v, *(torch.empty((pages, heads, page), dtype=torch.float32, device=device) for _ in range(2)))


def _integers(name: str, t, index: int, n: int) -> int:
    if t.get_device() != index:
        raise ValueError(f"{name} must be a GPU tensor on the device of the cache")
    if t.dtype is not _side().i32 or t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be {n} contiguous int32 values")
    return t.data_ptr()


def _batch(cache: KVCache, tokens: int, lens, starts, table) -> ct_kv_batch:
    index = cache.index
    if lens.dim() != 1:
        raise ValueError("lens must have one dimension")
    sequences = lens.shape[0]
    if (tokens | sequences) >> 31:
        raise ValueError(f"{tokens} tokens of {sequences} sequences do not fit 32 bits")
    sp = tp = None
    ldt = width = 0
    if starts is not None:
        sp = _integers("starts", starts, index, sequences + 1)
    if table is not None:
        if table.get_device() != index:
            raise ValueError("table must be a GPU tensor on the device of the cache")
        if table.dtype is not _side().i32 or table.dim() != 2 or table.shape[0] != sequences:
            raise ValueError(f"table must be int32 [{sequences}, columns]")
        width = table.shape[1]
        ldt, step = table.stride()
        if width >> 31 or (width > 1 and step != 1):
            raise ValueError("the elements of a table's row must be contiguous, fewer than 2^31")
        tp = table.data_ptr()
    return ct_kv_batch(tokens, sequences, _integers("lens", lens, index, sequences), sp, tp, ldt, width)


def _heads(name: str, t, index: int, dtype, shape):
    """Check [tokens, heads, dim] rows; the distances between tokens and heads."""
    if t.get_device() != index:
        raise ValueError(f"{name} must be a GPU tensor on the device of the cache")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    token, head, step = t.stride()
    if step != 1 and shape[2] > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return token, head


def kv_write(cache: KVCache, k, v, lens, table=None, starts=None, stream=None) -> None:
    """New tokens' k and v [tokens, heads, dim] into the cache (fp32, fp16 or
    bf16; slices of a fused projection's rows will do).

    lens int32 [sequences] counts each sequence's places in use with the new
    tokens, which are the last; starts int32 [sequences + 1] says which rows are
    whose (None: equally many each); table int32 [sequences, columns] names the
    pages (None: sequence b has page b).  All three are read on the device."""
    T = _side()
    index = cache.index
    if k.dim() != 3:
        raise ValueError("k must be [tokens, heads, dim]")
    if stream is not None or index != T.current_device():
        with _elsewhere(cache.device, stream):
            return kv_write(cache, k, v, lens, table, starts)
    shape = (k.shape[0], cache.heads, cache.dim)
    kt, kh = _heads("k", k, index, k.dtype, shape)
    vt, vh = _heads("v", v, index, k.dtype, shape)
    b = _batch(cache, shape[0], lens, starts, table)
    st = _load().ct_kv_write(cache._at, ctypes.addressof(b), k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, _code(k.dtype),
                             T.stream(index))
    if st:
        check(st, "kv_write")


def kv_read(cache: KVCache, tokens: int, lens, table=None, starts=None, dtype=None, k=None, v=None, stream=None):
    """The last tokens of every sequence out of the cache: (k, v), each
    [tokens, heads, dim] of dtype (by default the cache's, or bf16 from 8 bits).
    tokens counts them all; lens, table and starts as for kv_write.  Rows of
    tokens that belong to no sequence are left as they are (k and v may name
    the tensors to write)."""
    T = _side()
    index = cache.index
    if stream is not None or index != T.current_device():
        with _elsewhere(cache.device, stream):
            return kv_read(cache, tokens, lens, table, starts, dtype, k, v)
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    if dtype is None:
        dtype = k.dtype if k is not None else v.dtype if v is not None else T.bf16 if cache.dtype is T.e4m3 else cache.dtype
    shape = (tokens, cache.heads, cache.dim)
    b = _batch(cache, tokens, lens, starts, table)
    step = (cache.heads * cache.dim, cache.dim, 1)
    if k is None:
        k = T.empty(shape, step, dtype=dtype, device=cache.device)
    if v is None:
        v = T.empty(shape, step, dtype=dtype, device=cache.device)
    kt, kh = _heads("k", k, index, dtype, shape)
    vt, vh = _heads("v", v, index, dtype, shape)
    st = _load().ct_kv_read(cache._at, ctypes.addressof(b), k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, _code(dtype),
                            T.stream(index))
    if st:
        check(st, "kv_read")
    return k, v


@functools.lru_cache(maxsize=4096)
def _attention_bytes(*sizes) -> int:
    return max(0, _load().ct_kv_attention_workspace_bytes(*sizes))


def kv_attention(q, cache: KVCache, lens, table=None, starts=None, max_len=None, window: int = 0, sinks: int = 0,
                 tree=None, scale=None, out=None, stream=None):
    """Attention of new tokens q [tokens, heads, dim] (fp16 or bf16) over the
    cache, which holds their keys and values already: y like q.

    heads is a multiple of the cache's, whose heads groups of neighbours share.
    lens, table and starts as for kv_write.  Each token sees the places up to its
    own; with a window only the last `window` of them and the first `sinks`.
    With a tree, int64 [tokens] or [tokens, words], the new tokens are drafted
    nodes: node i sees the context before them and node j if bit j of its row is
    set, its own included.  max_len, the longest of lens where the program
    knows, guides how the work is divided (the table's reach by default); scale is
    dim ** -0.5 by default.  A token that sees nothing gives zeros; rows of tokens
    that belong to no sequence are left as they are (out may name the tensor to
    write, in a new one they hold what memory held)."""
    T = _side()
    index = cache.index
    if q.dim() != 3:
        raise ValueError("q must be [tokens, heads, dim]")
    if stream is not None or index != T.current_device():
        with _elsewhere(cache.device, stream):
            return kv_attention(q, cache, lens, table, starts, max_len, window, sinks, tree, scale, out)
    shape = q.shape
    tokens, heads, dim = shape
    if dim != cache.dim:
        raise ValueError(f"q has rows of {dim} and the cache of {cache.dim}")
    if heads >> 31:
        raise ValueError(f"{heads} heads do not fit 32 bits")
    dtype = q.dtype
    qt, qh = _heads("q", q, index, dtype, shape)
    b = _batch(cache, tokens, lens, starts, table)
    words, tp = 0, None
    if tree is not None:
        if tree.get_device() != index:
            raise ValueError("tree must be a GPU tensor on the device of the cache")
        if tree.dtype is not T.i64 or tree.dim() not in (1, 2) or tree.shape[0] != tokens or not tree.is_contiguous():
            raise ValueError(f"tree must be contiguous int64 [{tokens}] or [{tokens}, words]")
        words = 1 if tree.dim() == 1 else tree.shape[1]
        if words >> 31:
            raise ValueError(f"{words} words do not fit 32 bits")
        tp = tree.data_ptr()
    if not (0 <= window < 1 << 31 and 0 <= sinks < 1 << 31):
        raise ValueError("window and sinks must be counts of 31 bits")
    if max_len is not None and max_len < 0:
        raise ValueError("max_len must not be negative")
    mask = None
    if window or sinks or tp is not None:
        keep = ct_kv_mask(window, sinks, tp, words)
        mask = ctypes.addressof(keep)
    if out is None:
        out = T.empty(shape, (heads * dim, dim, 1), dtype=dtype, device=cache.device)
    yt, yh = _heads("out", out, index, dtype, shape)
    reach = (b.width if table is not None else 1) * cache.page
    longest = reach if max_len is None else max(1, min(max_len, reach))
    need = _attention_bytes(tokens, b.sequences, heads, cache.heads, dim, longest, window, sinks, cache._c.dtype)
    sp = None
    if need:
        space = T.empty((need,), (1,), dtype=T.uint8, device=cache.device)
        sp = space.data_ptr()
    st = _load().ct_kv_attention_fwd(cache._at, ctypes.addressof(b), mask, q.data_ptr(), qt, qh, out.data_ptr(), yt, yh,
                                     heads, _code(dtype), dim ** -0.5 if scale is None else scale, longest, sp, need,
                                     T.stream(index))
    if st:
        check(st, "kv_attention")
    return out


def broadcast(var, N: int, H: int, W: int, out_dtype=None, mode: int = CT_BC_AUTO, out=None,
              stream=None):
    """[1,C,1,1] -> [N,C,H,W] of exp(var[c])."""
    import torch
    _on_gpu(var=var, out=out)
    out_dtype = out_dtype or torch.float16
    C = var.numel()
    o = out if out is not None else torch.empty((N, C, H, W), dtype=out_dtype, device=var.device)
    st = ct_broadcast_nchw(var, o, N, C, H, W, dtype_code(o.dtype), CT_BC_EXP, mode, stream)
    check(st, "broadcast")
    return o


def make_program(c0=(), c1=(), v=()) -> ct_bcast_program:
    """A broadcast program from three step lists.  A step is (op,), (op, src)
    or (op, "imm", value) / (op, value): op a CHAIN_OPS name, src a
    CHAIN_SRCS name, a bare number meaning an immediate."""
    prog = ct_bcast_program()
    for c, steps in enumerate((c0, c1, v)):
        steps = list(steps)
        if len(steps) > CT_CHAIN_MAX_OPS:
            raise ValueError(f"chain {c} has {len(steps)} steps (at most {CT_CHAIN_MAX_OPS})")
        prog.n_ops[c] = len(steps)
        for k, st in enumerate(steps):
            op, rest = st[0], st[1:]
            src, imm = "imm", 0.0
            if len(rest) == 1:
                if isinstance(rest[0], str):
                    src = rest[0]
                else:
                    imm = float(rest[0])
            elif len(rest) == 2:
                src, imm = rest[0], float(rest[1])
            prog.ops[c][k].op = CHAIN_OPS[op]
            prog.ops[c][k].src = CHAIN_SRCS[src]
            prog.ops[c][k].imm = imm
    return prog


def broadcast_chain(prog: ct_bcast_program, outer: int, P: int, inner: int, arrays=(), x=None,
                    out_dtype=None, mode: int = CT_BC_AUTO, out=None, stream=None):
    """out[o][p][i] = the program's value ([outer][P][inner], torch-allocated
    unless `out` is given); arrays: up to four per-channel fp32 tensors of P
    floats; x: the producer's fp32 tensor of the output's size, or None."""
    import torch
    arrays = list(arrays) + [None] * (4 - len(arrays))
    _on_gpu(a0=arrays[0], a1=arrays[1], a2=arrays[2], a3=arrays[3], x=x, out=out)
    dev = next((t.device for t in arrays + [x, out] if t is not None), None)
    if dev is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    if out is None:
        out = torch.empty((outer, P, inner), dtype=out_dtype or torch.float32, device=dev)
    st = ct_broadcast_chain(prog, arrays[0], arrays[1], arrays[2], arrays[3], x, out,
                            dtype_code(out.dtype), outer, P, inner, mode, stream)
    check(st, "broadcast_chain")
    return out


def make_config(variant, split_k: int, stages: int, kc: int) -> ct_tile_config:
    c = ct_tile_config()
    c.variant = variant if isinstance(variant, int) else variant_id(variant)
    c.split_k, c.stages, c.kc, c.index = split_k, stages, kc, -1
    return c
