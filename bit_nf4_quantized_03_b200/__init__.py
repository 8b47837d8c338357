"""Python binding of libqlora (NF4 + double-quant QLoRA linear layer, B200).

Argument marshalling only: every function below forwards to the C entry point
of the same name in libqlora.so (see include/qlora.h); all arithmetic runs in
the library's CUDA kernels. Tensors are torch CUDA tensors (used purely as
device memory); the stream is torch's current stream unless one is given.
There is no CPU fallback: importing the binding without the built library, or
calling it without a CUDA device, raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# QLORA_BOUNDS_CHECK=1 selects the bounds-checking build (python -m bit_nf4_quantized_03_b200.build --bounds-check)
BOUNDS_CHECK = os.environ.get("QLORA_BOUNDS_CHECK", "") not in ("", "0")
LIB_PATH = os.path.join(_PKG, "libqlora_bounds.so" if BOUNDS_CHECK else "libqlora.so")

QLORA_OK = 0
QLORA_ERR_INVALID = 1
QLORA_ERR_UNSUPPORTED = 2
QLORA_ERR_CUDA = 3
QLORA_ERR_WORKSPACE = 4
QLORA_ERR_DEVICE = 5
QLORA_ERR_BOUNDS = 6
QLORA_SCALE_BF16 = 0
QLORA_SCALE_DQ_FP8 = 1
QLORA_DTYPE_BF16 = 0
QLORA_DTYPE_FP32 = 1
QLORA_BWD_ACCUMULATE_GRADS = 1
QLORA_BWD_ACCUMULATE_DX = 2
QLORA_ROTARY_HALF = 0
QLORA_ROTARY_INTERLEAVED = 1
QLORA_ROTARY_SCALE_NONE = 0
QLORA_ROTARY_SCALE_LINEAR = 1
QLORA_ROTARY_SCALE_BANDS = 2
QLORA_ROTARY_SCALE_YARN = 3
QLORA_BLOCKSIZE = BLOCKSIZE = 64
QLORA_DQ_BLOCKSIZE = DQ_BLOCKSIZE = 256

# every symbol include/qlora.h declares
EXPORTED = (
    "qlora_status_string", "qlora_version", "qlora_nf4_levels",
    "qlora_nf4_quantize_workspace_bytes", "qlora_nf4_quantize", "qlora_nf4_dequantize",
    "qlora_linear_workspace_bytes", "qlora_linear_fwd", "qlora_linear_bwd",
    "qlora_silu_gate_fwd", "qlora_silu_gate_bwd", "qlora_check_device_error",
    "qlora_launch_count", "qlora_timing_begin", "qlora_timing_end", "qlora_timing_launch",
    "qlora_nf4_quantize_noalloc", "qlora_selftest_wait_timeout", "qlora_lora_merge",
    "qlora_linear_workspace_bytes_ex", "qlora_linear_fwd_ex", "qlora_linear_bwd_ex",
    "qlora_adamw_step", "qlora_paged_alloc", "qlora_paged_free", "qlora_paged_prefetch",
    "qlora_expand_rate", "qlora_bounds_site", "qlora_linear_bwd_group", "qlora_linear_group_workspace_bytes",
    "qlora_rotary_init", "qlora_rotary_apply", "qlora_norm_residual_fwd", "qlora_norm_residual_bwd",
    "qlora_norm_residual_workspace_bytes", "qlora_attention_fwd", "qlora_attention_fwd_workspace_bytes",
    "qlora_attention_bwd",
    "qlora_attention_bwd_workspace_bytes",
)


class QloraError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class NF4Weight(ctypes.Structure):
    """Mirror of qlora_nf4_weight."""
    _fields_ = [
        ("n", ctypes.c_int64), ("k", ctypes.c_int64),
        ("blocksize", ctypes.c_int32), ("dq_blocksize", ctypes.c_int32),
        ("mode", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("codes", ctypes.c_void_p), ("scale_bf16", ctypes.c_void_p),
        ("scale_fp8", ctypes.c_void_p), ("dq_scale", ctypes.c_void_p),
        ("dq_mean", ctypes.c_void_p),
    ]


class Dropout(ctypes.Structure):
    """Mirror of qlora_dropout: LoRA dropout rate, Philox seed and offset, and the
    device mask buffer (m * k / 8 bytes) the forward writes and the backward reads."""
    _fields_ = [
        ("p", ctypes.c_float), ("reserved", ctypes.c_int32),
        ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
        ("mask", ctypes.c_void_p),
    ]

    def __init__(self, p: float, seed: int, offset: int, mask):
        super().__init__(float(p), 0, int(seed), int(offset), _ptr(mask, allow_addr=True))
        self._mask = mask


class AdamWConfig(ctypes.Structure):
    """Mirror of qlora_adamw_config."""
    _fields_ = [
        ("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float), ("eps", ctypes.c_float),
        ("weight_decay", ctypes.c_float), ("grad_scale", ctypes.c_float), ("step", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]

    def __init__(self, lr: float, step: int, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                 weight_decay: float = 0.0, grad_scale: float = 1.0):
        super().__init__(lr, beta1, beta2, eps, weight_decay, grad_scale, int(step), 0)


class RotaryConfig(ctypes.Structure):
    """Mirror of qlora_rotary_config."""
    _fields_ = [
        ("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
        ("scaling", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double), ("low", ctypes.c_double),
        ("high", ctypes.c_double), ("original_length", ctypes.c_double), ("magnitude", ctypes.c_double),
    ]


class Rotary(ctypes.Structure):
    """Mirror of qlora_rotary: the table of turns per position that qlora_rotary_init fills."""
    _fields_ = [
        ("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
        ("magnitude", ctypes.c_float), ("turns", ctypes.c_double * 128),
    ]


class Norm(ctypes.Structure):
    """Mirror of qlora_norm."""
    _fields_ = [
        ("rows", ctypes.c_int64), ("cols", ctypes.c_int32), ("res_dtype", ctypes.c_int32),
        ("eps", ctypes.c_float), ("scale", ctypes.c_float),
    ]


class Attention(ctypes.Structure):
    """Mirror of qlora_attention."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("heads_q", ctypes.c_int32), ("heads_kv", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("causal", ctypes.c_int32), ("window", ctypes.c_int32), ("scale", ctypes.c_float),
        ("reserved", ctypes.c_int32), ("tokens_q", ctypes.c_int64), ("tokens_k", ctypes.c_int64),
        ("ld_q", ctypes.c_int64), ("ld_k", ctypes.c_int64), ("ld_v", ctypes.c_int64), ("ld_o", ctypes.c_int64),
        ("cu_q", ctypes.c_void_p), ("cu_k", ctypes.c_void_p),
    ]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libqlora.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libqlora.so not built ({LIB_PATH}); run python -m bit_nf4_quantized_03_b200.build")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    pw = ctypes.POINTER(NF4Weight)
    pd = ctypes.POINTER(Dropout)
    sig = {
        "qlora_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "qlora_version": (ctypes.c_char_p, []),
        "qlora_nf4_levels": (ctypes.c_int, [vp, vp]),
        "qlora_nf4_quantize_workspace_bytes": (sz, [i64, i64, i32]),
        "qlora_nf4_quantize": (ctypes.c_int, [vp, pw, vp, sz, vp]),
        "qlora_nf4_dequantize": (ctypes.c_int, [pw, vp, vp]),
        "qlora_linear_workspace_bytes": (sz, [i64, i64, i64, i32]),
        "qlora_linear_fwd": (ctypes.c_int, [pw, vp, i64, vp, vp, i32, f32, vp, i32, vp, vp, sz, vp]),
        "qlora_linear_bwd": (ctypes.c_int, [pw, vp, vp, i64, vp, vp, i32, f32, vp, vp, i32, vp, vp, i32,
                                            vp, sz, vp]),
        "qlora_silu_gate_fwd": (ctypes.c_int, [vp, vp, vp, i64, vp]),
        "qlora_silu_gate_bwd": (ctypes.c_int, [vp, vp, vp, vp, vp, i64, vp]),
        "qlora_check_device_error": (ctypes.c_int, [vp]),
        "qlora_launch_count": (ctypes.c_int64, []),
        "qlora_timing_begin": (ctypes.c_int, [i32]),
        "qlora_timing_end": (ctypes.c_int, [vp, vp, vp]),
        "qlora_timing_launch": (ctypes.c_int, [i32, vp, vp]),
        "qlora_nf4_quantize_noalloc": (ctypes.c_int, [vp, pw, vp]),
        "qlora_selftest_wait_timeout": (ctypes.c_int, [i32, vp]),
        "qlora_expand_rate": (ctypes.c_int, [i32, vp, vp]),
        "qlora_bounds_site": (ctypes.c_int, []),
        "qlora_lora_merge": (ctypes.c_int, [pw, vp, vp, i32, f32, vp, i32, vp]),
        "qlora_linear_workspace_bytes_ex": (sz, [i64, i64, i64, i32, pd]),
        "qlora_linear_bwd_group": (ctypes.c_int, [i32, vp, vp, vp, i64, vp, vp, i32, f32, vp, vp, i32, vp, vp, i32,
                                                  vp, sz, vp]),
        "qlora_linear_group_workspace_bytes": (sz, [i32, i64, vp, i64, i32]),
        "qlora_adamw_step": (ctypes.c_int, [vp, vp, vp, vp, vp, i64, ctypes.POINTER(AdamWConfig), vp]),
        "qlora_paged_alloc": (ctypes.c_int, [sz, ctypes.POINTER(ctypes.c_void_p)]),
        "qlora_paged_free": (ctypes.c_int, [vp]),
        "qlora_paged_prefetch": (ctypes.c_int, [vp, sz, i32, vp]),
        "qlora_linear_fwd_ex": (ctypes.c_int, [pw, vp, i64, vp, vp, i32, f32, vp, i32, vp, pd, vp, sz, vp]),
        "qlora_linear_bwd_ex": (ctypes.c_int, [pw, vp, vp, i64, vp, vp, i32, f32, vp, vp, i32, vp, vp, i32,
                                               pd, vp, sz, vp]),
    }
    sig.update({
        "qlora_rotary_init": (ctypes.c_int, [ctypes.POINTER(RotaryConfig), ctypes.POINTER(Rotary)]),
        "qlora_rotary_apply": (ctypes.c_int, [ctypes.POINTER(Rotary), vp, i64, vp, i64, i32, vp, i64, vp, i64, i32, vp,
                                              i64, i32, vp]),
        "qlora_norm_residual_fwd": (ctypes.c_int, [ctypes.POINTER(Norm), vp, vp, vp, vp, vp, vp, vp, vp]),
        "qlora_norm_residual_workspace_bytes": (sz, [i64, i32]),
        "qlora_norm_residual_bwd": (ctypes.c_int, [ctypes.POINTER(Norm), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                   i32, vp, sz, vp]),
        "qlora_attention_fwd_workspace_bytes": (sz, [ctypes.POINTER(Attention)]),
        "qlora_attention_fwd": (ctypes.c_int, [ctypes.POINTER(Attention), vp, vp, vp, vp, vp, vp, sz, vp]),
        "qlora_attention_bwd_workspace_bytes": (sz, [i64, i32]),
        "qlora_attention_bwd": (ctypes.c_int, [ctypes.POINTER(Attention), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
    })
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().qlora_status_string(int(status)).decode()


def _ptr(t, allow_addr: bool = False) -> int | None:
    """Device address of a CUDA tensor. Raw integer addresses are accepted only where
    an entry point documents them (paged memory), so a stray integer cannot stand in
    for a tensor argument."""
    if t is None:
        return None
    if isinstance(t, int):
        if not allow_addr:
            raise TypeError("expected a CUDA tensor, got an integer address")
        return t
    if not t.is_cuda:
        raise ValueError("libqlora takes CUDA tensors only (no CPU fallback)")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


# torch's current stream as an integer; the wrapper object of current_stream() costs more than a small call's launch
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str) -> None:
    if rc != QLORA_OK:
        raise QloraError(rc, where)


# ----------------------------------------------------------------- weight --
class QuantizedWeight:
    """Device buffers of one NF4 weight plus the C struct that points at them."""

    def __init__(self, n: int, k: int, mode: int = QLORA_SCALE_DQ_FP8, device="cuda"):
        self.n, self.k, self.mode = int(n), int(k), int(mode)
        ne = self.n * self.k
        nblk = -(-ne // BLOCKSIZE)
        nblk2 = -(-nblk // DQ_BLOCKSIZE)
        u8 = torch.uint8
        self.codes = torch.zeros((ne + 1) // 2, dtype=u8, device=device)
        self.scale_bf16 = self.scale_fp8 = self.dq_scale = self.dq_mean = None
        if self.mode == QLORA_SCALE_BF16:
            self.scale_bf16 = torch.zeros(nblk, dtype=torch.int16, device=device)
        else:
            self.scale_fp8 = torch.zeros(nblk, dtype=u8, device=device)
            self.dq_scale = torch.zeros(nblk2, dtype=torch.float32, device=device)
            self.dq_mean = torch.zeros(1, dtype=torch.float32, device=device)
        self.struct = NF4Weight(self.n, self.k, BLOCKSIZE, DQ_BLOCKSIZE, self.mode, 0,
                                _ptr(self.codes), _ptr(self.scale_bf16), _ptr(self.scale_fp8),
                                _ptr(self.dq_scale), _ptr(self.dq_mean))

    def ref(self):
        return ctypes.byref(self.struct)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in
                   (self.codes, self.scale_bf16, self.scale_fp8, self.dq_scale, self.dq_mean) if t is not None)


# ------------------------------------------------------------ entry points --
def qlora_version() -> str:
    return lib().qlora_version().decode()


def qlora_nf4_levels():
    lv = (ctypes.c_float * 16)()
    mid = (ctypes.c_float * 15)()
    _check(lib().qlora_nf4_levels(ctypes.addressof(lv), ctypes.addressof(mid)), "qlora_nf4_levels")
    return list(lv), list(mid)


def qlora_nf4_quantize_workspace_bytes(n: int, k: int, mode: int) -> int:
    return int(lib().qlora_nf4_quantize_workspace_bytes(n, k, mode))


def qlora_nf4_quantize(W: torch.Tensor, w: QuantizedWeight, ws: torch.Tensor | None = None, stream=None):
    """Quantize fp32 W [n, k] into w (allocates a workspace tensor on the call's stream if none is given)."""
    at = _ptr(W)
    ws, ws_bytes = _workspace(ws, qlora_nf4_quantize_workspace_bytes(w.n, w.k, w.mode), W, stream)
    _check(lib().qlora_nf4_quantize(at, w.ref(), _ptr(ws), ws_bytes, _stream(stream)), "qlora_nf4_quantize")
    return w


def qlora_nf4_dequantize(w: QuantizedWeight, out: torch.Tensor, stream=None) -> torch.Tensor:
    _check(lib().qlora_nf4_dequantize(w.ref(), _ptr(out), _stream(stream)), "qlora_nf4_dequantize")
    return out


def qlora_lora_merge(w: QuantizedWeight, A, B, r: int, alpha: float, out, out_dtype: int, stream=None):
    """out[n, k] = dequant(w) + (alpha / r) B A, in bf16 or fp32 (out_dtype)."""
    _check(lib().qlora_lora_merge(w.ref(), _ptr(A), _ptr(B), r, alpha, _ptr(out), out_dtype, _stream(stream)),
           "qlora_lora_merge")
    return out


def qlora_linear_workspace_bytes(m: int, n: int, k: int, r: int) -> int:
    return int(lib().qlora_linear_workspace_bytes(m, n, k, r))


def qlora_linear_fwd(w: QuantizedWeight, X, A, B, r: int, alpha: float, Y, y_dtype: int,
                     U_save=None, ws=None, stream=None):
    m = X.shape[0]
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().qlora_linear_fwd(w.ref(), _ptr(X), m, _ptr(A), _ptr(B), r, float(alpha), _ptr(Y), y_dtype,
                                _ptr(U_save), _ptr(ws), ws_bytes, _stream(stream))
    _check(rc, "qlora_linear_fwd")
    return Y


def qlora_linear_bwd(w: QuantizedWeight, X, dY, A, B, r: int, alpha: float, U_saved, dX, dx_dtype: int,
                     dA, dB, flags: int = 0, ws=None, stream=None):
    m = X.shape[0]
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().qlora_linear_bwd(w.ref(), _ptr(X), _ptr(dY), m, _ptr(A), _ptr(B), r, float(alpha), _ptr(U_saved),
                                _ptr(dX), dx_dtype, _ptr(dA), _ptr(dB), flags, _ptr(ws), ws_bytes,
                                _stream(stream))
    _check(rc, "qlora_linear_bwd")


def _dref(drop):
    return None if drop is None else ctypes.byref(drop)


def qlora_linear_workspace_bytes_ex(m: int, n: int, k: int, r: int, drop=None) -> int:
    return int(lib().qlora_linear_workspace_bytes_ex(m, n, k, r, _dref(drop)))


def qlora_linear_fwd_ex(w: QuantizedWeight, X, A, B, r: int, alpha: float, Y, y_dtype: int,
                        U_save=None, drop=None, ws=None, stream=None):
    m = X.shape[0]
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().qlora_linear_fwd_ex(w.ref(), _ptr(X), m, _ptr(A), _ptr(B), r, float(alpha), _ptr(Y), y_dtype,
                                   _ptr(U_save), _dref(drop), _ptr(ws), ws_bytes, _stream(stream))
    _check(rc, "qlora_linear_fwd_ex")
    return Y


def qlora_linear_bwd_ex(w: QuantizedWeight, X, dY, A, B, r: int, alpha: float, U_saved, dX, dx_dtype: int,
                        dA, dB, flags: int = 0, drop=None, ws=None, stream=None):
    m = X.shape[0]
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().qlora_linear_bwd_ex(w.ref(), _ptr(X), _ptr(dY), m, _ptr(A), _ptr(B), r, float(alpha),
                                   _ptr(U_saved), _ptr(dX), dx_dtype, _ptr(dA), _ptr(dB), flags, _dref(drop),
                                   _ptr(ws), ws_bytes, _stream(stream))
    _check(rc, "qlora_linear_bwd_ex")


def _ptr_array(items):
    """A C array of device addresses (None entries stay NULL)."""
    return (ctypes.c_void_p * len(items))(*[_ptr(t) for t in items])


def qlora_linear_group_workspace_bytes(m: int, ns, k: int, r: int) -> int:
    arr = (ctypes.c_int64 * len(ns))(*[int(n) for n in ns])
    return int(lib().qlora_linear_group_workspace_bytes(len(ns), m, ctypes.addressof(arr), k, r))


def qlora_linear_bwd_group(ws_list, X, dYs, As, Bs, r: int, alpha: float, U_saved, dX, dx_dtype: int,
                           dAs, dBs, flags: int = 0, ws=None, stream=None):
    """Backward of len(ws_list) layers sharing the input X: dX (+)= sum of the layers' terms,
    each layer's dA, dB as qlora_linear_bwd gives them."""
    count = len(ws_list)
    wp = (ctypes.POINTER(NF4Weight) * count)(*[ctypes.pointer(w.struct) for w in ws_list])
    dy, a, b, da, db = (_ptr_array(t) for t in (dYs, As, Bs, dAs, dBs))
    us = None if U_saved is None else _ptr_array(U_saved)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().qlora_linear_bwd_group(count, ctypes.addressof(wp), _ptr(X), ctypes.addressof(dy), X.shape[0],
                                      ctypes.addressof(a), ctypes.addressof(b), r, float(alpha),
                                      None if us is None else ctypes.addressof(us), _ptr(dX), dx_dtype,
                                      ctypes.addressof(da), ctypes.addressof(db), flags, _ptr(ws), ws_bytes,
                                      _stream(stream))
    _check(rc, "qlora_linear_bwd_group")


def qlora_adamw_step(param, grad, m, v, param_bf16, count: int, cfg: AdamWConfig, stream=None):
    """One AdamW step on fp32 masters (tensors or device-accessible addresses)."""
    _check(lib().qlora_adamw_step(_ptr(param, True), _ptr(grad, True), _ptr(m, True), _ptr(v, True),
                                  _ptr(param_bf16, True), int(count), ctypes.byref(cfg), _stream(stream)),
           "qlora_adamw_step")


def qlora_paged_alloc(nbytes: int) -> int:
    """Managed (pageable unified) memory for optimizer states; returns its address."""
    out = ctypes.c_void_p(0)
    _check(lib().qlora_paged_alloc(int(nbytes), ctypes.byref(out)), "qlora_paged_alloc")
    return int(out.value)


def qlora_paged_free(addr: int):
    _check(lib().qlora_paged_free(addr), "qlora_paged_free")


def qlora_paged_prefetch(addr: int, nbytes: int, to_host: bool = False, stream=None):
    _check(lib().qlora_paged_prefetch(addr, int(nbytes), 1 if to_host else 0, _stream(stream)),
           "qlora_paged_prefetch")


def qlora_silu_gate_fwd(g, u, h, stream=None):
    _check(lib().qlora_silu_gate_fwd(_ptr(g), _ptr(u), _ptr(h), g.numel(), _stream(stream)), "qlora_silu_gate_fwd")
    return h


def qlora_silu_gate_bwd(dh, g, u, dg, du, stream=None):
    _check(lib().qlora_silu_gate_bwd(_ptr(dh), _ptr(g), _ptr(u), _ptr(dg), _ptr(du), g.numel(), _stream(stream)),
           "qlora_silu_gate_bwd")


# ------------------------------------------- decoder-layer operators --
# These check shapes and types, and run on the device of their tensors, whichever device is current.
def _want(t, name: str, dtype, shape):
    if t is None:
        raise ValueError(f"{name} is missing")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


_MOST = 2 ** 31 - 1


def _i32(x, name: str) -> int:
    """x for a 32-bit argument; ctypes alone would take its low bits."""
    x = int(x)
    if not -_MOST <= x <= _MOST:
        raise ValueError(f"{name}: {x} does not fit 32 bits")
    return x


def _device(*tensors) -> int:
    """Index of the device that every given tensor lives on."""
    index = None
    for t in tensors:
        if t is not None:
            i = t.get_device()
            if i != index:
                if i < 0:
                    raise ValueError("libqlora takes CUDA tensors only (no CPU fallback)")
                if index is not None:
                    raise ValueError(f"tensors on different devices (cuda:{index} and cuda:{i})")
                index = i
    return index


def _run(name: str, dev: int, args, stream) -> None:
    """Call an entry point with its arguments up to the stream, on device `dev` whichever is current."""
    fn = getattr(lib(), name)
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            rc = fn(*args, _stream(stream))
    elif stream is None and _raw_stream is not None:
        rc = fn(*args, _raw_stream(dev))
    else:
        rc = fn(*args, _stream(stream))
    if rc != QLORA_OK:
        raise QloraError(rc, name)


def _on(dev: int, fn, *args):
    """fn(*args) with `dev` the current device."""
    if torch.cuda.current_device() == dev:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def _addr(t):
    return None if t is None else t.data_ptr()


def _dense(t, name: str, dtype, shape):
    """Address of a contiguous tensor of this type and shape (None for none)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _want(t, name, dtype, shape)
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _workspace(ws, need: int, like: torch.Tensor, stream):
    """(tensor, bytes) of the caller's workspace, or of one allocated for this call on its stream."""
    if ws is None and need > 0:
        if stream is None:
            ws = torch.empty(need, dtype=torch.uint8, device=like.device)
        else:
            if not isinstance(stream, int):
                s = stream
            elif stream == 0:        # ExternalStream(0) is not the default stream but a new one
                s = torch.cuda.default_stream(like.device)
            else:
                s = torch.cuda.ExternalStream(stream, device=like.device)
            with torch.cuda.stream(s):
                ws = torch.empty(need, dtype=torch.uint8, device=like.device)
    if ws is not None and not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return ws, 0 if ws is None else ws.numel() * ws.element_size()


def _heads(t, name: str) -> int:
    """Elements between the tokens of t [tokens, heads, head_dim], whose heads have to be contiguous."""
    m, h, d = t.shape
    if t.is_contiguous():
        return h * d
    ld, sh, sd = t.stride()
    if (sd != 1 and d > 1) or (sh != d and h > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return ld if m > 1 else h * d


_ROTARY_LAYOUTS = {"half": QLORA_ROTARY_HALF, "interleaved": QLORA_ROTARY_INTERLEAVED}
_ROTARY_SCALINGS = {"none": QLORA_ROTARY_SCALE_NONE, "linear": QLORA_ROTARY_SCALE_LINEAR,
                    "bands": QLORA_ROTARY_SCALE_BANDS, "yarn": QLORA_ROTARY_SCALE_YARN}


def _head_rows(t, name: str, shape) -> int:
    """Elements between the tokens of a bf16 tensor of this shape [tokens, heads, head_dim]."""
    if t.dtype is not torch.bfloat16 or t.shape != shape:
        _want(t, name, torch.bfloat16, shape)
    return shape[1] * shape[2] if t.is_contiguous() else _heads(t, name)


def qlora_rotary_init(head_dim: int, rot_dim: int | None = None, layout: str = "half", base: float = 10000.0,
                      scaling: str = "none", factor: float = 1.0, low: float = 0.0, high: float = 0.0,
                      original_length: float = 0.0, magnitude: float = 1.0) -> Rotary:
    """Table of the pairs' turns per position: layout "half" or "interleaved"; scaling "none", "linear", "bands" or "yarn"."""
    if layout not in _ROTARY_LAYOUTS or scaling not in _ROTARY_SCALINGS:
        raise ValueError(f"unknown layout {layout!r} or scaling {scaling!r}")
    cfg = RotaryConfig(_i32(head_dim, "head_dim"), _i32(head_dim if rot_dim is None else rot_dim, "rot_dim"),
                       _ROTARY_LAYOUTS[layout], _ROTARY_SCALINGS[scaling], base, factor, low, high, original_length,
                       magnitude)
    rot = Rotary()
    _check(lib().qlora_rotary_init(ctypes.byref(cfg), ctypes.byref(rot)), "qlora_rotary_init")
    return rot


def qlora_rotary_apply(rot: Rotary, positions, q, q_out=None, k=None, k_out=None, transpose: bool = False, stream=None):
    """Turn q (and k) [m, heads, head_dim] by their tokens' positions (int32 [m]); in place where no output is given.
    transpose: the backward map. Returns (q_out, k_out)."""
    q_out = q if q_out is None else q_out
    k_out = k if k_out is None else k_out
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    d = rot.head_dim
    if q is None or q.dim() != 3 or q.shape[2] != d or (k is not None and k.dim() != 3):
        raise ValueError("q and k are [tokens, heads, head_dim]")
    m, hq, _ = q.shape
    at = _dense(positions, "positions", torch.int32, (m,))
    if at is None:
        raise ValueError("positions is missing")
    ldq, ldqo = _head_rows(q, "q", q.shape), _head_rows(q_out, "q_out", q.shape)
    hk = ldk = ldko = 0
    if k is not None:
        hk = k.shape[1]
        ldk, ldko = _head_rows(k, "k", (m, hk, d)), _head_rows(k_out, "k_out", (m, hk, d))
    if hq > _MOST or hk > _MOST:
        raise ValueError("more heads than fit 32 bits")
    _run("qlora_rotary_apply", _device(q, q_out, positions, k, k_out),
         (ctypes.byref(rot), at, m, q.data_ptr(), ldq, hq, q_out.data_ptr(), ldqo, _addr(k), ldk, hk,
          _addr(k_out), ldko, 1 if transpose else 0), stream)
    return q_out, k_out


def _residual(x):
    """(shape, type, its code) of the residual stream x [rows, cols]."""
    if x is None or x.dim() != 2:
        raise ValueError("the residual stream is [rows, cols], bf16 or fp32")
    if x.shape[1] > _MOST:
        raise ValueError(f"cols: {x.shape[1]} does not fit 32 bits")
    if x.dtype is torch.bfloat16:
        return x.shape, torch.bfloat16, QLORA_DTYPE_BF16
    if x.dtype is torch.float32:
        return x.shape, torch.float32, QLORA_DTYPE_FP32
    raise ValueError("the residual stream is [rows, cols], bf16 or fp32")


def qlora_norm_residual_fwd(x, y, w_post, gate, w_pre, r, h, scale: float = 1.0, eps: float = 1e-5, stream=None):
    """r = x + scale * gate * (rms(y) w_post, or y); h = rms(r) w_pre. y, w_post, gate, w_pre with h, and r may be None."""
    bf, f32 = torch.bfloat16, torch.float32
    shape, res, dt = _residual(x)
    rows, cols = shape
    vec = (cols,)
    args = (ctypes.byref(Norm(rows, cols, dt, eps, scale)), _dense(x, "x", res, shape), _dense(y, "y", bf, shape),
            _dense(w_post, "w_post", f32, vec), _dense(gate, "gate", f32, vec), _dense(w_pre, "w_pre", f32, vec),
            _dense(r, "r", res, shape), _dense(h, "h", bf, shape))
    _run("qlora_norm_residual_fwd", _device(x, y, w_post, gate, w_pre, r, h), args, stream)
    return r, h


def qlora_norm_residual_workspace_bytes(rows: int, cols: int) -> int:
    return int(lib().qlora_norm_residual_workspace_bytes(rows, _i32(cols, "cols")))


def qlora_norm_residual_bwd(dr, dh, r, y, w_post, gate, w_pre, dx, dy=None, dw_post=None, dgate=None, dw_pre=None,
                            scale: float = 1.0, eps: float = 1e-5, flags: int = 0, ws=None, stream=None):
    """Backward of qlora_norm_residual_fwd from the gradients dr (of r) and dh (of h); a workspace is allocated if none
    is given and a weight gradient is asked for."""
    bf, f32 = torch.bfloat16, torch.float32
    shape, res, dt = _residual(r)
    rows, cols = shape
    vec = (cols,)
    args = (ctypes.byref(Norm(rows, cols, dt, eps, scale)), _dense(dr, "dr", res, shape), _dense(dh, "dh", bf, shape),
            _dense(r, "r", res, shape), _dense(y, "y", bf, shape), _dense(w_post, "w_post", f32, vec),
            _dense(gate, "gate", f32, vec), _dense(w_pre, "w_pre", f32, vec), _dense(dx, "dx", res, shape),
            _dense(dy, "dy", bf, shape), _dense(dw_post, "dw_post", f32, vec), _dense(dgate, "dgate", f32, vec),
            _dense(dw_pre, "dw_pre", f32, vec), _i32(flags, "flags"))
    dev = _device(r, dr, dh, y, w_post, gate, w_pre, dx, dy, dw_post, dgate, dw_pre, ws)
    need = 0
    if ws is None and (dw_post is not None or dgate is not None or dw_pre is not None):
        need = _on(dev, qlora_norm_residual_workspace_bytes, rows, cols)
    ws, ws_bytes = _workspace(ws, need, r, stream)
    _run("qlora_norm_residual_bwd", dev, (*args, _addr(ws), ws_bytes), stream)


def _attention(Q, K, V, O, lse, batch, causal, window, scale, cu_q, cu_k) -> Attention:
    """The qlora_attention of a call on Q, O [tokens_q, heads_q, d] and K, V [tokens_k, heads_kv, d]."""
    for name, t in (("Q", Q), ("K", K)):
        if t is None or t.dim() != 3:
            raise ValueError(f"{name} is [tokens, heads, head_dim]")
    bf = torch.bfloat16
    qs, ks = Q.shape, K.shape
    (tq, hq, d), (tk, hk, dk) = qs, ks
    if (V is None or O is None or dk != d or Q.dtype is not bf or K.dtype is not bf or V.dtype is not bf
            or O.dtype is not bf or V.shape != ks or O.shape != qs):
        _want(Q, "Q", bf, qs)
        _want(K, "K", bf, (tk, hk, d))
        _want(V, "V", bf, (tk, hk, d))
        _want(O, "O", bf, qs)
    if lse is not None:
        _want(lse, "lse", torch.float32, (tq, hq))
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
    if (cu_q is None) != (cu_k is None):
        raise ValueError("cu_q and cu_k come together")
    at_q = at_k = None
    if cu_q is not None:
        n = cu_q.shape[0]
        if batch is not None and batch != n - 1:
            raise ValueError(f"batch is {batch}, the offsets hold {n - 1} sequences")
        batch = n - 1
        for name, t in (("cu_q", cu_q), ("cu_k", cu_k)):
            _want(t, name, torch.int32, (n,))
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        at_q, at_k = cu_q.data_ptr(), cu_k.data_ptr()
    if Q.is_contiguous() and K.is_contiguous() and V.is_contiguous() and O.is_contiguous():
        ld_q = ld_o = hq * d
        ld_k = ld_v = hk * d
    else:
        ld_q, ld_k, ld_v, ld_o = _heads(Q, "Q"), _heads(K, "K"), _heads(V, "V"), _heads(O, "O")
    if hq > _MOST or hk > _MOST or d > _MOST:
        raise ValueError("more heads, or elements of one, than fit 32 bits")
    return Attention(1 if batch is None else _i32(batch, "batch"), hq, hk, d, 1 if causal else 0, _i32(window, "window"),
                     d ** -0.5 if scale is None and d > 0 else float(scale or 0.0), 0, tq, tk, ld_q, ld_k, ld_v, ld_o,
                     at_q, at_k)


def qlora_attention_fwd(Q, K, V, O, lse=None, batch: int | None = None, causal: bool = False, window: int = 0,
                        scale: float | None = None, cu_q=None, cu_k=None, ws=None, stream=None):
    """O = softmax(scale Q K^T) V and lse over packed sequences (int32 offsets cu_q, cu_k on the device) or `batch`
    equal ones. scale: 1 / sqrt(head_dim) when not given. A workspace is allocated if none is given and one is needed."""
    a = _attention(Q, K, V, O, lse, batch, causal, window, scale, cu_q, cu_k)
    dev = _device(Q, K, V, O, lse, cu_q, cu_k, ws)
    need = 0 if ws is not None else _on(dev, lib().qlora_attention_fwd_workspace_bytes, ctypes.byref(a))
    ws, ws_bytes = _workspace(ws, need, Q, stream)
    _run("qlora_attention_fwd", dev,
         (ctypes.byref(a), Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), _addr(lse), _addr(ws), ws_bytes), stream)
    return O, lse


def qlora_attention_bwd_workspace_bytes(tokens_q: int, heads_q: int) -> int:
    return int(lib().qlora_attention_bwd_workspace_bytes(tokens_q, _i32(heads_q, "heads_q")))


def qlora_attention_bwd(Q, K, V, O, dO, lse, dQ, dK, dV, batch: int | None = None, causal: bool = False, window: int = 0,
                        scale: float | None = None, cu_q=None, cu_k=None, ws=None, stream=None):
    """Gradients of qlora_attention_fwd from its O and lse and the gradient dO. dO is laid out as O, and dQ, dK, dV as
    Q, K, V; a workspace is allocated if none is given."""
    if lse is None:
        raise ValueError("lse is missing")
    a = _attention(Q, K, V, O, lse, batch, causal, window, scale, cu_q, cu_k)
    for name, t, like in (("dO", dO, O), ("dQ", dQ, Q), ("dK", dK, K), ("dV", dV, V)):
        if t is None or t.dtype is not torch.bfloat16 or t.shape != like.shape:
            _want(t, name, torch.bfloat16, like.shape)
        if not (t.is_contiguous() and like.is_contiguous()) and _heads(t, name) != _heads(like, name[1:]):
            raise ValueError(f"{name} must be laid out as {name[1:]}")
    dev = _device(Q, K, V, O, dO, lse, dQ, dK, dV, cu_q, cu_k, ws)
    need = qlora_attention_bwd_workspace_bytes(Q.shape[0], Q.shape[1]) if ws is None else 0
    ws, ws_bytes = _workspace(ws, need, Q, stream)
    _run("qlora_attention_bwd", dev,
         (ctypes.byref(a), Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), dO.data_ptr(), lse.data_ptr(),
          dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), _addr(ws), ws_bytes), stream)
    return dQ, dK, dV


def qlora_selftest_wait_timeout(limit_ms: int = 100, stream=None) -> None:
    _check(lib().qlora_selftest_wait_timeout(int(limit_ms), _stream(stream)), "qlora_selftest_wait_timeout")


def qlora_expand_rate(iters: int = 2048):
    """(weights expanded per SM-clock, per second) of the NF4 table expansion alone."""
    per_clk, per_s = ctypes.c_double(0), ctypes.c_double(0)
    _check(lib().qlora_expand_rate(int(iters), ctypes.addressof(per_clk), ctypes.addressof(per_s)),
           "qlora_expand_rate")
    return per_clk.value, per_s.value


def qlora_bounds_site() -> int:
    """Site of the first failed bounds check since the last call (0: none); bounds-check build only."""
    return int(lib().qlora_bounds_site())


def qlora_check_device_error(stream=None) -> None:
    rc = lib().qlora_check_device_error(_stream(stream))
    if rc != QLORA_OK and BOUNDS_CHECK:
        raise QloraError(rc, f"qlora_check_device_error (first failed bounds check: site {qlora_bounds_site()})")
    _check(rc, "qlora_check_device_error")


def qlora_launch_count() -> int:
    return int(lib().qlora_launch_count())


def qlora_timing_begin(max_launches: int) -> None:
    _check(lib().qlora_timing_begin(int(max_launches)), "qlora_timing_begin")


def qlora_timing_end():
    """Returns (total device ms, launches timed, algorithmic flops) of the fused GEMMs."""
    ms, n, fl = ctypes.c_double(0), ctypes.c_int32(0), ctypes.c_double(0)
    _check(lib().qlora_timing_end(ctypes.addressof(ms), ctypes.addressof(n), ctypes.addressof(fl)),
           "qlora_timing_end")
    return ms.value, n.value, fl.value


def qlora_timing_launches(count: int):
    """Per-launch (device ms, algorithmic flops) of the last qlora_timing_end, in launch order."""
    out = []
    for i in range(int(count)):
        ms, fl = ctypes.c_double(0), ctypes.c_double(0)
        _check(lib().qlora_timing_launch(i, ctypes.addressof(ms), ctypes.addressof(fl)), "qlora_timing_launch")
        out.append((ms.value, fl.value))
    return out


def qlora_nf4_quantize_noalloc(W: torch.Tensor, w: QuantizedWeight, stream=None):
    """qlora_nf4_quantize for callers that cannot allocate: no workspace, the
    library's fixed scratch array is used (calls must not overlap on the GPU)."""
    _check(lib().qlora_nf4_quantize_noalloc(_ptr(W), w.ref(), _stream(stream)), "qlora_nf4_quantize_noalloc")
    return w
