"""Python binding of libslim (include/slim.h). Argument marshalling only.

Every function has the name of the C entry point it calls. Device arrays are
torch CUDA tensors (PyTorch provides the memory and the stream); outputs that
are not supplied are allocated with torch.empty on the input's device. All the
arithmetic runs in the library's kernels. There is no fallback: if libslim.so
is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libslim.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "slim.h")

SLIM_X_F32, SLIM_X_BF16 = 0, 1
SLIM_OBJ_KL, SLIM_OBJ_MSE = 0, 1
OBJECTIVES = {"kl": SLIM_OBJ_KL, "mse": SLIM_OBJ_MSE}
SLIM_SBA_ADAPTIVE, SLIM_SBA_FULL = 0, 1
PRECISIONS = {"adaptive": SLIM_SBA_ADAPTIVE, "full": SLIM_SBA_FULL}
STATUS = {0: "SLIM_OK", 1: "SLIM_EINVAL", 2: "SLIM_ENOMEM", 3: "SLIM_ECUDA", 4: "SLIM_ETIMEOUT",
          5: "SLIM_ENOTPD", 6: "SLIM_ENODEV", 7: "SLIM_EINJECTED", 8: "SLIM_ERANGE"}


class SlimError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        self.device_detail = _lib().slim_last_status_detail()
        if self.device_detail:
            detail = (detail + " " if detail else "") + f"[device detail {self.device_detail}]"
        super().__init__(f"{where}: {STATUS.get(status, status)} ({_lib().slim_status_string(status).decode()})"
                         + (f" {detail}" if detail else ""))


_L = None
i64, i32, dbl, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_double, ctypes.c_void_p, ctypes.c_size_t


class SlimDiag(ctypes.Structure):
    _fields_ = [("H", vp), ("h", vp), ("S", vp), ("order", vp), ("kl", vp), ("tau_idx", vp),
                ("p_star", ctypes.c_int32), ("stage_ms", ctypes.c_float * 8), ("sba_split", vp)]


class SlimOptions(ctypes.Structure):
    _fields_ = [("objective", ctypes.c_int), ("sba_precision", ctypes.c_int), ("gptq", ctypes.c_int),
                ("order", vp)]


_SIGS = {
    "slim_status_string": (ctypes.c_char_p, [i32]),
    "slim_last_cuda_error": (ctypes.c_char_p, []),
    "slim_last_status_detail": (i32, []),
    "slim_version": (ctypes.c_char_p, []),
    "slim_num_candidates": (i32, [i64, i32]),
    "slim_row_words": (i64, [i64, i32]),
    "slim_launch_count": (i64, []),
    "slim_peak_fp64": (i32, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double), vp]),
    "slim_hessian_workspace_bytes": (sz, [i64, i64, i32]),
    "slim_hessian": (i32, [vp, i32, i64, i64, vp, vp, sz, vp]),
    "slim_hinv_diag_workspace_bytes": (sz, [i64]),
    "slim_hinv_diag": (i32, [vp, i64, dbl, vp, vp, sz, vp]),
    "slim_salience_workspace_bytes": (sz, [i64, i64, i32]),
    "slim_salience": (i32, [vp, i64, i64, vp, i32, vp, vp, vp, sz, vp]),
    "slim_salience_noalloc": (i32, [vp, i64, i64, vp, i32, vp, vp, vp]),
    "slim_sba_workspace_bytes": (sz, [i64, i64, i64, i32, i32]),
    "slim_sba_search": (i32, [vp, i64, i64, vp, i32, i64, i32, i32, vp, vp, vp, vp, vp, sz, vp]),
    "slim_sba_search_ex": (i32, [vp, i64, i64, vp, i32, i64, i32, i32, vp, i32, i32, vp, vp, vp, vp, sz, vp]),
    "slim_sba_split_workspace_bytes": (sz, [i64, i64, i64, i32, i32]),
    "slim_sba_search_split": (i32, [vp, i64, i64, vp, i32, i64, i32, i32, vp, vp, vp, vp, i64, vp, sz, vp]),
    "slim_sqc": (i32, [vp, i64, i64, vp, vp, i32, i32, dbl, i32, vp, vp, vp, vp, vp]),
    "slim_gptq_workspace_bytes": (sz, [i64, i64]),
    "slim_gptq": (i32, [vp, i64, i64, vp, vp, i32, i32, dbl, i32, vp, vp, vp, vp, vp, sz, vp]),
    "slim_dequant_gemv_workspace_bytes": (sz, [i64, i64, i32, i32, i64]),
    "slim_dequant_gemv": (i32, [vp, vp, vp, vp, i64, i64, i32, i32, vp, i32, i64, vp, vp, sz, vp]),
    "slim_dequant_grouped_gemm_workspace_bytes": (sz, [i64, i64, i64, i32, i32, i32, i32, i64]),
    "slim_dequant_grouped_gemm": (i32, [vp, vp, vp, vp, i64, i64, i64, i32, i32, vp, i32, i64, vp, vp, i64, vp, i32,
                                        vp, sz, vp]),
    "slim_async_status": (i32, [vp]),
    "slim_token_logprobs": (i32, [vp, i32, i64, i64, i64, vp, i32, vp, vp, vp, vp, vp]),
    "slim_workspace_bytes": (sz, [i64, i64, i64, i32, i32, i32]),
    "slim_quantize_layer": (i32, [vp, i64, i64, vp, i32, i64, i32, i32, dbl, i32, vp, vp, vp, vp, vp, sz, vp]),
    "slim_quantize_layer_ex": (i32, [vp, i64, i64, vp, i32, i64, i32, i32, dbl, i32, vp, vp, vp, vp, vp, sz, vp,
                                     ctypes.POINTER(SlimDiag)]),
    "slim_quantize_layer_opts": (i32, [vp, i64, i64, vp, i32, i64, i32, i32, dbl, i32, vp, vp, vp, vp, vp, sz, vp,
                                       ctypes.POINTER(SlimOptions), ctypes.POINTER(SlimDiag)]),
    "slim_quantize_layer_host": (i32, [vp, i64, i64, vp, i32, i64, i32, i32, dbl, i32, vp, vp, vp, vp, vp]),
}


def header_functions() -> list:
    """Names of every function declared in include/slim.h."""
    txt = open(HEADER).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    return sorted(set(re.findall(r"\b(slim_[a-z0-9_]+)\s*\(", txt)))


def _lib():
    global _L
    if _L is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -m post_weight_quantization_hessian_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _L = L
    return _L


def lib_path() -> str:
    _lib()
    return LIB_PATH


def _check(rc: int, where: str):
    if rc != 0:
        raise SlimError(rc, where, _lib().slim_last_cuda_error().decode())


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        return t.data_ptr()
    return int(t)


def _xdtype(X: torch.Tensor) -> int:
    if X.dtype in (torch.bfloat16, torch.uint16, torch.int16):
        return SLIM_X_BF16
    if X.dtype == torch.float32:
        return SLIM_X_F32
    raise ValueError(f"X must be bf16 (or its uint16 bits) or float32, got {X.dtype}")


def _x_np_dtype(X: np.ndarray) -> int:
    if X.dtype == np.uint16:
        return SLIM_X_BF16
    if X.dtype == np.float32:
        return SLIM_X_F32
    raise ValueError("host X must be uint16 bf16 bits or float32")


# --------------------------------------------------------------------- host-only queries
def slim_num_candidates(n: int, group: int) -> int:
    return _lib().slim_num_candidates(n, group)


def slim_row_words(n: int, avg_bits: int) -> int:
    return _lib().slim_row_words(n, avg_bits)


def slim_workspace_bytes(m, n, N, xdtype, group, avg_bits) -> int:
    return _lib().slim_workspace_bytes(m, n, N, xdtype, group, avg_bits)


def slim_launch_count() -> int:
    return _lib().slim_launch_count()


def slim_version() -> str:
    return _lib().slim_version().decode()


def slim_peak_fp64(stream=None):
    """(fp64 tensor-core MMA, fp64 FMA) rates of the current device, TFLOP/s."""
    a, b = ctypes.c_double(), ctypes.c_double()
    _check(_lib().slim_peak_fp64(ctypes.byref(a), ctypes.byref(b), _stream(stream)), "slim_peak_fp64")
    return a.value, b.value


# --------------------------------------------------------------------- stages
def slim_hessian(X: torch.Tensor, H: Optional[torch.Tensor] = None, ws=None, stream=None) -> torch.Tensor:
    N, n = X.shape
    if H is None:
        H = torch.empty((n, n), dtype=torch.float64, device=X.device)
    wsb = ws.numel() * ws.element_size() if isinstance(ws, torch.Tensor) else 0
    _check(_lib().slim_hessian(_ptr(X), _xdtype(X), N, n, _ptr(H), _ptr(ws), wsb, _stream(stream)), "slim_hessian")
    return H


def slim_hinv_diag(H: torch.Tensor, alpha: float = 0.01, h: Optional[torch.Tensor] = None, ws=None,
                   stream=None) -> torch.Tensor:
    n = H.shape[0]
    if h is None:
        h = torch.empty(n, dtype=torch.float64, device=H.device)
    wsb = ws.numel() * ws.element_size() if isinstance(ws, torch.Tensor) else 0
    _check(_lib().slim_hinv_diag(_ptr(H), n, float(alpha), _ptr(h), _ptr(ws), wsb, _stream(stream)),
           "slim_hinv_diag")
    return h


def slim_salience(W: torch.Tensor, h: torch.Tensor, group: int, S=None, order=None, ws=None, stream=None):
    m, n = W.shape
    k = n // group
    if S is None:
        S = torch.empty(k, dtype=torch.float64, device=W.device)
    if order is None:
        order = torch.empty(k, dtype=torch.int32, device=W.device)
    wsb = ws.numel() * ws.element_size() if isinstance(ws, torch.Tensor) else 0
    _check(_lib().slim_salience(_ptr(W), m, n, _ptr(h), group, _ptr(S), _ptr(order), _ptr(ws), wsb,
                                _stream(stream)), "slim_salience")
    return S, order


def slim_salience_noalloc(W: torch.Tensor, h: torch.Tensor, group: int, S=None, order=None, stream=None):
    """slim_salience without any device allocation by the library (fixed internal scratch)."""
    m, n = W.shape
    k = n // group
    if S is None:
        S = torch.empty(k, dtype=torch.float64, device=W.device)
    if order is None:
        order = torch.empty(k, dtype=torch.int32, device=W.device)
    _check(_lib().slim_salience_noalloc(_ptr(W), m, n, _ptr(h), group, _ptr(S), _ptr(order), _stream(stream)),
           "slim_salience_noalloc")
    return S, order


def slim_sba_search(W: torch.Tensor, X: torch.Tensor, group: int, avg_bits: int, order: torch.Tensor, ws=None,
                    stream=None):
    m, n = W.shape
    N = X.shape[0]
    k = n // group
    P = k // 2 + 1
    kl = torch.empty(P, dtype=torch.float64, device=W.device)
    p_star = torch.empty(1, dtype=torch.int32, device=W.device)
    bits = torch.empty(k, dtype=torch.uint8, device=W.device)
    wsb = ws.numel() * ws.element_size() if isinstance(ws, torch.Tensor) else 0
    _check(_lib().slim_sba_search(_ptr(W), m, n, _ptr(X), _xdtype(X), N, group, avg_bits, _ptr(order), _ptr(kl),
                                  _ptr(p_star), _ptr(bits), _ptr(ws), wsb, _stream(stream)), "slim_sba_search")
    return kl, p_star, bits


def slim_sba_search_ex(W: torch.Tensor, X: torch.Tensor, group: int, avg_bits: int, order: torch.Tensor,
                       objective: str = "kl", precision: str = "adaptive", ws=None, stream=None):
    """slim_sba_search with the objective "kl" or "mse" and the operand precision "adaptive" or
    "full"; order is any permutation of the groups."""
    m, n = W.shape
    N = X.shape[0]
    k = n // group
    P = k // 2 + 1
    kl = torch.empty(P, dtype=torch.float64, device=W.device)
    p_star = torch.empty(1, dtype=torch.int32, device=W.device)
    bits = torch.empty(k, dtype=torch.uint8, device=W.device)
    wsb = ws.numel() * ws.element_size() if isinstance(ws, torch.Tensor) else 0
    _check(_lib().slim_sba_search_ex(_ptr(W), m, n, _ptr(X), _xdtype(X), N, group, avg_bits, _ptr(order),
                                     OBJECTIVES[objective], PRECISIONS[precision], _ptr(kl), _ptr(p_star), _ptr(bits),
                                     _ptr(ws), wsb,
                                     _stream(stream)), "slim_sba_search_ex")
    return kl, p_star, bits


def slim_sba_search_split(W: torch.Tensor, X: torch.Tensor, group: int, avg_bits: int, order: torch.Tensor,
                          chunk_tokens: int, ws=None, stream=None):
    """slim_sba_search's outputs from the two-part schedule: phase A per chunk of
    chunk_tokens tokens (a multiple of 256), then the candidate steps."""
    m, n = W.shape
    N = X.shape[0]
    k = n // group
    P = k // 2 + 1
    kl = torch.empty(P, dtype=torch.float64, device=W.device)
    p_star = torch.empty(1, dtype=torch.int32, device=W.device)
    bits = torch.empty(k, dtype=torch.uint8, device=W.device)
    wsb = ws.numel() * ws.element_size() if isinstance(ws, torch.Tensor) else 0
    _check(_lib().slim_sba_search_split(_ptr(W), m, n, _ptr(X), _xdtype(X), N, group, avg_bits, _ptr(order),
                                        _ptr(kl), _ptr(p_star), _ptr(bits), int(chunk_tokens), _ptr(ws), wsb,
                                        _stream(stream)), "slim_sba_search_split")
    return kl, p_star, bits


def slim_sqc(W: torch.Tensor, h: torch.Tensor, bits: torch.Tensor, group: int, avg_bits: int, lam: float,
             n_tau: int, stream=None):
    m, n = W.shape
    k = n // group
    codes = torch.empty((m, n * avg_bits // 32), dtype=torch.int32, device=W.device)
    scale = torch.empty((m, k), dtype=torch.float32, device=W.device)
    zero = torch.empty((m, k), dtype=torch.float32, device=W.device)
    tau = torch.empty((m, k), dtype=torch.uint8, device=W.device)
    _check(_lib().slim_sqc(_ptr(W), m, n, _ptr(h), _ptr(bits), group, avg_bits, float(lam), n_tau, _ptr(codes),
                           _ptr(scale), _ptr(zero), _ptr(tau), _stream(stream)), "slim_sqc")
    return codes, scale, zero, tau


def slim_gptq(W: torch.Tensor, H: torch.Tensor, bits: torch.Tensor, group: int, avg_bits: int, lam: float,
              n_tau: int, ws=None, stream=None):
    """SQC's quantizer inside the GPTQ column loop (error compensation along U)."""
    m, n = W.shape
    k = n // group
    codes = torch.empty((m, n * avg_bits // 32), dtype=torch.int32, device=W.device)
    scale = torch.empty((m, k), dtype=torch.float32, device=W.device)
    zero = torch.empty((m, k), dtype=torch.float32, device=W.device)
    tau = torch.empty((m, k), dtype=torch.uint8, device=W.device)
    wsb = ws.numel() * ws.element_size() if isinstance(ws, torch.Tensor) else 0
    _check(_lib().slim_gptq(_ptr(W), m, n, _ptr(H), _ptr(bits), group, avg_bits, float(lam), n_tau, _ptr(codes),
                            _ptr(scale), _ptr(zero), _ptr(tau), _ptr(ws), wsb, _stream(stream)), "slim_gptq")
    return codes, scale, zero, tau


def slim_dequant_gemv(codes: torch.Tensor, bits: torch.Tensor, scale: torch.Tensor, zero: torch.Tensor, group: int,
                      avg_bits: int, x: torch.Tensor, y: Optional[torch.Tensor] = None, ws=None, stream=None):
    """y = x W_hat^T for a packed layer; x is [batch, n] (batch <= 8), float32 or bf16."""
    m, k = scale.shape
    n = k * group
    if x.dim() == 1:
        x = x.view(1, -1)
    B = x.shape[0]
    if y is None:
        y = torch.empty((B, m), dtype=torch.float32, device=codes.device)
    wsb = ws.numel() * ws.element_size() if isinstance(ws, torch.Tensor) else 0
    _check(_lib().slim_dequant_gemv(_ptr(codes), _ptr(bits), _ptr(scale), _ptr(zero), m, n, group, avg_bits, _ptr(x),
                                    _xdtype(x), B, _ptr(y), _ptr(ws), wsb, _stream(stream)), "slim_dequant_gemv")
    return y


# the current stream's handle without a Stream object around it (2 us of a call of 15)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_DTYPES = {torch.float32: SLIM_X_F32, torch.bfloat16: SLIM_X_BF16}


class _on:
    """The device of the tensors current, and new tensors allocated for the stream that the call runs on."""

    __slots__ = ("guards", "raw")

    def __init__(self, device, stream):
        self.guards = ()
        if stream is None and device.index == torch.cuda.current_device():  # the usual call: nothing to change
            self.raw = _raw_stream(device.index)
            return
        self.guards = [torch.cuda.device(device)]
        if stream is None:
            self.raw = torch.cuda.current_stream(device).cuda_stream
        else:
            self.raw = _stream(stream)
            if not hasattr(stream, "cuda_stream"):
                # 0 is the default stream's handle; as a handle from outside, torch takes it for "none given" and
                # returns a stream of its own pool
                stream = (torch.cuda.ExternalStream(self.raw, device=device) if self.raw
                          else torch.cuda.default_stream(device))
            self.guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self.guards:
            g.__enter__()
        return self.raw

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def slim_dequant_grouped_gemm(codes: torch.Tensor, bits: torch.Tensor, scale: torch.Tensor, zero: torch.Tensor,
                              group: int, avg_bits: int, x: torch.Tensor, offsets: torch.Tensor,
                              row_index: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                              y_dtype: Optional[torch.dtype] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """Y_e = X_e W_hat_e^T for packed layers codes [E, m, words], bits [E, k], scale and zero [E, m, k];
    expert e takes the rows offsets[e]..offsets[e + 1] of x [T, n], or with row_index [R] those rows
    of it. y is [R, m], of y_dtype (x's by default); rows of no expert are left as they are."""
    if scale.dim() != 3 or x.dim() != 2:
        raise ValueError("scale must be [E, m, k] and x [T, n]")
    E, m, k = scale.shape
    n = k * group
    dev = x.device
    T, xn = x.shape
    R = T if row_index is None else row_index.numel()
    if xn != n or x.dtype not in _DTYPES:
        raise ValueError("x must be [T, n], bf16 or float32")
    if codes.shape != (E, m, n * avg_bits // 32) or codes.dtype not in (torch.int32, torch.uint32):
        raise ValueError("codes must be [E, m, n * avg_bits / 32] int32")
    if bits.shape != (E, k) or bits.dtype != torch.uint8:
        raise ValueError("bits must be [E, k] uint8")
    if zero.shape != scale.shape or scale.dtype != torch.float32 or zero.dtype != torch.float32:
        raise ValueError("scale and zero must be [E, m, k] float32")
    if offsets.shape != (E + 1,) or offsets.dtype != torch.int32:
        raise ValueError("offsets must be [E + 1] int32")
    if row_index is not None and (row_index.dim() != 1 or row_index.dtype != torch.int32):
        raise ValueError("row_index must be [R] int32")
    if y is not None:
        if y.shape != (R, m) or y.dtype not in _DTYPES or y_dtype not in (None, y.dtype):
            raise ValueError("y must be [R, m], bf16 or float32")
    else:
        y_dtype = x.dtype if y_dtype is None else y_dtype
        if y_dtype not in _DTYPES:
            raise ValueError("y must be [R, m], bf16 or float32")
    if not (x.is_cuda and codes.device == bits.device == scale.device == zero.device == offsets.device == dev
            and (row_index is None or row_index.device == dev) and (y is None or y.device == dev)
            and (ws is None or ws.device == dev)):
        raise ValueError("all tensors must be on one CUDA device")
    lib = _lib()
    with _on(dev, stream) as s:
        if y is None:
            y = torch.empty((R, m), dtype=y_dtype, device=dev)
        if ws is None:
            wsb = lib.slim_dequant_grouped_gemm_workspace_bytes(E, m, n, group, avg_bits, _DTYPES[x.dtype],
                                                                row_index is not None, R)
            ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
        else:
            wsb = ws.numel() * ws.element_size()
        _check(lib.slim_dequant_grouped_gemm(_ptr(codes), _ptr(bits), _ptr(scale), _ptr(zero), E, m, n, group,
                                             avg_bits, _ptr(x), _DTYPES[x.dtype], x.shape[0], _ptr(row_index),
                                             _ptr(offsets), R, _ptr(y), _DTYPES[y.dtype], _ptr(ws), wsb, s),
               "slim_dequant_grouped_gemm")
    return y


def slim_async_status(stream=None, device=None):
    """Raises SlimError if an asynchronous call failed on the device since the last query; waits for the stream."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with _on(dev, stream) as s:
        _check(_lib().slim_async_status(s), "slim_async_status")


def slim_token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, top_k: int = 0, stream=None):
    """(logp, entropy, top_logp, top_id) of logits [N, V] (rows may be strided): the log probability of
    tokens [N] int64 (None without tokens; 0 where a token is outside [0, V)), the entropy, and the
    top_k largest log probabilities with their indices (None when top_k is 0)."""
    if logits.dim() != 2 or logits.dtype not in _DTYPES:
        raise ValueError("logits must be [N, V], bf16 or float32")
    N, V = logits.shape
    dev = logits.device
    ld, step = logits.stride()
    if N <= 1:
        ld = V
    if V < 1 or (step != 1 and V > 1) or ld < V:
        raise ValueError("the rows of logits must be contiguous")
    if tokens is not None and (tokens.shape != (N,) or tokens.dtype != torch.int64 or tokens.device != dev
                               or not tokens.is_contiguous()):
        raise ValueError("tokens must be [N] int64 on the logits' device")
    if not 0 <= top_k <= 32 or top_k > V:
        raise ValueError("top_k must be in 0..32 and at most V")
    if not logits.is_cuda:
        raise ValueError("logits must be on a CUDA device")
    with _on(dev, stream) as s:
        logp = None if tokens is None else torch.empty(N, dtype=torch.float32, device=dev)
        entropy = torch.empty(N, dtype=torch.float32, device=dev)
        top_logp = top_id = None
        if top_k:
            top_logp = torch.empty((N, top_k), dtype=torch.float32, device=dev)
            top_id = torch.empty((N, top_k), dtype=torch.int32, device=dev)
        _check(_lib().slim_token_logprobs(logits.data_ptr(), _DTYPES[logits.dtype], N, V, ld, _ptr(tokens), top_k,
                                          _ptr(logp), _ptr(entropy), _ptr(top_logp), _ptr(top_id), s),
               "slim_token_logprobs")
    return logp, entropy, top_logp, top_id


# --------------------------------------------------------------------- whole layer
def _layer_outputs(W, group, avg_bits):
    m, n = W.shape
    k = n // group
    return (torch.empty((m, n * avg_bits // 32), dtype=torch.int32, device=W.device),
            torch.empty((m, k), dtype=torch.float32, device=W.device),
            torch.empty((m, k), dtype=torch.float32, device=W.device),
            torch.empty(k, dtype=torch.uint8, device=W.device))


def alloc_workspace(W: torch.Tensor, X: torch.Tensor, group: int, avg_bits: int) -> torch.Tensor:
    m, n = W.shape
    nb = slim_workspace_bytes(m, n, X.shape[0], _xdtype(X), group, avg_bits)
    if nb == 0:
        raise ValueError("invalid layer shape")
    return torch.empty(nb, dtype=torch.uint8, device=W.device)


def slim_quantize_layer(W: torch.Tensor, X: torch.Tensor, group: int, avg_bits: int, lam: float = 0.1,
                        n_tau: int = 50, ws: Optional[torch.Tensor] = None, out=None, stream=None):
    m, n = W.shape
    codes, scale, zero, bits = out if out is not None else _layer_outputs(W, group, avg_bits)
    wsb = ws.numel() if isinstance(ws, torch.Tensor) else 0
    _check(_lib().slim_quantize_layer(_ptr(W), m, n, _ptr(X), _xdtype(X), X.shape[0], group, avg_bits, float(lam),
                                      n_tau, _ptr(codes), _ptr(scale), _ptr(zero), _ptr(bits), _ptr(ws), wsb,
                                      _stream(stream)), "slim_quantize_layer")
    return codes, scale, zero, bits


def slim_quantize_layer_ex(W: torch.Tensor, X: torch.Tensor, group: int, avg_bits: int, lam: float = 0.1,
                           n_tau: int = 50, ws: Optional[torch.Tensor] = None, want_H: bool = True, stream=None,
                           bufs: Optional[dict] = None):
    return slim_quantize_layer_opts(W, X, group, avg_bits, lam, n_tau, ws=ws, want_H=want_H, stream=stream,
                                    bufs=bufs)


def layer_buffers(W: torch.Tensor, group: int, avg_bits: int, want_H: bool = True) -> dict:
    """Output and diagnostic tensors of slim_quantize_layer_ex / _opts for a layer shape, to
    pass as bufs= to repeated calls (the same device addresses every call)."""
    m, n = W.shape
    k = n // group
    P = k // 2 + 1
    dev = W.device
    codes, scale, zero, bits = _layer_outputs(W, group, avg_bits)
    return {"codes": codes, "scale": scale, "zero": zero, "bits": bits,
            "H": torch.empty((n, n), dtype=torch.float64, device=dev) if want_H else None,
            "h": torch.empty(n, dtype=torch.float64, device=dev),
            "S": torch.empty(k, dtype=torch.float64, device=dev),
            "order": torch.empty(k, dtype=torch.int32, device=dev),
            "kl": torch.empty(P, dtype=torch.float64, device=dev),
            "tau_idx": torch.empty((m, k), dtype=torch.uint8, device=dev),
            "sba_split": torch.empty((n + 63) // 64, dtype=torch.uint8, device=dev)}


def slim_quantize_layer_opts(W: torch.Tensor, X: torch.Tensor, group: int, avg_bits: int, lam: float = 0.1,
                             n_tau: int = 50, ws: Optional[torch.Tensor] = None, want_H: bool = True,
                             objective: str = "kl", order: Optional[torch.Tensor] = None,
                             precision: str = "adaptive", gptq: bool = False, stream=None,
                             bufs: Optional[dict] = None):
    """The whole path with every intermediate (slim_quantize_layer_ex when the options are the
    defaults, else slim_quantize_layer_opts): objective "kl" or "mse", and optionally a
    caller's group order (device int32 permutation) in place of the salience order."""
    m, n = W.shape
    b = bufs if bufs is not None else layer_buffers(W, group, avg_bits, want_H)
    codes, scale, zero, bits = b["codes"], b["scale"], b["zero"], b["bits"]
    d = {key: b[key] for key in ("H", "h", "S", "order", "kl", "tau_idx", "sba_split")}
    diag = SlimDiag(H=_ptr(d["H"]), h=_ptr(d["h"]), S=_ptr(d["S"]), order=_ptr(d["order"]), kl=_ptr(d["kl"]),
                    tau_idx=_ptr(d["tau_idx"]), sba_split=_ptr(d["sba_split"]))
    wsb = ws.numel() if isinstance(ws, torch.Tensor) else 0
    if objective == "kl" and order is None and precision == "adaptive" and not gptq:
        _check(_lib().slim_quantize_layer_ex(_ptr(W), m, n, _ptr(X), _xdtype(X), X.shape[0], group, avg_bits,
                                             float(lam), n_tau, _ptr(codes), _ptr(scale), _ptr(zero), _ptr(bits),
                                             _ptr(ws), wsb, _stream(stream), ctypes.byref(diag)),
               "slim_quantize_layer_ex")
    else:
        opt = SlimOptions(objective=OBJECTIVES[objective], sba_precision=PRECISIONS[precision], gptq=int(gptq),
                          order=_ptr(order))
        _check(_lib().slim_quantize_layer_opts(_ptr(W), m, n, _ptr(X), _xdtype(X), X.shape[0], group, avg_bits,
                                               float(lam), n_tau, _ptr(codes), _ptr(scale), _ptr(zero), _ptr(bits),
                                               _ptr(ws), wsb, _stream(stream), ctypes.byref(opt),
                                               ctypes.byref(diag)), "slim_quantize_layer_opts")
    d.update(codes=codes, scale=scale, zero=zero, bits=bits, p_star=int(diag.p_star),
             stage_ms=list(diag.stage_ms)[:6], kernel_ms=list(diag.stage_ms)[6:8])
    return d


def slim_quantize_layer_host(W: np.ndarray, X: np.ndarray, group: int, avg_bits: int, lam: float = 0.1,
                             n_tau: int = 50, out=None, stream=None):
    """HOST arrays in and out (numpy, or pinned torch CPU tensors via .numpy())."""
    m, n = W.shape
    k = n // group
    if out is None:
        out = (np.empty((m, n * avg_bits // 32), np.uint32), np.empty((m, k), np.float32),
               np.empty((m, k), np.float32), np.empty(k, np.uint8))
    codes, scale, zero, bits = out
    for a in (W, X, codes, scale, zero, bits):
        if not a.flags["C_CONTIGUOUS"]:
            raise ValueError("host arrays must be C-contiguous")
    _check(_lib().slim_quantize_layer_host(W.ctypes.data, m, n, X.ctypes.data, _x_np_dtype(X), X.shape[0], group,
                                           avg_bits, float(lam), n_tau, codes.ctypes.data, scale.ctypes.data,
                                           zero.ctypes.data, bits.ctypes.data, _stream(stream)),
           "slim_quantize_layer_host")
    return codes, scale, zero, bits
