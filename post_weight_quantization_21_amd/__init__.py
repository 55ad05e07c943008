"""Python binding of libgptq (GPTQ layer quantization on MI355X / gfx950).

Thin argument marshalling over the C ABI declared in ``include/gptq.h``:
every step of the method runs in the library's HIP kernels.  PyTorch only
provides device memory (tensors, workspaces) and the current HIP stream.
The binding refuses to run without the built library: there is no fallback.

Names follow the C ABI: ``hessian_accumulate``, ``prepare_hinv``,
``quantize_layer``, ``rtn_quantize``, ``layer_loss``, ``workspace_bytes``.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgptq.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_HIP = 0, -1, -2, -3, -4
DT_F32, DT_BF16, DT_F16 = 0, 1, 2
OP_HESSIAN, OP_PREPARE, OP_QUANTIZE, OP_LOSS, OP_W4A16, OP_HESSIAN_TOKENS, OP_SMOOTH, OP_AWQ = 0, 1, 2, 3, 4, 5, 6, 7
OP_CALIBRATE, OP_GEMV = 8, 10
GEMV_GATHERS = 4096  # with M * d_in up to this, gemv and gemv_gated need no workspace under a column order

EXPORTED = (
    "gptq_hessian_accumulate", "gptq_prepare_hinv", "gptq_quantize_layer", "gptq_rtn_quantize",
    "gptq_layer_loss", "gptq_workspace_bytes", "gptq_status_string", "gptq_last_error",
    "gptq_pack_codes", "gptq_w4a16_gemm", "gptq_hessian_accumulate_tokens",
    "gptq_channel_stats", "gptq_smooth_scales", "gptq_awq_search", "gptq_scale_layer",
    "gptq_quantize_layer_noalloc", "gptq_timing_enable", "gptq_timing_read",
    "gptq_linear_forward", "gptq_calibrate_hessian", "gptq_calibrate_chunk_tokens",
    "gptq_gemv", "gptq_gemv_gated", "gptq_moe_layer", "gptq_moe_workspace_bytes",
)
TIMED_LAZY, TIMED_BATCH, TIMED_LAZY_SPLIT = 0, 1, 2
NOALLOC_SCRATCH_BYTES = 64 << 20  # GPTQ_NOALLOC_SCRATCH_BYTES


class GptqError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"gptq status {status}: {message}")
        self.status = status


class Config(ctypes.Structure):
    """Mirror of ``gptq_config``."""
    _fields_ = [("bits", ctypes.c_int32), ("symmetric", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("damp_rel", ctypes.c_float), ("act_order", ctypes.c_int32),
                ("grid", ctypes.c_int32), ("super_cols", ctypes.c_int32)]


class Packed(ctypes.Structure):
    """Mirror of ``gptq_packed``."""
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p),
                ("kperm", ctypes.c_void_p), ("d_out", ctypes.c_int64), ("d_in", ctypes.c_int64),
                ("bits", ctypes.c_int32), ("group_size", ctypes.c_int32)]


# gptq_grid: when the quantization grids are fitted
GRIDS = {"dynamic": 0, "static": 1, "tensor": 2}


def config(bits: int = 4, symmetric: bool = False, group_size: int = 128, block_size: int = 128,
           damp_rel: float = 0.01, act_order: bool = False, grid: str = "dynamic", super_cols: int = 0) -> Config:
    return Config(int(bits), int(bool(symmetric)), int(group_size), int(block_size), float(damp_rel),
                  int(bool(act_order)), GRIDS[grid], int(super_cols))


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libgptq.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m post_weight_quantization_21_amd.build`")
    lib = ctypes.CDLL(path)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    cfgp, pkp = ctypes.POINTER(Config), ctypes.POINTER(Packed)
    sig = {
        "gptq_hessian_accumulate": [vp, vp, vp, i32, i64, i64, i64, vp, sz, vp],
        "gptq_prepare_hinv": [vp, vp, i64, cfgp, vp, vp, vp, vp, sz, vp],
        "gptq_quantize_layer": [vp, i64, i64, vp, vp, cfgp, vp, vp, vp, vp, vp, sz, vp],
        "gptq_quantize_layer_noalloc": [vp, i64, i64, vp, vp, cfgp, vp, vp, vp, vp, vp],
        "gptq_rtn_quantize": [vp, i64, i64, cfgp, vp, vp, vp, vp],
        "gptq_layer_loss": [vp, vp, vp, vp, vp, vp, i64, i64, i32, vp, vp, sz, vp],
        "gptq_workspace_bytes": [ctypes.c_int, i64, i64, i64, cfgp, ctypes.POINTER(sz)],
        "gptq_pack_codes": [vp, i64, i64, i32, vp, vp, vp],
        "gptq_channel_stats": [vp, i32, i64, i64, i64, vp, vp, vp],
        "gptq_smooth_scales": [vp, vp, i64, i64, ctypes.c_float, vp, vp, sz, vp],
        "gptq_awq_search": [vp, i64, i64, vp, vp, i64, cfgp, i32, vp, vp, vp, vp, sz, vp],
        "gptq_scale_layer": [vp, i64, i64, vp, vp, vp, vp],
        "gptq_hessian_accumulate_tokens": [vp, vp, vp, i32, i64, i64, i64, vp, sz, vp],
        "gptq_w4a16_gemm": [vp, i32, i64, i64, i64, vp, vp, vp, vp, i32, i64, vp, i64, vp, sz, vp],
        "gptq_linear_forward": [vp, i64, vp, i64, vp, i64, i64, i64, i64, vp],
        "gptq_calibrate_hessian": [vp, vp, vp, i64, vp, i64, i64, i64, i64, vp, sz, vp],
        "gptq_calibrate_chunk_tokens": [i64],
        "gptq_gemv": [vp, i32, i64, i64, pkp, vp, vp, i32, i64, vp, sz, vp],
        "gptq_gemv_gated": [vp, i32, i64, i64, pkp, pkp, vp, i32, i64, vp, sz, vp],
        "gptq_moe_layer": [vp, i32, i64, i64, vp, i32, i32, i32, i32, pkp, pkp, pkp, vp, vp, vp, i32, i64, vp, sz, vp],
        "gptq_moe_workspace_bytes": [i64, i64, i64, i32, i32, ctypes.POINTER(sz)],
        "gptq_timing_enable": [i32],
        "gptq_timing_read": [i32, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i64), ctypes.POINTER(ctypes.c_double)],
        "gptq_status_string": [ctypes.c_int],
        "gptq_last_error": [],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = (ctypes.c_char_p if name in ("gptq_status_string", "gptq_last_error")
                     else ctypes.c_int64 if name == "gptq_calibrate_chunk_tokens" else ctypes.c_int)
    _lib = lib
    return lib


def _check(status: int) -> None:
    if status != OK:
        msg = load_library().gptq_last_error().decode(errors="replace")
        raise GptqError(status, msg)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous device tensors")


def timing_enable(on: bool = True) -> None:
    """Record HIP events around the column pass's update products and batch kernels (benchmarks)."""
    _check(load_library().gptq_timing_enable(int(bool(on))))


def timing_read(op: int, with_flops: bool = False):
    """(summed milliseconds, launches[, fp32 flops]) of the recorded kernels of one kind, then forget them."""
    ms, n, fl = ctypes.c_double(0.0), ctypes.c_int64(0), ctypes.c_double(0.0)
    _check(load_library().gptq_timing_read(int(op), ctypes.byref(ms), ctypes.byref(n), ctypes.byref(fl)))
    return (ms.value, n.value, fl.value) if with_flops else (ms.value, n.value)


def workspace_bytes(op: int, d_out: int, d_in: int, n_tok: int = 0, cfg: Config | None = None) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().gptq_workspace_bytes(op, d_out, d_in, n_tok, ctypes.byref(cfg) if cfg else None,
                                               ctypes.byref(out)))
    return int(out.value)


def _workspace(nbytes: int, device):
    import torch
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def hessian_accumulate(H, X, hdiag=None, ws=None, stream=None) -> None:
    """H (fp32 [d,d], upper) += 2 X X^T; hdiag (fp64 [d]) += 2 sum x^2.  X: bf16 or fp32 [d][n]."""
    import torch
    _need_cuda(H, hdiag)
    if not X.is_cuda or X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be a 2-D device tensor with unit stride along tokens")
    if X.dtype == torch.bfloat16:
        dt = DT_BF16
    elif X.dtype == torch.float32:
        dt = DT_F32
    else:
        raise ValueError("X must be bfloat16 or float32")
    d, n = X.shape
    if ws is None:
        ws = _workspace(workspace_bytes(OP_HESSIAN, 0, d, n), X.device)
    _check(load_library().gptq_hessian_accumulate(_ptr(H), _ptr(hdiag), _ptr(X), dt, d, n, X.stride(0), _ptr(ws),
                                                  ws.numel(), _stream(stream)))


def hessian_accumulate_tokens(H, X, hdiag=None, ws=None, stream=None) -> None:
    """H (fp32 [d,d], upper) += 2 X^T X for token-major X: bf16 or fp32 [n_tok][d], one row per token.
    bf16 rows must be a multiple of 4 elements apart (X.stride(0) % 4 == 0) and 8-byte aligned."""
    import torch
    _need_cuda(H, hdiag)
    if not X.is_cuda or X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be a 2-D device tensor with unit stride along channels")
    if X.dtype == torch.bfloat16:
        dt = DT_BF16
    elif X.dtype == torch.float32:
        dt = DT_F32
    else:
        raise ValueError("X must be bfloat16 or float32")
    n, d = X.shape
    if ws is None:
        ws = _workspace(workspace_bytes(OP_HESSIAN_TOKENS, 0, d, n), X.device)
    _check(load_library().gptq_hessian_accumulate_tokens(_ptr(H), _ptr(hdiag), _ptr(X), dt, d, n, X.stride(0),
                                                         _ptr(ws), ws.numel(), _stream(stream)))


def _bf16_rows(t, name):
    import torch
    if not t.is_cuda or t.dim() != 2 or t.stride(1) != 1 or t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be a 2-D bfloat16 device tensor with unit stride along its rows")


def linear_forward(Y, X, W, stream=None) -> None:
    """Y [n_tok][d_out] (bf16) = bf16(X W^T): X bf16 [n_tok][d_prev] token-major, W bf16 [d_out][d_prev]."""
    for t, n in ((Y, "Y"), (X, "X"), (W, "W")):
        _bf16_rows(t, n)
    n, dp = X.shape
    do = W.shape[0]
    if W.shape[1] != dp or tuple(Y.shape) != (n, do):
        raise ValueError("shapes: X [n][d_prev], W [d_out][d_prev], Y [n][d_out]")
    _check(load_library().gptq_linear_forward(_ptr(Y), Y.stride(0), _ptr(X), X.stride(0), _ptr(W), W.stride(0), n, dp,
                                              do, _stream(stream)))


def calibrate_chunk_tokens(d_in: int) -> int:
    return int(load_library().gptq_calibrate_chunk_tokens(d_in))


def calibrate_hessian(H, X, W, hdiag=None, ws=None, stream=None) -> None:
    """H (fp32 [d_in,d_in], upper) += 2 Y^T Y with Y = bf16(X W^T) made chunk by chunk on the device:
    X bf16 [n_tok][d_prev] (the previous layer's inputs), W bf16 [d_in][d_prev]."""
    _need_cuda(H, hdiag)
    _bf16_rows(X, "X")
    _bf16_rows(W, "W")
    n, dp = X.shape
    di = W.shape[0]
    if W.shape[1] != dp or tuple(H.shape) != (di, di):
        raise ValueError("shapes: X [n][d_prev], W [d_in][d_prev], H [d_in][d_in]")
    if ws is None:
        ws = _workspace(workspace_bytes(OP_CALIBRATE, 0, di, n), X.device)
    _check(load_library().gptq_calibrate_hessian(_ptr(H), _ptr(hdiag), _ptr(X), X.stride(0), _ptr(W), W.stride(0), n,
                                                 dp, di, _ptr(ws), ws.numel(), _stream(stream)))


def prepare_hinv(H, cfg: Config, U, perm=None, info=None, hdiag=None, ws=None, stream=None):
    """U = upper Cholesky factor of the damped (and ordered) inverse Hessian.  Returns the info tensor."""
    import torch
    _need_cuda(H, U, perm, info, hdiag)
    d = H.shape[0]
    if info is None:
        info = torch.empty(1, dtype=torch.int32, device=H.device)
    if ws is None:
        ws = _workspace(workspace_bytes(OP_PREPARE, 0, d, 0, cfg), H.device)
    _check(load_library().gptq_prepare_hinv(_ptr(H), _ptr(hdiag), d, ctypes.byref(cfg), _ptr(U), _ptr(perm),
                                            _ptr(info), _ptr(ws), ws.numel(), _stream(stream)))
    return info


def quantize_layer(W, U, cfg: Config, codes, scales, zeros, perm=None, g_idx=None, ws=None, stream=None) -> None:
    """GPTQ column pass (in place on W); writes codes/scales/zeros/g_idx."""
    _need_cuda(W, U, codes, scales, zeros, perm, g_idx)
    d_out, d_in = W.shape
    if ws is None:
        ws = _workspace(workspace_bytes(OP_QUANTIZE, d_out, d_in, 0, cfg), W.device)
    _check(load_library().gptq_quantize_layer(_ptr(W), d_out, d_in, _ptr(U), _ptr(perm), ctypes.byref(cfg),
                                              _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(g_idx), _ptr(ws),
                                              ws.numel(), _stream(stream)))


def quantize_layer_noalloc(W, U, cfg: Config, codes, scales, zeros, perm=None, g_idx=None, stream=None) -> None:
    """quantize_layer without a workspace: the library's fixed scratch array (NOALLOC_SCRATCH_BYTES)."""
    _need_cuda(W, U, codes, scales, zeros, perm, g_idx)
    d_out, d_in = W.shape
    _check(load_library().gptq_quantize_layer_noalloc(_ptr(W), d_out, d_in, _ptr(U), _ptr(perm), ctypes.byref(cfg),
                                                      _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(g_idx),
                                                      _stream(stream)))


def rtn_quantize(W, cfg: Config, codes, scales, zeros, stream=None) -> None:
    _need_cuda(W, codes, scales, zeros)
    d_out, d_in = W.shape
    _check(load_library().gptq_rtn_quantize(_ptr(W), d_out, d_in, ctypes.byref(cfg), _ptr(codes), _ptr(scales),
                                            _ptr(zeros), _stream(stream)))


def layer_loss(W, codes, scales, zeros, H, group_size: int, g_idx=None, out=None, ws=None, stream=None):
    """||W X - W_hat X||^2 through H (device fp64 scalar tensor)."""
    import torch
    _need_cuda(W, codes, scales, zeros, H, g_idx, out)
    d_out, d_in = W.shape
    if out is None:
        out = torch.empty(1, dtype=torch.float64, device=W.device)
    if ws is None:
        ws = _workspace(workspace_bytes(OP_LOSS, d_out, d_in), W.device)
    _check(load_library().gptq_layer_loss(_ptr(W), _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(g_idx), _ptr(H),
                                          d_out, d_in, int(group_size), _ptr(out), _ptr(ws), ws.numel(),
                                          _stream(stream)))
    return out


def channel_stats(X, absmax=None, abssum=None, stream=None):
    """Per input channel of X ([d][n], bf16 or fp32): (max |x| fp32, sum |x| fp64), accumulated."""
    import torch
    if not X.is_cuda or X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be a 2-D device tensor with unit stride along tokens")
    dt = DT_BF16 if X.dtype == torch.bfloat16 else DT_F32
    if X.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("X must be bfloat16 or float32")
    d, n = X.shape
    if absmax is None:
        absmax = torch.zeros(d, dtype=torch.float32, device=X.device)
    if abssum is None:
        abssum = torch.zeros(d, dtype=torch.float64, device=X.device)
    _need_cuda(absmax, abssum)
    _check(load_library().gptq_channel_stats(_ptr(X), dt, d, n, X.stride(0), _ptr(absmax), _ptr(abssum),
                                             _stream(stream)))
    return absmax, abssum


def smooth_scales(act_absmax, W, alpha: float = 0.5, s=None, ws=None, stream=None):
    """SmoothQuant scales s_j = max|X_j|^alpha / max|W_j|^(1 - alpha)."""
    import torch
    _need_cuda(act_absmax, W, s)
    d_out, d_in = W.shape
    if s is None:
        s = torch.empty(d_in, dtype=torch.float32, device=W.device)
    if ws is None:
        ws = _workspace(workspace_bytes(OP_SMOOTH, d_out, d_in), W.device)
    _check(load_library().gptq_smooth_scales(_ptr(act_absmax), _ptr(W), d_out, d_in, float(alpha), _ptr(s), _ptr(ws),
                                             ws.numel(), _stream(stream)))
    return s


def awq_search(W, H, act_abssum, n_tok: int, cfg: Config, n_grid: int = 20, ws=None, stream=None):
    """AWQ's grid search; returns device tensors (s [d_in], losses [n_grid] fp64, best [1] int32)."""
    import torch
    _need_cuda(W, H, act_abssum)
    d_out, d_in = W.shape
    s = torch.empty(d_in, dtype=torch.float32, device=W.device)
    losses = torch.empty(n_grid, dtype=torch.float64, device=W.device)
    best = torch.empty(1, dtype=torch.int32, device=W.device)
    if ws is None:
        ws = _workspace(workspace_bytes(OP_AWQ, d_out, d_in, 0, cfg), W.device)
    _check(load_library().gptq_awq_search(_ptr(W), d_out, d_in, _ptr(H), _ptr(act_abssum), int(n_tok), ctypes.byref(cfg),
                                          int(n_grid), _ptr(s), _ptr(losses), _ptr(best), _ptr(ws), ws.numel(),
                                          _stream(stream)))
    return s, losses, best


def scale_layer(s, W=None, H=None, hdiag=None, stream=None) -> None:
    """In place: W <- W diag(s), H <- diag(s)^-1 H diag(s)^-1 (upper), hdiag <- hdiag / s^2."""
    _need_cuda(s, W, H, hdiag)
    d_in = s.shape[0]
    d_out = W.shape[0] if W is not None else 0
    _check(load_library().gptq_scale_layer(_ptr(W), d_out, d_in, _ptr(H), _ptr(hdiag), _ptr(s), _stream(stream)))


def packed_words(d_in: int, bits: int) -> int:
    """32-bit words per packed row."""
    return (d_in * bits + 31) // 32


def pack_codes(codes, bits: int, packed=None, perm=None, stream=None):
    """Codes [d_out][d_in] u8 -> rows of little-endian bit streams (u32 [d_out][words])."""
    import torch
    _need_cuda(codes, packed, perm)
    d_out, d_in = codes.shape
    if packed is None:
        packed = torch.empty(d_out, packed_words(d_in, bits), dtype=torch.int32, device=codes.device)
    _check(load_library().gptq_pack_codes(_ptr(codes), d_out, d_in, int(bits), _ptr(perm), _ptr(packed),
                                          _stream(stream)))
    return packed


def w4a16_gemm(X, packed, scales, zeros, group_size: int, d_out: int, kperm=None, Y=None, ws=None, stream=None):
    """Y = X' W_hat^T with fp16 X [M][d_in] and 4-bit packed weights; Y fp32 [M][d_out].  Up to 16 rows gemv is faster."""
    import torch
    _need_cuda(packed, scales, zeros, kperm, Y)
    if not X.is_cuda:
        raise ValueError("X must be a device tensor")
    if X.dtype != torch.float16:
        raise TypeError("X must be float16")
    M, d_in = X.shape
    if X.stride(1) != 1:  # rows may sit at any pitch (ldx = X.stride(0)); within a row, contiguous
        raise ValueError("X rows must be contiguous")
    if Y is None:
        Y = torch.empty(M, d_out, dtype=torch.float32, device=X.device)
    if ws is None:
        ws = _workspace(workspace_bytes(OP_W4A16, d_out, d_in, M), X.device)
    _check(load_library().gptq_w4a16_gemm(_ptr(X), DT_F16, M, d_in, X.stride(0), _ptr(kperm), _ptr(packed),
                                          _ptr(scales), _ptr(zeros), int(group_size), d_out, _ptr(Y), Y.stride(0),
                                          _ptr(ws), ws.numel(), _stream(stream)))
    return Y


class PackedWeight:
    """A packed layer (or a stack of equal ones) for ``gemv``, ``gemv_gated`` and ``moe_layer``: the tensors and
    their ``gptq_packed``.  Built once, next to the weights; it keeps the tensors alive."""
    __slots__ = ("packed", "scales", "zeros", "kperm", "stack", "d_out", "d_in", "device", "c", "ref")

    def __init__(self, packed, scales, zeros, bits, group_size, kperm):
        import torch
        _need_cuda(packed, scales, zeros, kperm)
        if packed.dtype != torch.int32 or scales.dtype != torch.float32 or zeros.dtype != torch.float32 or \
                (kperm is not None and kperm.dtype != torch.int32):
            raise TypeError("packed and kperm must be int32, scales and zeros float32")
        if any(t.device != packed.device for t in (scales, zeros, kperm) if t is not None):
            raise ValueError("the tensors of a packed weight must be on one device")
        if bits not in (2, 3, 4, 8):
            raise ValueError("bits must be 2, 3, 4 or 8")
        if packed.dim() not in (2, 3) or packed.shape[-1] % bits or packed.numel() == 0:
            raise ValueError("packed must be [d_out][words] or [n][d_out][words], words = d_in * bits / 32 of a d_in "
                             "that is a multiple of 32")
        self.stack = packed.shape[0] if packed.dim() == 3 else None
        self.d_out, self.d_in = packed.shape[-2], packed.shape[-1] // bits * 32
        if group_size < 0 or (group_size and self.d_in % group_size):
            raise ValueError("group_size must divide d_in (0: one group per row)")
        lead = tuple(packed.shape[:-2])
        grid = lead + (self.d_out, n_groups(self.d_in, group_size))
        if tuple(scales.shape) != grid or tuple(zeros.shape) != grid:
            raise ValueError(f"scales and zeros must be {list(grid)}")
        if kperm is not None and tuple(kperm.shape) != lead + (self.d_in,):
            raise ValueError(f"kperm must be {list(lead + (self.d_in,))}")
        self.packed, self.scales, self.zeros, self.kperm, self.device = packed, scales, zeros, kperm, packed.device
        self.c = Packed(packed.data_ptr(), scales.data_ptr(), zeros.data_ptr(),
                        None if kperm is None else kperm.data_ptr(), self.d_out, self.d_in, bits, group_size)
        self.ref = ctypes.byref(self.c)


def packed_weight(packed, scales, zeros, bits: int = 4, group_size: int = 128, kperm=None) -> PackedWeight:
    """The packed layer of ``pack_codes`` (int32 [d_out][words]) with its grids (fp32 [d_out][d_in/g]) and, under a
    column order, the perm it was packed with; or a stack of equal layers, every tensor with a leading dimension."""
    return PackedWeight(packed, scales, zeros, int(bits), int(group_size), kperm)


# The few-token calls are made once per layer and token, so their host side is kept short: torch's types and the
# library's functions are looked up once, and pointers pass as integers.
_few_state = None


def _few_init():
    global _few_state
    if _few_state is None:
        import torch
        lib = load_library()
        _few_state = (torch, lib, {torch.float16: DT_F16, torch.bfloat16: DT_BF16},
                      {torch.float16: DT_F16, torch.bfloat16: DT_BF16, torch.float32: DT_F32})
    return _few_state


def _few_check_x(X, d_in, device, dtypes):
    dt = dtypes.get(X.dtype)
    if dt is None:
        raise TypeError("X must be float16 or bfloat16")
    if X.device != device or X.dim() != 2 or X.shape[1] != d_in or X.stride(1) != 1:
        raise ValueError(f"X must be [tokens][{d_in}] on the weights' device, contiguous within a row")
    return dt


def _few_result(X, Y, rows, d_out, out_dtype, device, torch, dtypes):
    if Y is None:
        Y = torch.empty((rows, d_out), dtype=out_dtype or X.dtype, device=device)
    elif out_dtype is not None and Y.dtype != out_dtype:
        raise TypeError("out_dtype is not the given result's type")
    elif Y.device != device or tuple(Y.shape) != (rows, d_out) or Y.stride(1) != 1:
        raise ValueError(f"the result must be [tokens][{d_out}] on the weights' device, contiguous within a row")
    dt = dtypes.get(Y.dtype)
    if dt is None:
        raise TypeError("the result must be float16, bfloat16 or float32")
    return Y, dt


def _few_on(stream, device, torch, layers, *tensors):
    """`stream` as the current stream: the call's result and workspace then come from, and go back to, the memory that
    this stream orders.  (From the caller's, either could still be in use there, or be handed out again too early.)  What
    the caller gives may be dropped when the call returns: its memory is not handed out before this stream is done."""
    if stream.device != device:
        raise ValueError("the stream must be on the weights' device")
    for w in layers:
        tensors += (w.packed, w.scales, w.zeros, w.kperm)
    for t in tensors:
        if t is not None and t.is_cuda:
            t.record_stream(stream)
    return torch.cuda.stream(stream)


def _few_launch(fn, device, torch, *args):
    """fn(*args, stream) with the weights' device current, on that device's current stream."""
    raw = torch._C._cuda_getCurrentRawStream(device.index)
    if torch.cuda.current_device() == device.index:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            status = fn(*args, raw)
    if status != OK:
        _check(status)


def _few_ws(ws, device):
    if ws is None:
        return None, 0
    if ws.device != device or not ws.is_contiguous():
        raise ValueError("the workspace must be a contiguous tensor on the weights' device")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _gemv_ws(ws, w, M, device):
    if ws is None:
        if w.kperm is None or M * w.d_in <= GEMV_GATHERS:  # not used
            return None, 0
        ws = _workspace(workspace_bytes(OP_GEMV, w.d_out, w.d_in, M), device)
    return _few_ws(ws, device)


def _pitch(t, rows, cols):
    """Elements between rows (a single row has no next one: torch may report any stride for it)."""
    return t.stride(0) if rows > 1 else cols


def gemv(X, w: PackedWeight, bias=None, Y=None, out_dtype=None, ws=None, stream=None):
    """Y = X' W_hat^T (+ bias) for at most 16 tokens: X fp16 or bf16 [M][d_in], w a packed layer of 2, 3, 4 or 8 bits,
    bias fp32 [d_out]; Y [M][d_out], apart from X, in X's type or in out_dtype (fp16, bf16, fp32)."""
    torch, lib, act, res = _few_init()
    if stream is not None:
        with _few_on(stream, w.device, torch, (w,), X, bias, Y, ws):
            return gemv(X, w, bias, Y, out_dtype, ws)
    if w.stack is not None:
        raise ValueError("gemv takes a single layer, not a stack")
    dev, d_in, d_out, M = w.device, w.d_in, w.d_out, X.shape[0]
    xd = _few_check_x(X, d_in, dev, act)
    Y, yd = _few_result(X, Y, M, d_out, out_dtype, dev, torch, res)
    if bias is not None and (bias.device != dev or bias.dtype != torch.float32 or tuple(bias.shape) != (d_out,)
                             or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous float32 [{d_out}] on the weights' device")
    wp, wn = _gemv_ws(ws, w, M, dev)
    _few_launch(lib.gptq_gemv, dev, torch, X.data_ptr(), xd, M, _pitch(X, M, d_in), w.ref,
                None if bias is None else bias.data_ptr(), Y.data_ptr(), yd, _pitch(Y, M, d_out), wp, wn)
    return Y


def gemv_gated(X, gate: PackedWeight, up: PackedWeight, H=None, out_dtype=None, ws=None, stream=None):
    """H = silu(X' W_gate^T) * (X' W_up^T), the first half of a gated MLP, for at most 16 tokens; types as in gemv.
    gate and up share one column order (the same kperm tensor), as they share their inputs."""
    torch, lib, act, res = _few_init()
    if stream is not None:
        with _few_on(stream, gate.device, torch, (gate, up), X, H, ws):
            return gemv_gated(X, gate, up, H, out_dtype, ws)
    if gate.stack is not None or up.stack is not None:
        raise ValueError("gemv_gated takes single layers, not stacks")
    dev, d_in, d_ff, M = gate.device, gate.d_in, gate.d_out, X.shape[0]
    if up.device != dev:
        raise ValueError("gate and up must be on one device")
    xd = _few_check_x(X, d_in, dev, act)
    H, hd = _few_result(X, H, M, d_ff, out_dtype, dev, torch, res)
    wp, wn = _gemv_ws(ws, gate, M, dev)
    _few_launch(lib.gptq_gemv_gated, dev, torch, X.data_ptr(), xd, M, _pitch(X, M, d_in), gate.ref, up.ref,
                H.data_ptr(), hd, _pitch(H, M, d_ff), wp, wn)
    return H


def moe_workspace_bytes(n_tok: int, d: int, d_ff: int, n_experts: int, top_k: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().gptq_moe_workspace_bytes(n_tok, d, d_ff, n_experts, top_k, ctypes.byref(out)))
    return int(out.value)


def moe_layer(X, gate: PackedWeight, up: PackedWeight, down: PackedWeight, router=None, top_k=None,
              renormalize: bool = True, ids=None, weights=None, Y=None, out_dtype=None, ws=None, stream=None):
    """A mixture-of-experts layer for at most 16 tokens: gate, up (stacks [E][d_ff][d]) and down ([E][d][d_ff]) packed,
    X fp16 or bf16 [T][d].  With a router ([E][d], fp32 or X's type) it chooses top_k experts per token; without one,
    ids (int32 [T][top_k]) and weights (fp32 [T][top_k]) are the caller's routing.  Returns (Y, ids, weights)."""
    torch, lib, act, res = _few_init()
    if stream is not None:
        with _few_on(stream, gate.device, torch, (gate, up, down), X, router, ids, weights, Y, ws):
            return moe_layer(X, gate, up, down, router, top_k, renormalize, ids, weights, Y, out_dtype, ws)
    E, dev, d, T = gate.stack, gate.device, gate.d_in, X.shape[0]
    if E is None or up.stack != E or down.stack != E:
        raise ValueError("gate, up and down must be stacks of the same number of experts")
    if up.device != dev or down.device != dev:
        raise ValueError("gate, up and down must be on one device")
    xd = _few_check_x(X, d, dev, act)
    Y, yd = _few_result(X, Y, T, d, out_dtype, dev, torch, res)
    rp, rd = None, DT_F32
    if router is None:
        if ids is None or weights is None:
            raise ValueError("without a router, ids and weights are needed")
        if top_k is None:
            top_k = ids.shape[-1] if ids.dim() else 0
    else:
        if top_k is None:
            raise ValueError("a router needs top_k")
        if router.device != dev or tuple(router.shape) != (E, d) or not router.is_contiguous():
            raise ValueError(f"router must be a contiguous [{E}][{d}] on the weights' device")
        rp, rd = router.data_ptr(), res.get(router.dtype)
        if rd is None:
            raise TypeError("router must be float32 or of X's type")
    top_k = int(top_k)
    if not 1 <= top_k <= E:
        raise ValueError("top_k must be 1 .. the number of experts")
    if ids is None:
        ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    elif ids.device != dev or ids.dtype != torch.int32 or tuple(ids.shape) != (T, top_k) or not ids.is_contiguous():
        raise ValueError(f"ids must be a contiguous int32 [{T}][{top_k}] on the weights' device")
    if weights is None:
        weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    elif weights.device != dev or weights.dtype != torch.float32 or tuple(weights.shape) != (T, top_k) or \
            not weights.is_contiguous():
        raise ValueError(f"weights must be a contiguous float32 [{T}][{top_k}] on the weights' device")
    if ws is None:
        ws = _workspace(moe_workspace_bytes(T, d, gate.d_out, E, top_k), dev)
    wp, wn = _few_ws(ws, dev)
    _few_launch(lib.gptq_moe_layer, dev, torch, X.data_ptr(), xd, T, _pitch(X, T, d), rp, rd, E, top_k,
                1 if renormalize else 0, gate.ref, up.ref, down.ref, ids.data_ptr(), weights.data_ptr(), Y.data_ptr(), yd,
                _pitch(Y, T, d), wp, wn)
    return Y, ids, weights


@dataclass
class LayerResult:
    codes: object
    scales: object
    zeros: object
    g_idx: object
    perm: object
    info: object


def n_groups(d_in: int, group_size: int) -> int:
    return d_in // group_size if group_size > 0 else 1


def gptq_layer(W, X, cfg: Config, H=None, hdiag=None):
    """Convenience: all four steps on device tensors (W is overwritten)."""
    import torch
    dev = W.device
    d_out, d_in = W.shape
    if H is None:
        H = torch.zeros(d_in, d_in, dtype=torch.float32, device=dev)
        if cfg.act_order and hdiag is None:
            hdiag = torch.zeros(d_in, dtype=torch.float64, device=dev)
        hessian_accumulate(H, X, hdiag)
    U = torch.empty(d_in, d_in, dtype=torch.float32, device=dev)
    perm = torch.empty(d_in, dtype=torch.int32, device=dev)
    info = prepare_hinv(H, cfg, U, perm, hdiag=hdiag)
    ng = n_groups(d_in, cfg.group_size)
    codes = torch.empty(d_out, d_in, dtype=torch.uint8, device=dev)
    scales = torch.empty(d_out, ng, dtype=torch.float32, device=dev)
    zeros = torch.empty(d_out, ng, dtype=torch.float32, device=dev)
    g_idx = torch.empty(d_in, dtype=torch.int32, device=dev)
    quantize_layer(W, U, cfg, codes, scales, zeros, perm, g_idx)
    return LayerResult(codes, scales, zeros, g_idx, perm, info), H, U
