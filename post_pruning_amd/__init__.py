"""SparseGPT layer solver for AMD Instinct MI355X (gfx950).

Thin ctypes binding over the C ABI of ``libsg.so`` (declared in include/sg.h).
The functions carry the same names as the C entry points; they only marshal
torch tensors (device memory and the current HIP stream) into the calls.  All
arithmetic runs in the library's HIP kernels: there is no fallback, and every
call raises if the library is missing or the device is not gfx950.

Pipeline for one linear layer (W: m x n, calibration X token-major [N, n]):

    H = torch.zeros(n, n, device="cuda")
    for Xc in chunks: sg_hessian_accumulate(H, Xc)
    Hinv, info = sg_prepare_hinv(H, damp=0.01)
    W_hat, mask = sg_prune_layer(W, Hinv, 0.5 or "2:4", blocksize=128)
    err = sg_reconstruction_error(W, W_hat, Xc)      # optional validation

Running and training a layer that was pruned and quantized:

    W_hat, mask, codes, scale, zero = sg_prune_quantize_layer(W, Hinv, "2:4", 8)
    layer = sg_pack_w8(codes, scale, zero)           # once
    q, x_scale, x_sum = sg_quantize_tokens(X)        # X [T, n] in 8 bits
    Y = sg_linear_w8a8(q, x_scale, x_sum, layer)     # X W_hat^T
    dX = sg_linear_w8_grad_input(dY, layer)
    dW = sg_linear_w8_grad_weight(dY, q, x_scale, mask)   # q is the checkpoint
    Y = linear_w8(X, W, layer, mask)                 # the same for autograd

The same in 8-bit floating point, with a scale for every block of 128, and with
dropout whose mask is never stored:

    layer = sg_pack_f8(W_hat)                        # once, or once a training step
    q, qt = sg_quantize_f8(X, form="both")           # rows, and transposed for dW
    Y = sg_linear_f8(q, layer)                       # X W_hat^T
    dy, dyt = sg_quantize_f8(dY, form="both")
    dX = sg_linear_f8_grad_input(dy, layer)
    dW = sg_linear_f8_grad_weight(dyt, qt, mask)
    Y = linear_f8(X, W, mask=mask, drop=Dropout(0.1, seed))   # the same for autograd
    Z = dropout(Y, Dropout(0.1, seed, offset=1), residual=X0) # drop(Y) + X0
"""

from __future__ import annotations

import ctypes
import functools
import operator
import os
from typing import Optional, Tuple, Union

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsg.so")

SG_OK, SG_ERR_INVALID_ARGUMENT, SG_ERR_UNSUPPORTED, SG_ERR_WORKSPACE, SG_ERR_HIP = range(5)
SG_F32, SG_BF16 = 0, 1
SG_UNSTRUCTURED, SG_NM, SG_UNSTRUCTURED_ROW = 0, 1, 2
SG_OP_HESSIAN, SG_OP_PREPARE_HINV, SG_OP_PRUNE, SG_OP_RECON = range(4)
SG_OP_LINEAR_W8A8, SG_OP_GRAD_INPUT, SG_OP_GRAD_WEIGHT = range(4, 7)
SG_OP_LINEAR_F8, SG_OP_F8_GRAD_INPUT, SG_OP_F8_GRAD_WEIGHT = range(7, 10)
SG_E4M3, SG_E5M2 = 0, 1
SG_F8_BLOCK, SG_F8_SCALE_PITCH = 128, 16
SG_CODE_PITCH = 64
SG_MAX_PITCH = 1 << 23  # bytes between rows of the 8-bit linear layer's operands
SG_MAX_BLOCKSIZE = 128
SG_MAX_SEGMENTS = 16
SG_NOALLOC_SCRATCH_BYTES = 64 << 20

_lib = None


class SGError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: {message} (status {status})")
        self.status = status


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libsg.so (built by __graft_entry__.build()); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build the HIP library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    c_i32, c_i64, c_sz, c_vp, c_dbl = (ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                                        ctypes.c_void_p, ctypes.c_double)
    lib.sg_hessian_accumulate.argtypes = [c_vp, c_i64, c_vp, c_i32, c_i64, c_i64, c_vp, c_sz, c_vp]
    lib.sg_prepare_hinv.argtypes = [c_vp, c_vp, c_i64, c_dbl, c_vp, c_vp, c_sz, c_vp, c_vp, c_vp, c_vp]
    lib.sg_prune_layer.argtypes = [c_vp, c_vp, c_vp, c_i32, c_i64, c_i64, c_i64, c_vp, c_i32,
                                   c_dbl, c_i32, c_i32, c_i32, c_vp, c_vp, c_sz, c_vp]
    lib.sg_reconstruction_error.argtypes = [c_vp, c_i32, c_vp, c_i32, c_i64, c_vp, c_i64, c_i64,
                                            c_vp, c_i32, c_i64, c_i64, c_vp, c_sz, c_vp]
    lib.sg_pack_two_four.argtypes = [c_vp, c_i32, c_vp, c_vp, c_vp, c_vp, c_i64, c_i64, c_vp]
    lib.sg_prune_quantize_layer.argtypes = [c_vp, c_vp, c_vp, c_vp, c_vp, c_i32, c_vp, c_i32, c_i64,
                                            c_i64, c_i64, c_vp, c_i32, c_dbl, c_i32, c_i32, c_i32,
                                            c_vp, c_vp, c_sz, c_vp]
    lib.sg_prune_layers_shared.argtypes = [c_vp, c_vp, c_vp, c_vp, c_vp, c_i32, c_vp, c_i32, c_i64,
                                           c_i64, c_i64, c_vp, c_i32, c_vp, c_i32, c_dbl, c_i32,
                                           c_i32, c_i32, c_vp, c_vp, c_sz, c_vp]
    lib.sg_prune_layer_noalloc.argtypes = [c_vp, c_vp, c_vp, c_i32, c_i64, c_i64, c_i64, c_vp, c_i32,
                                           c_dbl, c_i32, c_i32, c_i32, c_vp, c_vp]
    lib.sg_prune_layers_batched.argtypes = [c_vp, c_vp, c_vp, c_vp, c_vp, c_i32, c_vp, c_i32, c_i64,
                                            c_i64, c_i64, c_vp, c_i32, c_vp, c_i32, c_dbl, c_i32,
                                            c_i32, c_i32, c_vp, c_vp, c_sz, c_vp]
    lib.sg_prepare_hinv_batched.argtypes = [c_vp, c_vp, c_i32, c_i64, c_dbl, c_vp, c_vp, c_sz, c_vp, c_vp,
                                            c_vp, c_vp]
    lib.sg_prune_layer_vector.argtypes = [c_vp, c_vp, c_vp, c_i32, c_i64, c_i64, c_i64, c_vp, c_i32,
                                          c_dbl, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_sz, c_vp]
    lib.sg_quantize_tokens.argtypes = [c_vp, c_i64, c_vp, c_vp, c_vp, c_i32, c_i64, c_i64, c_i64, c_vp]
    lib.sg_dequantize_tokens.argtypes = [c_vp, c_i32, c_i64, c_vp, c_i64, c_vp, c_i64, c_i64, c_vp]
    lib.sg_pack_w8.argtypes = [c_vp, c_i64, c_vp, c_vp, c_vp, c_vp, c_vp, c_i64, c_i64, c_vp]
    lib.sg_linear_w8a8.argtypes = [c_vp, c_i32, c_i64, c_vp, c_i64, c_vp, c_vp, c_i64, c_vp, c_i64, c_vp,
                                   c_vp, c_i64, c_i64, c_vp, c_sz, c_vp]
    lib.sg_linear_w8_grad_input.argtypes = [c_vp, c_i32, c_i64, c_vp, c_i32, c_i64, c_i64, c_vp, c_i64, c_vp,
                                            c_vp, c_i64, c_i64, c_vp, c_sz, c_vp]
    lib.sg_linear_w8_grad_weight.argtypes = [c_vp, c_i32, c_i64, c_i32, c_vp, c_i32, c_i64, c_vp, c_i64, c_vp,
                                             c_i64, c_vp, c_i64, c_i64, c_vp, c_sz, c_vp]
    lib.sg_dropout.argtypes = [c_vp, c_i64, c_vp, c_i32, c_i64, c_vp, c_i64, c_i64, c_i64, c_vp, c_vp]
    lib.sg_quantize_f8.argtypes = [c_vp, c_i64, c_vp, c_i64, c_vp, c_i64, c_vp, c_i64, c_i32, c_vp, c_i32, c_i64,
                                   c_i64, c_i64, c_vp, c_vp]
    lib.sg_dequantize_f8.argtypes = [c_vp, c_i32, c_i64, c_vp, c_i64, c_vp, c_i64, c_i32, c_i64, c_i64, c_vp]
    lib.sg_pack_f8.argtypes = [c_vp, c_i64, c_vp, c_i64, c_vp, c_i64, c_vp, c_i64, c_vp, c_i32, c_i64, c_i64, c_i64,
                               c_vp]
    lib.sg_linear_f8.argtypes = [c_vp, c_i32, c_i64, c_vp, c_i64, c_vp, c_i64, c_i32, c_i64, c_vp, c_i64, c_vp, c_i64,
                                 c_i64, c_i64, c_vp, c_sz, c_vp]
    lib.sg_linear_f8_grad_input.argtypes = [c_vp, c_i32, c_i64, c_vp, c_i64, c_vp, c_i64, c_i32, c_i64, c_vp, c_i64,
                                            c_vp, c_i64, c_i64, c_i64, c_vp, c_vp, c_sz, c_vp]
    lib.sg_linear_f8_grad_weight.argtypes = [c_vp, c_i32, c_i64, c_i32, c_vp, c_i64, c_vp, c_i64, c_i32, c_vp, c_i64,
                                             c_vp, c_i64, c_i64, c_vp, c_i64, c_i64, c_vp, c_sz, c_vp]
    for f in ("sg_dropout", "sg_quantize_f8", "sg_dequantize_f8", "sg_pack_f8", "sg_linear_f8",
              "sg_linear_f8_grad_input", "sg_linear_f8_grad_weight"):
        getattr(lib, f).restype = c_i32
    for f in ("sg_quantize_tokens", "sg_dequantize_tokens", "sg_pack_w8", "sg_linear_w8a8",
              "sg_linear_w8_grad_input", "sg_linear_w8_grad_weight"):
        getattr(lib, f).restype = c_i32
    for f in ("sg_hessian_accumulate", "sg_prepare_hinv", "sg_prune_layer",
              "sg_reconstruction_error", "sg_pack_two_four", "sg_prune_quantize_layer",
              "sg_prune_layers_shared", "sg_prune_layer_vector", "sg_prune_layer_noalloc",
              "sg_prune_layers_batched", "sg_prepare_hinv_batched"):
        getattr(lib, f).restype = c_i32
    lib.sg_workspace_bytes.argtypes = [c_i32, c_i64, c_i64, c_i64, c_i32]
    lib.sg_workspace_bytes.restype = c_sz
    lib.sg_status_string.argtypes = [c_i32]
    lib.sg_status_string.restype = ctypes.c_char_p
    lib.sg_last_error_message.argtypes = []
    lib.sg_last_error_message.restype = ctypes.c_char_p
    lib.sg_abi_version.argtypes = []
    lib.sg_abi_version.restype = c_i32
    _lib = lib
    return lib


def sg_abi_version() -> int:
    return int(load_library().sg_abi_version())


def sg_status_string(s: int) -> str:
    return load_library().sg_status_string(int(s)).decode()


def sg_last_error_message() -> str:
    return load_library().sg_last_error_message().decode()


def sg_workspace_bytes(op: int, m: int = 0, n: int = 0, T: int = 0, blocksize: int = 0) -> int:
    return int(load_library().sg_workspace_bytes(op, m, n, T, blocksize))


def _check(status: int, where: str):
    if status != SG_OK:
        raise SGError(status, where, sg_last_error_message() or sg_status_string(status))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SG_F32
    if t.dtype == torch.bfloat16:
        return SG_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _require_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors must live on the GPU")


def _row_major(t: torch.Tensor, name: str) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D row-major tensor (unit column stride)")
    return t.stride(0)


def _stream(dev) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


def _workspace(nbytes: int, dev, workspace: Optional[torch.Tensor]):
    if nbytes == 0:
        return None, 0
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace of {nbytes} bytes needed")
        return workspace, workspace.numel() * workspace.element_size()
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    return ws, nbytes


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def sg_hessian_accumulate(H: torch.Tensor, X: torch.Tensor,
                          workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """H += X^T X for a token-major chunk X [T, n] (bf16 or fp32); H is [n, n] fp32."""
    lib = load_library()
    _require_cuda(H, X)
    if H.dtype != torch.float32 or not H.is_contiguous() or H.dim() != 2 or H.shape[0] != H.shape[1]:
        raise ValueError("H must be a contiguous square float32 tensor")
    n = H.shape[0]
    if X.dim() != 2 or X.shape[1] != n:
        raise ValueError("X must be [T, n]")
    ldx = _row_major(X, "X")
    T = X.shape[0]
    need = sg_workspace_bytes(SG_OP_HESSIAN, 0, n, T, 0)
    ws, nb = _workspace(need, H.device, workspace)
    _check(lib.sg_hessian_accumulate(_ptr(H), n, _ptr(X), _dtype_code(X), T, ldx, _ptr(ws), nb,
                                     ctypes.c_void_p(_stream(H.device))), "sg_hessian_accumulate")
    return H


# Above this n the factorisation's trailing updates can run on a second stream
# (the library's fused single-stream form is used up to it either way).
FACTOR_SPLIT_MIN_N = 4097


def sg_prepare_hinv(H: torch.Tensor, damp: float = 0.01, Hinv: Optional[torch.Tensor] = None,
                    info: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None,
                    update_stream: Union[str, None, "torch.cuda.Stream"] = "auto",
                    ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Upper Cholesky factor of (H + damp*mean(diag H) I)^{-1}; returns (Hinv, info).

    ``update_stream``: "auto" takes a stream from torch's pool and two fresh
    events for this call when n > 4096 (the trailing updates then overlap the
    panel chain); a torch.cuda.Stream uses that stream; None keeps every
    kernel on the current stream.  The library itself creates no stream."""
    lib = load_library()
    _require_cuda(H)
    n = H.shape[0]
    if H.dtype != torch.float32 or not H.is_contiguous() or H.shape != (n, n):
        raise ValueError("H must be a contiguous square float32 tensor")
    if Hinv is None:
        Hinv = torch.empty_like(H)
    if info is None:
        info = torch.empty(1, dtype=torch.int32, device=H.device)
    need = sg_workspace_bytes(SG_OP_PREPARE_HINV, 0, n, 0, 0)
    ws, nb = _workspace(need, H.device, workspace)
    side = ev_a = ev_b = None
    if isinstance(update_stream, str):
        if update_stream != "auto":
            raise ValueError("update_stream must be 'auto', None or a torch.cuda.Stream")
        if n >= FACTOR_SPLIT_MIN_N:
            side = torch.cuda.Stream(device=H.device)
    else:
        side = update_stream
    if side is not None:
        # events owned by this call (created by their first record)
        ev_a, ev_b = torch.cuda.Event(), torch.cuda.Event()
        ev_a.record(side)
        ev_b.record(side)
    _check(lib.sg_prepare_hinv(_ptr(Hinv), _ptr(H), n, float(damp), _ptr(info), _ptr(ws), nb,
                               ctypes.c_void_p(_stream(H.device)),
                               None if side is None else ctypes.c_void_p(side.cuda_stream),
                               None if ev_a is None else ctypes.c_void_p(ev_a.cuda_event),
                               None if ev_b is None else ctypes.c_void_p(ev_b.cuda_event)),
           "sg_prepare_hinv")
    return Hinv, info


def sg_prepare_hinv_batched(Hs, damp: float = 0.01, Hinvs=None, info: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None,
                            update_stream: Union[str, None, "torch.cuda.Stream"] = "auto"):
    """sg_prepare_hinv for several [n, n] matrices of one order n in one call;
    returns (Hinvs, info) with info an int32 tensor of one status per matrix.
    Each factor equals sg_prepare_hinv's of the same matrix, bit for bit."""
    lib = load_library()
    Hs = list(Hs)
    if not Hs:
        raise ValueError("at least one matrix")
    _require_cuda(*Hs)
    n = Hs[0].shape[0]
    for H in Hs:
        if H.dtype != torch.float32 or not H.is_contiguous() or H.shape != (n, n):
            raise ValueError("every H must be a contiguous square float32 tensor of the same order")
    nl = len(Hs)
    dev = Hs[0].device
    if Hinvs is None:
        Hinvs = [torch.empty_like(H) for H in Hs]
    if info is None:
        info = torch.empty(nl, dtype=torch.int32, device=dev)
    need = nl * sg_workspace_bytes(SG_OP_PREPARE_HINV, 0, n, 0, 0)
    ws, nb = _workspace(need, dev, workspace)
    side = ev_a = ev_b = None
    if isinstance(update_stream, str):
        if update_stream != "auto":
            raise ValueError("update_stream must be 'auto', None or a torch.cuda.Stream")
        if n >= FACTOR_SPLIT_MIN_N:
            side = torch.cuda.Stream(device=dev)
    else:
        side = update_stream
    if side is not None:
        ev_a, ev_b = torch.cuda.Event(), torch.cuda.Event()
        ev_a.record(side)
        ev_b.record(side)
    hp = (ctypes.c_void_p * nl)(*[h.data_ptr() for h in Hs])
    up = (ctypes.c_void_p * nl)(*[u.data_ptr() for u in Hinvs])
    _check(lib.sg_prepare_hinv_batched(ctypes.cast(up, ctypes.c_void_p), ctypes.cast(hp, ctypes.c_void_p), nl, n,
                                       float(damp), _ptr(info), _ptr(ws), nb, ctypes.c_void_p(_stream(dev)),
                                       None if side is None else ctypes.c_void_p(side.cuda_stream),
                                       None if ev_a is None else ctypes.c_void_p(ev_a.cuda_event),
                                       None if ev_b is None else ctypes.c_void_p(ev_b.cuda_event)),
           "sg_prepare_hinv_batched")
    return Hinvs, info


def parse_pattern(pattern: Union[float, str]):
    """0.5 -> (SG_UNSTRUCTURED, 0.5, 0, 1); "0.5/row" -> (SG_UNSTRUCTURED_ROW,
    0.5, 0, 1); "2:4" -> (SG_NM, 0.0, 2, 4)."""
    if isinstance(pattern, str) and ":" in pattern:
        a, b = pattern.split(":")
        return SG_NM, 0.0, int(a), int(b)
    if isinstance(pattern, str) and pattern.endswith("/row"):
        return SG_UNSTRUCTURED_ROW, float(pattern[:-4]), 0, 1
    return SG_UNSTRUCTURED, float(pattern), 0, 1


def sg_prune_layer(W: torch.Tensor, Hinv: torch.Tensor, pattern: Union[float, str],
                   blocksize: int = 128, mask_in: Optional[torch.Tensor] = None,
                   W_out: Optional[torch.Tensor] = None, mask_out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None):
    """Prune W ([m, n] bf16/fp32) with the factor Hinv; returns (W_hat fp32, mask uint8)."""
    lib = load_library()
    _require_cuda(W, Hinv, mask_in)
    m, n = W.shape
    ldw = _row_major(W, "W")
    if Hinv.shape != (n, n) or Hinv.dtype != torch.float32 or not Hinv.is_contiguous():
        raise ValueError("Hinv must be a contiguous [n, n] float32 tensor")
    if mask_in is not None:
        if mask_in.shape != (m, n) or not mask_in.is_contiguous():
            raise ValueError("mask_in must be a contiguous [m, n] tensor")
        mask_in = mask_in.to(torch.uint8)
    if W_out is None:
        W_out = torch.empty(m, n, dtype=torch.float32, device=W.device)
    if mask_out is None:
        mask_out = torch.empty(m, n, dtype=torch.uint8, device=W.device)
    kind, sp, nk, mg = parse_pattern(pattern)
    need = sg_workspace_bytes(SG_OP_PRUNE, m, n, 0, blocksize)
    ws, nb = _workspace(need, W.device, workspace)
    _check(lib.sg_prune_layer(_ptr(W_out), _ptr(mask_out), _ptr(W), _dtype_code(W), m, n, ldw,
                              _ptr(Hinv), kind, sp, nk, mg, int(blocksize), _ptr(mask_in), _ptr(ws),
                              nb, ctypes.c_void_p(_stream(W.device))), "sg_prune_layer")
    return W_out, mask_out


def sg_prune_layer_noalloc(W: torch.Tensor, Hinv: torch.Tensor, pattern: Union[float, str],
                           blocksize: int = 128, mask_in: Optional[torch.Tensor] = None,
                           W_out: Optional[torch.Tensor] = None,
                           mask_out: Optional[torch.Tensor] = None):
    """sg_prune_layer with the library's per-GPU scratch array in place of a
    workspace (the C call allocates nothing; pass W_out and mask_out to keep
    this wrapper from allocating them).  Calls overlapping on one GPU race."""
    lib = load_library()
    _require_cuda(W, Hinv, mask_in)
    m, n = W.shape
    ldw = _row_major(W, "W")
    if Hinv.shape != (n, n) or Hinv.dtype != torch.float32 or not Hinv.is_contiguous():
        raise ValueError("Hinv must be a contiguous [n, n] float32 tensor")
    if mask_in is not None:
        if mask_in.shape != (m, n) or not mask_in.is_contiguous() or mask_in.dtype != torch.uint8:
            raise ValueError("mask_in must be a contiguous [m, n] uint8 tensor")
    if W_out is None:
        W_out = torch.empty(m, n, dtype=torch.float32, device=W.device)
    if mask_out is None:
        mask_out = torch.empty(m, n, dtype=torch.uint8, device=W.device)
    kind, sp, nk, mg = parse_pattern(pattern)
    _check(lib.sg_prune_layer_noalloc(_ptr(W_out), _ptr(mask_out), _ptr(W), _dtype_code(W), m, n, ldw,
                                      _ptr(Hinv), kind, sp, nk, mg, int(blocksize), _ptr(mask_in),
                                      ctypes.c_void_p(_stream(W.device))), "sg_prune_layer_noalloc")
    return W_out, mask_out


def sg_prune_layer_vector(W: torch.Tensor, Hinv: torch.Tensor, pattern: Union[float, str], vec: int = 16,
                          blocksize: int = 128, mask_in: Optional[torch.Tensor] = None,
                          W_out: Optional[torch.Tensor] = None, mask_out: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None):
    """Prune W with the chosen weights of each range of ``vec`` columns removed
    together (vec = 16; vec = 1 is sg_prune_layer); returns (W_hat, mask)."""
    lib = load_library()
    _require_cuda(W, Hinv, mask_in)
    m, n = W.shape
    ldw = _row_major(W, "W")
    if Hinv.shape != (n, n) or Hinv.dtype != torch.float32 or not Hinv.is_contiguous():
        raise ValueError("Hinv must be a contiguous [n, n] float32 tensor")
    if mask_in is not None:
        if mask_in.shape != (m, n) or not mask_in.is_contiguous():
            raise ValueError("mask_in must be a contiguous [m, n] tensor")
        mask_in = mask_in.to(torch.uint8)
    if W_out is None:
        W_out = torch.empty(m, n, dtype=torch.float32, device=W.device)
    if mask_out is None:
        mask_out = torch.empty(m, n, dtype=torch.uint8, device=W.device)
    kind, sp, nk, mg = parse_pattern(pattern)
    need = sg_workspace_bytes(SG_OP_PRUNE, m, n, 0, blocksize)
    ws, nb = _workspace(need, W.device, workspace)
    _check(lib.sg_prune_layer_vector(_ptr(W_out), _ptr(mask_out), _ptr(W), _dtype_code(W), m, n, ldw,
                                     _ptr(Hinv), kind, sp, nk, mg, int(blocksize), int(vec),
                                     _ptr(mask_in), _ptr(ws), nb, ctypes.c_void_p(_stream(W.device))),
           "sg_prune_layer_vector")
    return W_out, mask_out


def sg_prune_quantize_layer(W: torch.Tensor, Hinv: torch.Tensor, pattern: Union[float, str], bits: int,
                            blocksize: int = 128, mask_in: Optional[torch.Tensor] = None,
                            W_out: Optional[torch.Tensor] = None,
                            mask_out: Optional[torch.Tensor] = None,
                            codes_out: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None):
    """Prune W and round its kept weights to a per-row grid of 2^bits levels in
    one sweep; returns (W_hat fp32, mask uint8, codes uint8, scale fp32 [m],
    zero fp32 [m]) with W_hat = scale * (codes - zero)."""
    lib = load_library()
    _require_cuda(W, Hinv, mask_in)
    m, n = W.shape
    ldw = _row_major(W, "W")
    if Hinv.shape != (n, n) or Hinv.dtype != torch.float32 or not Hinv.is_contiguous():
        raise ValueError("Hinv must be a contiguous [n, n] float32 tensor")
    if mask_in is not None:
        if mask_in.shape != (m, n) or not mask_in.is_contiguous():
            raise ValueError("mask_in must be a contiguous [m, n] tensor")
        mask_in = mask_in.to(torch.uint8)
    if W_out is None:
        W_out = torch.empty(m, n, dtype=torch.float32, device=W.device)
    if mask_out is None:
        mask_out = torch.empty(m, n, dtype=torch.uint8, device=W.device)
    if codes_out is None:
        codes_out = torch.empty(m, n, dtype=torch.uint8, device=W.device)
    scale = torch.empty(m, dtype=torch.float32, device=W.device)
    zero = torch.empty(m, dtype=torch.float32, device=W.device)
    kind, sp, nk, mg = parse_pattern(pattern)
    need = sg_workspace_bytes(SG_OP_PRUNE, m, n, 0, blocksize)
    ws, nb = _workspace(need, W.device, workspace)
    _check(lib.sg_prune_quantize_layer(_ptr(W_out), _ptr(mask_out), _ptr(codes_out), _ptr(scale),
                                       _ptr(zero), int(bits), _ptr(W), _dtype_code(W), m, n, ldw,
                                       _ptr(Hinv), kind, sp, nk, mg, int(blocksize), _ptr(mask_in),
                                       _ptr(ws), nb, ctypes.c_void_p(_stream(W.device))),
           "sg_prune_quantize_layer")
    return W_out, mask_out, codes_out, scale, zero


def sg_prune_layers_shared(W: torch.Tensor, row_splits, Hinv: torch.Tensor,
                           pattern: Union[float, str], blocksize: int = 128, bits: int = 0,
                           mask_in: Optional[torch.Tensor] = None,
                           W_out: Optional[torch.Tensor] = None,
                           mask_out: Optional[torch.Tensor] = None,
                           codes_out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None):
    """Prune matrices that share one input (stacked by rows in W, matrix p =
    rows row_splits[p]:row_splits[p+1]) with their shared factor in one call.

    Returns (W_hat, mask), or (W_hat, mask, codes, scale, zero) for bits > 0;
    each matrix's rows equal its own sg_prune_layer / sg_prune_quantize_layer
    result."""
    lib = load_library()
    _require_cuda(W, Hinv, mask_in)
    m, n = W.shape
    ldw = _row_major(W, "W")
    splits = [int(x) for x in row_splits]
    nseg = len(splits) - 1
    if Hinv.shape != (n, n) or Hinv.dtype != torch.float32 or not Hinv.is_contiguous():
        raise ValueError("Hinv must be a contiguous [n, n] float32 tensor")
    if mask_in is not None:
        if mask_in.shape != (m, n) or not mask_in.is_contiguous():
            raise ValueError("mask_in must be a contiguous [m, n] tensor")
        mask_in = mask_in.to(torch.uint8)
    if W_out is None:
        W_out = torch.empty(m, n, dtype=torch.float32, device=W.device)
    if mask_out is None:
        mask_out = torch.empty(m, n, dtype=torch.uint8, device=W.device)
    scale = zero = None
    if bits:
        if codes_out is None:
            codes_out = torch.empty(m, n, dtype=torch.uint8, device=W.device)
        scale = torch.empty(m, dtype=torch.float32, device=W.device)
        zero = torch.empty(m, dtype=torch.float32, device=W.device)
    kind, sp, nk, mg = parse_pattern(pattern)
    need = sg_workspace_bytes(SG_OP_PRUNE, m, n, 0, blocksize)
    ws, nb = _workspace(need, W.device, workspace)
    arr = (ctypes.c_int64 * max(1, len(splits)))(*splits)
    _check(lib.sg_prune_layers_shared(_ptr(W_out), _ptr(mask_out), _ptr(codes_out), _ptr(scale),
                                      _ptr(zero), int(bits), _ptr(W), _dtype_code(W), m, n, ldw,
                                      ctypes.cast(arr, ctypes.c_void_p), nseg, _ptr(Hinv), kind, sp,
                                      nk, mg, int(blocksize), _ptr(mask_in), _ptr(ws), nb,
                                      ctypes.c_void_p(_stream(W.device))), "sg_prune_layers_shared")
    if bits:
        return W_out, mask_out, codes_out, scale, zero
    return W_out, mask_out


def sg_prune_layers_batched(W: torch.Tensor, row_splits, Hinvs, pattern: Union[float, str],
                            blocksize: int = 128, bits: int = 0,
                            mask_in: Optional[torch.Tensor] = None,
                            W_out: Optional[torch.Tensor] = None,
                            mask_out: Optional[torch.Tensor] = None,
                            codes_out: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None):
    """Prune several layers' matrices (stacked by rows in W, matrix p = rows
    row_splits[p]:row_splits[p+1]), matrix p with its own factor Hinvs[p], in
    one call.  Returns (W_hat, mask), or (W_hat, mask, codes, scale, zero) for
    bits > 0; each matrix's rows equal its own sg_prune_layer /
    sg_prune_quantize_layer result with its own factor."""
    lib = load_library()
    _require_cuda(W, mask_in, *Hinvs)
    m, n = W.shape
    ldw = _row_major(W, "W")
    splits = [int(x) for x in row_splits]
    nseg = len(splits) - 1
    if len(Hinvs) != nseg:
        raise ValueError("one factor per matrix")
    for Hinv in Hinvs:
        if Hinv.shape != (n, n) or Hinv.dtype != torch.float32 or not Hinv.is_contiguous():
            raise ValueError("every factor must be a contiguous [n, n] float32 tensor")
    if mask_in is not None:
        if mask_in.shape != (m, n) or not mask_in.is_contiguous():
            raise ValueError("mask_in must be a contiguous [m, n] tensor")
        mask_in = mask_in.to(torch.uint8)
    if W_out is None:
        W_out = torch.empty(m, n, dtype=torch.float32, device=W.device)
    if mask_out is None:
        mask_out = torch.empty(m, n, dtype=torch.uint8, device=W.device)
    scale = zero = None
    if bits:
        if codes_out is None:
            codes_out = torch.empty(m, n, dtype=torch.uint8, device=W.device)
        scale = torch.empty(m, dtype=torch.float32, device=W.device)
        zero = torch.empty(m, dtype=torch.float32, device=W.device)
    kind, sp, nk, mg = parse_pattern(pattern)
    need = sg_workspace_bytes(SG_OP_PRUNE, m, n, 0, blocksize)
    ws, nb = _workspace(need, W.device, workspace)
    arr = (ctypes.c_int64 * max(1, len(splits)))(*splits)
    ptrs = (ctypes.c_void_p * max(1, nseg))(*[h.data_ptr() for h in Hinvs])
    _check(lib.sg_prune_layers_batched(_ptr(W_out), _ptr(mask_out), _ptr(codes_out), _ptr(scale),
                                       _ptr(zero), int(bits), _ptr(W), _dtype_code(W), m, n, ldw,
                                       ctypes.cast(arr, ctypes.c_void_p), nseg,
                                       ctypes.cast(ptrs, ctypes.c_void_p), kind, sp, nk, mg,
                                       int(blocksize), _ptr(mask_in), _ptr(ws), nb,
                                       ctypes.c_void_p(_stream(W.device))), "sg_prune_layers_batched")
    if bits:
        return W_out, mask_out, codes_out, scale, zero
    return W_out, mask_out


def sg_reconstruction_error(W: torch.Tensor, W_hat: torch.Tensor, X: torch.Tensor,
                            err: Optional[torch.Tensor] = None, accumulate: bool = False,
                            workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """||(W - W_hat) X^T||_F^2 over a token-major chunk X; returns a device float64 scalar."""
    lib = load_library()
    _require_cuda(W, W_hat, X)
    m, n = W.shape
    ldw = _row_major(W, "W")
    ldx = _row_major(X, "X")
    if W_hat.shape != (m, n) or W_hat.dtype != torch.float32 or not W_hat.is_contiguous():
        raise ValueError("W_hat must be a contiguous [m, n] float32 tensor")
    if X.shape[1] != n:
        raise ValueError("X must be [T, n]")
    if err is None:
        err = torch.zeros(1, dtype=torch.float64, device=W.device)
    T = X.shape[0]
    need = sg_workspace_bytes(SG_OP_RECON, m, n, T, 0)
    ws, nb = _workspace(need, W.device, workspace)
    _check(lib.sg_reconstruction_error(_ptr(err), int(bool(accumulate)), _ptr(W), _dtype_code(W),
                                       ldw, _ptr(W_hat), m, n, _ptr(X), _dtype_code(X), T, ldx,
                                       _ptr(ws), nb, ctypes.c_void_p(_stream(W.device))),
           "sg_reconstruction_error")
    return err


def sg_pack_two_four(W_hat: torch.Tensor, mask: torch.Tensor,
                     value_dtype: torch.dtype = torch.float32,
                     values: Optional[torch.Tensor] = None, meta: Optional[torch.Tensor] = None):
    """2:4 compressed form of a pruned [m, n] matrix.

    Returns (values [m, n/2] of ``value_dtype`` (float32 or bfloat16),
    meta [m, ceil(n/8)] uint8, bad: device int32 count of groups with more than
    two kept positions)."""
    lib = load_library()
    _require_cuda(W_hat, mask)
    m, n = W_hat.shape
    if W_hat.dtype != torch.float32 or not W_hat.is_contiguous():
        raise ValueError("W_hat must be a contiguous float32 tensor")
    if mask.shape != (m, n) or not mask.is_contiguous():
        raise ValueError("mask must be a contiguous [m, n] tensor")
    mask = mask.to(torch.uint8)
    if value_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("value_dtype must be float32 or bfloat16")
    if values is None:
        values = torch.empty(m, n // 2, dtype=value_dtype, device=W_hat.device)
    elif (values.shape != (m, n // 2) or values.dtype != value_dtype or not values.is_contiguous()
          or not values.is_cuda):
        raise ValueError("values must be a contiguous [m, n/2] GPU tensor of value_dtype")
    if meta is None:
        meta = torch.empty(m, (n + 7) // 8, dtype=torch.uint8, device=W_hat.device)
    elif meta.shape != (m, (n + 7) // 8) or meta.dtype != torch.uint8 or not meta.is_contiguous() \
            or not meta.is_cuda:
        raise ValueError("meta must be a contiguous [m, ceil(n/8)] uint8 GPU tensor")
    bad = torch.empty(1, dtype=torch.int32, device=W_hat.device)
    _check(lib.sg_pack_two_four(_ptr(values), _dtype_code(values), _ptr(meta), _ptr(bad),
                                _ptr(W_hat), _ptr(mask), m, n,
                                ctypes.c_void_p(_stream(W_hat.device))), "sg_pack_two_four")
    return values, meta, bad


# ---------------------------------------------------------------------------
# The 8-bit linear layer
# ---------------------------------------------------------------------------
class W8Layer:
    """A quantized layer as sg_pack_w8 lays it out: ``codes`` int8 [m, n] (a view
    of rows padded to SG_CODE_PITCH bytes), ``offset`` int32 [m] and ``scale``
    fp32 [m]; W_hat = scale * (codes + offset).  Its parts are checked once,
    here, and are not to be replaced or resized.  The padding of the rows has to
    hold zeros (a column slice of a wider layer does not): making a layer of
    tensors reads it back, so that belongs before a stream capture."""
    __slots__ = ("codes", "offset", "scale", "m", "n", "pitch")

    def __init__(self, codes: torch.Tensor, offset: torch.Tensor, scale: torch.Tensor):
        self._take(codes, offset, scale)
        pad = -(-self.n // SG_CODE_PITCH) * SG_CODE_PITCH
        if self.m > 0 and pad > self.n:
            rest = codes.as_strided((self.m, pad - self.n), (self.pitch, 1), codes.storage_offset() + self.n)
            if bool(rest.any()):
                raise ValueError(f"the rows of the layer's codes must be padded with zeros to a multiple of "
                                 f"{SG_CODE_PITCH} bytes (as sg_pack_w8 lays them out)")

    @classmethod
    def _unwritten(cls, m, n, device):
        """The tensors of a layer that sg_pack_w8 is about to write."""
        layer = cls.__new__(cls)
        layer._take(_code_rows(m, n, device), torch.empty(m, dtype=torch.int32, device=device),
                    torch.empty(m, dtype=torch.float32, device=device))
        return layer

    def _take(self, codes, offset, scale):
        self.m, self.n, self.pitch = _codes(codes, "the layer's codes")
        _shaped(offset, "the layer's offset", (self.m,), torch.int32)
        _shaped(scale, "the layer's scale", (self.m,), torch.float32)
        if not codes.device == offset.device == scale.device:
            raise ValueError("the layer's tensors must live on one GPU")
        self.codes, self.offset, self.scale = codes, offset, scale


# The raw handle of a device's current stream, without building a Stream object
# (a call of a few microseconds would notice that).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _same_gpu(first, *others) -> int:
    """The index of the one GPU that all tensors live on."""
    index = first.get_device()
    if index < 0:
        raise ValueError("tensors must live on the GPU")
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors must live on one GPU")
    return index


def _call(where, index, fn, *args):
    """One library call on the current stream of GPU ``index``, with that device current."""
    if _current_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status != SG_OK:
        _check(status, where)


def _shaped(t, name, shape, dtype):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)} {str(dtype)[6:]} tensor")
    return t


def _rows(t, name, rows, cols):
    """Checks a row-major fp32 or bf16 operand; returns its dtype code and pitch."""
    code = SG_BF16 if t.dtype is torch.bfloat16 else SG_F32 if t.dtype is torch.float32 else None
    if code is None or t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}] of float32 or bfloat16")
    pitch, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must be row-major (unit column stride)")
    # a single row (or none) has no pitch of its own, whatever its stride says:
    # one that keeps its pieces aligned
    return code, pitch if rows > 1 else -(-cols // 8) * 8


def _codes(t, name, cols=None):
    """Checks rows of codes; returns (rows, columns, pitch)."""
    if t.dtype is not torch.int8 or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D row-major int8 tensor")
    rows, n = t.shape
    pitch, step = t.stride()
    if step != 1 and n > 1:
        raise ValueError(f"{name} must be a 2-D row-major int8 tensor")
    if cols is not None and n != cols:
        raise ValueError(f"{name} must have {cols} columns")
    pad = -(-n // SG_CODE_PITCH) * SG_CODE_PITCH
    if pad != n and rows > 0:
        # rows are read up to the padded width: the storage has to hold them
        end = t.storage_offset() + (rows - 1) * pitch + pad
        if end > t.untyped_storage().nbytes():
            raise ValueError(f"the rows of {name} must be padded to a multiple of {SG_CODE_PITCH} bytes "
                             "(as the package's calls return them)")
    return rows, n, pitch if rows > 1 else pad


def _code_rows(rows, cols, device):
    pad = -(-cols // SG_CODE_PITCH) * SG_CODE_PITCH
    t = torch.empty(rows, pad, dtype=torch.int8, device=device)
    return t if pad == cols else t[:, :cols]


def _float_code(dtype, name):
    if dtype is torch.bfloat16:
        return SG_BF16
    if dtype is torch.float32:
        return SG_F32
    raise ValueError(f"{name} must be float32 or bfloat16")


def _out_rows(t, name, rows, cols, dtype, like):
    """An output operand, made here if it was not given: (tensor, dtype code, pitch)."""
    if t is None:
        code = _float_code(dtype, name)
        return like.new_empty((rows, cols), dtype=dtype), code, cols
    return (t, *_rows(t, name, rows, cols))


@functools.lru_cache(maxsize=4096)
def _ws_bytes(op, m, n, T):
    return sg_workspace_bytes(op, m, n, T, 0)


def _scratch(op, m, n, T, device, workspace):
    """(tensor that holds it, pointer, bytes) of an operation's workspace."""
    ws, nbytes = _workspace(_ws_bytes(op, m, n, T), device, workspace)
    return ws, (None if ws is None else ws.data_ptr()), nbytes


def _wrote(t):
    """A call wrote into a tensor that the caller holds: autograd is told, as it
    may have saved it (inference tensors have no version)."""
    if not t.is_inference():
        torch.autograd.graph.increment_version(t)


_FLOATS = (torch.float32, torch.bfloat16)


def sg_quantize_tokens(X: torch.Tensor, q: Optional[torch.Tensor] = None,
                       scale: Optional[torch.Tensor] = None, total: Optional[torch.Tensor] = None):
    """8-bit codes of X [T, n] (bf16 or fp32), one scale a token; returns
    (q int8 [T, n], scale fp32 [T], total int32 [T]): X ~ scale * q, total the
    sum of a token's codes.  q is a view of rows padded to SG_CODE_PITCH bytes;
    a given q is written up to that width too (zeros behind column n)."""
    lib = load_library()
    gpu = _same_gpu(X, q, scale, total)
    if X.dim() != 2:
        raise ValueError("X must be [T, n]")
    T, n = X.shape
    x_dtype, ldx = _rows(X, "X", T, n)
    given = q, scale, total
    if q is None:
        q = _code_rows(T, n, X.device)
        ldq = -(-n // SG_CODE_PITCH) * SG_CODE_PITCH
    else:
        rows, _, ldq = _codes(q, "q", n)
        if rows != T:
            raise ValueError(f"q must have {T} rows")
    if scale is None:
        scale = X.new_empty(T, dtype=torch.float32)
    else:
        _shaped(scale, "scale", (T,), torch.float32)
    if total is None:
        total = X.new_empty(T, dtype=torch.int32)
    else:
        _shaped(total, "total", (T,), torch.int32)
    _call("sg_quantize_tokens", gpu, lib.sg_quantize_tokens, q.data_ptr(), ldq, scale.data_ptr(),
          total.data_ptr(), X.data_ptr(), x_dtype, T, n, ldx)
    for t in given:
        if t is not None:
            _wrote(t)
    return q, scale, total


def sg_dequantize_tokens(q: torch.Tensor, scale: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                         X_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The [T, n] tensor that the codes of sg_quantize_tokens stand for, in
    ``dtype`` (bfloat16 or float32)."""
    lib = load_library()
    gpu = _same_gpu(q, scale, X_out)
    T, n, ldq = _codes(q, "q")
    _shaped(scale, "scale", (T,), torch.float32)
    given = X_out is not None
    X_out, x_dtype, ldx = _out_rows(X_out, "X_out", T, n, dtype, q)
    _call("sg_dequantize_tokens", gpu, lib.sg_dequantize_tokens, X_out.data_ptr(), x_dtype, ldx,
          q.data_ptr(), ldq, scale.data_ptr(), T, n)
    if given:
        _wrote(X_out)
    return X_out


def sg_pack_w8(codes: torch.Tensor, scale: torch.Tensor, zero: torch.Tensor) -> W8Layer:
    """Lays the (codes uint8 [m, n], scale [m], zero [m]) of a quantized layer
    (sg_prune_quantize_layer) out for the calls below, once."""
    lib = load_library()
    gpu = _same_gpu(codes, scale, zero)
    if codes.dim() != 2:
        raise ValueError("codes must be [m, n]")
    m, n = codes.shape
    _shaped(codes, "codes", (m, n), torch.uint8)
    _shaped(scale, "scale", (m,), torch.float32)
    _shaped(zero, "zero", (m,), torch.float32)
    layer = W8Layer._unwritten(m, n, codes.device)
    _call("sg_pack_w8", gpu, lib.sg_pack_w8, layer.codes.data_ptr(), layer.pitch, layer.offset.data_ptr(),
          layer.scale.data_ptr(), codes.data_ptr(), scale.data_ptr(), zero.data_ptr(), m, n)
    return layer


def sg_linear_w8a8(q: torch.Tensor, x_scale: torch.Tensor, x_sum: torch.Tensor, layer: W8Layer,
                   dtype: torch.dtype = torch.bfloat16, Y: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y [T, m] = X_hat W_hat^T as a product of 8-bit integers, from the codes of
    sg_quantize_tokens and a packed layer; ``dtype`` bfloat16 or float32."""
    lib = load_library()
    gpu = _same_gpu(q, x_scale, x_sum, layer.codes, Y, workspace)
    m, n = layer.m, layer.n
    T, _, ldq = _codes(q, "q", n)
    _shaped(x_scale, "x_scale", (T,), torch.float32)
    _shaped(x_sum, "x_sum", (T,), torch.int32)
    given = Y is not None
    Y, y_dtype, ldy = _out_rows(Y, "Y", T, m, dtype, q)
    _keep, ws, nb = _scratch(SG_OP_LINEAR_W8A8, m, n, T, q.device, workspace)
    _call("sg_linear_w8a8", gpu, lib.sg_linear_w8a8, Y.data_ptr(), y_dtype, ldy, q.data_ptr(), ldq,
          x_scale.data_ptr(), x_sum.data_ptr(), T, layer.codes.data_ptr(), layer.pitch, layer.offset.data_ptr(),
          layer.scale.data_ptr(), m, n, ws, nb)
    if given:
        _wrote(Y)
    return Y


def sg_linear_w8_grad_input(dY: torch.Tensor, layer: W8Layer, dtype: torch.dtype = torch.bfloat16,
                            dX: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dX [T, n] = dY bf16(W_hat) from a packed layer; dY [T, m] bf16."""
    lib = load_library()
    gpu = _same_gpu(dY, layer.codes, dX, workspace)
    m, n = layer.m, layer.n
    if dY.dim() != 2:
        raise ValueError("dY must be [T, m]")
    T = dY.shape[0]
    dy_dtype, lddy = _rows(dY, "dY", T, m)
    given = dX is not None
    dX, dx_dtype, lddx = _out_rows(dX, "dX", T, n, dtype, dY)
    _keep, ws, nb = _scratch(SG_OP_GRAD_INPUT, m, n, T, dY.device, workspace)
    _call("sg_linear_w8_grad_input", gpu, lib.sg_linear_w8_grad_input, dX.data_ptr(), dx_dtype, lddx,
          dY.data_ptr(), dy_dtype, lddy, T, layer.codes.data_ptr(), layer.pitch, layer.offset.data_ptr(),
          layer.scale.data_ptr(), m, n, ws, nb)
    if given:
        _wrote(dX)
    return dX


def sg_linear_w8_grad_weight(dY: torch.Tensor, q: torch.Tensor, x_scale: torch.Tensor,
                             mask: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
                             dW: Optional[torch.Tensor] = None, accumulate: bool = False,
                             workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dW [m, n] = dY^T X_hat from the layer's 8-bit checkpoint (q, x_scale), 0
    where mask [m, n] uint8 is 1 (pruned); dY [T, m] bf16.  ``accumulate`` adds
    to ``dW``."""
    lib = load_library()
    gpu = _same_gpu(dY, q, x_scale, mask, dW, workspace)
    if dY.dim() != 2:
        raise ValueError("dY must be [T, m]")
    T, m = dY.shape
    dy_dtype, lddy = _rows(dY, "dY", T, m)
    rows, n, ldq = _codes(q, "q")
    if rows != T:
        raise ValueError(f"q must have {T} rows")
    _shaped(x_scale, "x_scale", (T,), torch.float32)
    if mask is not None:
        _shaped(mask, "mask", (m, n), torch.uint8)
    if dW is None and accumulate:
        raise ValueError("accumulate needs dW")
    given = dW is not None
    dW, dw_dtype, lddw = _out_rows(dW, "dW", m, n, dtype, dY)
    _keep, ws, nb = _scratch(SG_OP_GRAD_WEIGHT, m, n, T, dY.device, workspace)
    _call("sg_linear_w8_grad_weight", gpu, lib.sg_linear_w8_grad_weight, dW.data_ptr(), dw_dtype, lddw,
          1 if accumulate else 0, dY.data_ptr(), dy_dtype, lddy, q.data_ptr(), ldq, x_scale.data_ptr(), T,
          None if mask is None else mask.data_ptr(), m, n, ws, nb)
    if given:
        _wrote(dW)
    return dW


def _as_rows(t):
    """[..., n] as row-major [rows, n], copied only where its strides need it
    (an expanded or transposed tensor, rows further apart than the library takes)."""
    if t.dim() != 2:
        t = t.reshape(-1, t.shape[-1])
    rows, n = t.shape
    if (n > 1 and t.stride(1) != 1) or \
            (rows > 1 and not n <= t.stride(0) <= SG_MAX_PITCH // t.element_size()):
        # (an empty tensor counts as contiguous whatever its strides are)
        t = t.contiguous() if rows > 0 else t.new_empty((rows, n))
    return t


def _versions(layer):
    """Counters that in-place changes of a layer's tensors raise (inference
    tensors have none)."""
    return tuple(0 if t.is_inference() else t._version for t in (layer.codes, layer.offset, layer.scale))


class _LinearW8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, W, layer, mask):
        q, x_scale, x_sum = sg_quantize_tokens(_as_rows(X))
        Y = sg_linear_w8a8(q, x_scale, x_sum, layer, dtype=X.dtype)
        # the codes are the checkpoint: X itself is not kept.  Their padding is,
        # for hooks that store saved tensors elsewhere and keep no strides
        pitch = q.stride(0)
        ctx.save_for_backward(q if pitch == q.shape[1] else q.as_strided((q.shape[0], pitch), (pitch, 1)), x_scale, mask)
        ctx.layer, ctx.versions = layer, _versions(layer)
        ctx.x_shape, ctx.x_dtype = X.shape, X.dtype
        ctx.w_dtype = None if W is None else W.dtype
        return Y if X.dim() == 2 else Y.view(*X.shape[:-1], Y.shape[1])

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY):
        q, x_scale, mask = ctx.saved_tensors
        if _versions(ctx.layer) != ctx.versions:
            raise RuntimeError("the layer of linear_w8 was changed in place between the forward and the backward pass")
        dY = _as_rows(dY)
        if q.shape[1] != ctx.layer.n:
            q = q[:, :ctx.layer.n]
        dX = dW = None
        if ctx.needs_input_grad[0]:
            dX = sg_linear_w8_grad_input(dY, ctx.layer, dtype=ctx.x_dtype).view(ctx.x_shape)
        if ctx.needs_input_grad[1]:
            dW = sg_linear_w8_grad_weight(dY, q, x_scale, mask, dtype=ctx.w_dtype)
        return dX, dW, None, None


def linear_w8(X: torch.Tensor, W: Optional[torch.Tensor], layer: W8Layer,
              mask: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The 8-bit linear layer for autograd: X [..., n] -> [..., m] in X's type.

    ``W`` [m, n] is the trained weight that the packed ``layer`` was quantized
    from (or None): its values are not read, its gradient is that of the
    layer's weights, 0 where ``mask`` is 1.  What is kept for the backward pass
    is X in 8 bits, and the layer, which must not change in between (an in-place
    change of its tensors by torch is an error of the backward pass).  Gradients
    need a bf16 X; there is no second derivative."""
    m, n = layer.m, layer.n
    if X.dim() < 1 or X.shape[-1] != n:
        raise ValueError(f"X must have {n} columns")
    if X.dtype not in _FLOATS:
        raise TypeError(f"unsupported dtype {X.dtype} (float32 or bfloat16)")
    if W is not None and (W.shape != (m, n) or W.dtype not in _FLOATS):
        raise ValueError(f"W must be [{m}, {n}] of float32 or bfloat16")
    if mask is not None:
        _shaped(mask, "mask", (m, n), torch.uint8)
    wants = torch.is_grad_enabled() and (X.requires_grad or (W is not None and W.requires_grad))
    if wants and X.dtype != torch.bfloat16:
        raise TypeError("gradients need a bfloat16 X")
    return _LinearW8.apply(X, W, layer, mask)


# ---------------------------------------------------------------------------
# Dropout and the linear layer in 8-bit floating point
# ---------------------------------------------------------------------------
class _DropStruct(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("state", ctypes.c_void_p)]


class Dropout:
    """A dropout by numbers from a counter: element (t, c) of a matrix is kept or
    dropped by (seed, offset, t, c) alone, so its mask is made anew wherever it
    is needed and never stored.  ``p`` in [0, 1) is the share that is dropped;
    kept elements are multiplied by 1 / (1 - p).  ``seed`` and ``offset`` are
    whole numbers (taken modulo 2^64); give every place and step an offset of
    its own.  ``state``, an int64 tensor [2] on the GPU, is added to (seed,
    offset) when the kernels run: a captured graph that advances it draws other
    numbers in every replay.  It must hold the same in the backward pass as in
    the forward pass.

    A Dropout does not change (a backward pass may still need it): for another p
    or offset make another.  A deep copy has a state of its own."""
    __slots__ = ("_p", "_seed", "_offset", "_state", "_struct", "_address")
    p, seed, offset, state = (property(operator.attrgetter(k)) for k in __slots__[:4])

    def __init__(self, p: float, seed: int, offset: int = 0, state: Optional[torch.Tensor] = None):
        p = float(p)
        if not 0.0 <= p < 1.0 or round(p * 2.0 ** 32) >= 2 ** 32:
            raise ValueError("p must lie in [0, 1 - 2^-32)")
        if state is not None:
            _shaped(state, "state", (2,), torch.int64)
            if not state.is_cuda:
                raise ValueError("state must live on the GPU")
        self._p, self._seed, self._offset, self._state = p, int(seed) % 2 ** 64, int(offset) % 2 ** 64, state
        self._struct = _DropStruct(p, self._seed, self._offset, None)
        self._address = ctypes.addressof(self._struct)

    def __reduce__(self):
        return type(self), (self._p, self._seed, self._offset, self._state)

    def _version(self):
        """What tells whether the state may have changed: its version and its memory."""
        state = self._state
        if state is None:
            return None
        return 0 if state.is_inference() else state._version, state.data_ptr()


def _drop_address(drop):
    if drop is None:
        return None
    if drop._state is not None:
        # (its memory may have been replaced since: state.data = ...)
        drop._struct.state = _shaped(drop._state, "state", (2,), torch.int64).data_ptr()
    return drop._address


def _drop_state(drop):
    return None if drop is None else drop._state


_F8_FORMATS = {torch.float8_e4m3fn: SG_E4M3, torch.float8_e5m2: SG_E5M2}


_CODE_DTYPES = {SG_F32: torch.float32, SG_BF16: torch.bfloat16}


def _f8_format(dtype):
    code = _F8_FORMATS.get(dtype)
    if code is None:
        raise ValueError("the format must be torch.float8_e4m3fn or torch.float8_e5m2")
    return code


@functools.lru_cache(maxsize=4096)
def _f8_room(rows, cols):
    """(pitch of the codes, offset of the scale bytes, their pitch, bytes) of a
    matrix in 8-bit floating point that lies in one piece of memory."""
    pitch = -(-cols // SG_F8_BLOCK) * SG_F8_BLOCK
    scale_pitch = -(-rows // SG_F8_SCALE_PITCH) * SG_F8_SCALE_PITCH
    size = rows * pitch
    return pitch, size, scale_pitch, size + -(-pitch // SG_F8_BLOCK * scale_pitch // SG_F8_BLOCK) * SG_F8_BLOCK


class F8Tensor:
    """A matrix in 8-bit floating point with a scale for every 128 neighbours of
    a row: ``codes`` [rows, cols] in torch.float8_e4m3fn or torch.float8_e5m2
    (a view of rows padded with zeros to a multiple of SG_F8_BLOCK bytes) and
    ``scale`` uint8 [ceil(cols / 128), rows] (a view of padded rows): element
    (r, c) stands for codes[r, c] * 2^(scale[c // 128, r] - 127).

    Tensors that are not laid out like that are copied.  Its parts are checked
    once, here, and are not to be replaced or resized."""
    __slots__ = ("rows", "cols", "pitch", "scale_pitch", "format", "dtype", "_codes", "_scale", "_store", "_gpu", "_args")

    def __init__(self, codes: torch.Tensor, scale: torch.Tensor):
        _f8_format(codes.dtype)
        if codes.dim() != 2:
            raise ValueError("codes must be a matrix")
        rows, cols = codes.shape
        blocks = -(-cols // SG_F8_BLOCK)
        if scale.dtype is not torch.uint8 or scale.shape != (blocks, rows):
            raise ValueError(f"scale must be [{blocks}, {rows}] of uint8")
        if not codes.is_cuda or codes.device != scale.device:
            raise ValueError("codes and scale must live on one GPU")
        if cols % SG_F8_BLOCK or codes.stride(1) != 1 or codes.stride(0) % SG_F8_BLOCK or codes.stride(0) < cols \
                or codes.stride(0) > SG_MAX_PITCH or codes.data_ptr() % 16:
            wide = torch.zeros(rows, blocks * SG_F8_BLOCK, dtype=torch.uint8, device=codes.device)
            wide[:, :cols].copy_(codes.view(torch.uint8))
            codes = wide.view(codes.dtype)[:, :cols]
        # the last row of scale bytes is read up to its padded width too
        pad = -(-rows // SG_F8_SCALE_PITCH) * SG_F8_SCALE_PITCH
        if scale.data_ptr() % 16 or (rows > 1 and scale.stride(1) != 1) or scale.stride(0) % SG_F8_SCALE_PITCH \
                or scale.stride(0) < pad or \
                scale.storage_offset() + (blocks - 1) * scale.stride(0) + pad > scale.untyped_storage().nbytes():
            wide = torch.zeros(blocks, pad, dtype=torch.uint8, device=scale.device)
            wide[:, :rows].copy_(scale)
            scale = wide[:, :rows]
        self._take(codes, scale)

    @classmethod
    def _unwritten(cls, rows, cols, dtype, like, store=None):
        """A matrix on like's GPU that a call is about to write (or one that
        ``store`` holds), in one piece of memory: its two tensors are made when they
        are asked for."""
        t = cls.__new__(cls)
        t.rows, t.cols = rows, cols
        t.pitch, size, t.scale_pitch, total = _f8_room(rows, cols)
        t.dtype, t.format = dtype, _F8_FORMATS[dtype]
        t._codes = t._scale = None
        t._store = like.new_empty(total, dtype=torch.uint8) if store is None else store
        t._gpu = t._store.get_device()
        address = t._store.data_ptr()
        t._args = address, t.pitch, address + size, t.scale_pitch
        return t

    @classmethod
    def _of(cls, wide, wide_scale, rows, cols, dtype=None):
        """The matrix whose padded codes (bytes of ``dtype``) and scale are whole tensors."""
        t = cls.__new__(cls)
        if dtype is not None:
            wide = wide.view(dtype)
        t._take(wide if wide.shape[1] == cols else wide[:, :cols],
                wide_scale if wide_scale.shape[1] == rows else wide_scale[:, :rows])
        return t

    def _take(self, codes, scale):
        self._codes, self._scale, self._store = codes, scale, None
        self.rows, self.cols = codes.shape
        # (a stride says nothing where there is a single row, or nothing at all)
        pitch, _, scale_pitch, _ = _f8_room(self.rows, self.cols)
        self.pitch = codes.stride(0) if self.rows > 1 and self.cols > 0 else pitch
        self.scale_pitch = scale.stride(0) if scale.shape[0] > 1 and self.rows > 0 else scale_pitch
        self.dtype, self.format = codes.dtype, _F8_FORMATS[codes.dtype]
        self._gpu = codes.get_device()
        # what the calls take of it
        self._args = codes.data_ptr(), self.pitch, scale.data_ptr(), self.scale_pitch

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            wide = self._store[:self.rows * self.pitch].view(self.dtype).view(self.rows, self.pitch)
            self._codes = wide if self.pitch == self.cols else wide[:, :self.cols]
        return self._codes

    @property
    def scale(self) -> torch.Tensor:
        if self._scale is None:
            blocks = -(-self.cols // SG_F8_BLOCK)
            size = self.rows * self.pitch
            wide = self._store[size:size + blocks * self.scale_pitch].view(blocks, self.scale_pitch)
            self._scale = wide if self.scale_pitch == self.rows else wide[:, :self.rows]
        return self._scale

    def __reduce__(self):
        # (a copy takes addresses of its own)
        if self._store is not None:
            return F8Tensor._unwritten, (self.rows, self.cols, self.dtype, None, self._store)
        codes, scale = self._wide()  # (as bytes: torch pickles no storage of this type)
        return F8Tensor._of, (codes.view(torch.uint8), scale, self.rows, self.cols, self.dtype)

    def _any(self):
        """A tensor of the same GPU."""
        return self._codes if self._store is None else self._store

    def _written(self):
        """A call wrote into it: autograd is told, as it may have kept it."""
        for t in (self._codes, self._scale) if self._store is None else (self._store,):
            _wrote(t)

    def _wide(self):
        """(codes, scale) with their padding, as autograd may store them elsewhere."""
        pad, _, spad, _ = _f8_room(self.rows, self.cols)
        codes, scale = self.codes, self.scale
        if codes.shape[1] != pad:
            codes = codes.as_strided((self.rows, pad), (self.pitch, 1))
        if scale.shape[1] != spad:
            scale = scale.as_strided((scale.shape[0], spad), (self.scale_pitch, 1))
        return codes, scale


class F8Layer:
    """A layer's weights [m, n] in 8-bit floating point as sg_pack_f8 leaves
    them: ``w``, an e4m3 F8Tensor [m, n], and, for the input gradient, ``wt``,
    the same values transposed [n, m] (or None).  Its parts are not replaced;
    sg_pack_f8(W, layer=layer) writes them anew."""
    __slots__ = ("_w", "_wt", "_m", "_n")
    w, wt, m, n = (property(operator.attrgetter(k)) for k in __slots__)

    def __init__(self, w: F8Tensor, wt: Optional[F8Tensor] = None):
        for t in (w, wt):
            if t is not None and t.format != SG_E4M3:
                raise ValueError("a layer's weights are held in torch.float8_e4m3fn")
        if wt is not None and (wt.rows, wt.cols) != (w.cols, w.rows):
            raise ValueError(f"wt must be [{w.cols}, {w.rows}]")
        if wt is not None:
            _one_gpu(w._gpu, wt)
        self._w, self._wt, self._m, self._n = w, wt, w.rows, w.cols


_NO_F8 = (None, 0, None, 0)


def _one_gpu(index, *matrices):
    """``index``, if the F8Tensors live there too."""
    for t in matrices:
        if t is not None and t._gpu != index:
            raise ValueError("tensors must live on one GPU")
    return index


def sg_dropout(X: torch.Tensor, drop: Dropout, residual: Optional[torch.Tensor] = None,
               Y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """drop(X) (+ residual) of a matrix X [T, n] (bf16 or fp32), in X's type.
    ``Y`` may be X or the residual itself."""
    lib = load_library()
    gpu = _same_gpu(X, residual, Y, drop._state)
    if X.dim() != 2:
        raise ValueError("X must be [T, n]")
    T, n = X.shape
    x_dtype, ldx = _rows(X, "X", T, n)
    ldr = n
    if residual is not None:
        r_dtype, ldr = _rows(residual, "residual", T, n)
        if r_dtype != x_dtype:
            raise ValueError("the residual must have X's type")
    given = Y is not None
    Y, y_dtype, ldy = _out_rows(Y, "Y", T, n, X.dtype, X)
    if y_dtype != x_dtype:
        raise ValueError("Y must have X's type")
    _call("sg_dropout", gpu, lib.sg_dropout, Y.data_ptr(), ldy, X.data_ptr(), x_dtype, ldx,
          None if residual is None else residual.data_ptr(), ldr, T, n, _drop_address(drop))
    if given:
        _wrote(Y)
    return Y


def sg_quantize_f8(X: torch.Tensor, dtype: torch.dtype = torch.float8_e4m3fn, form: str = "rows",
                   drop: Optional[Dropout] = None, q: Optional[F8Tensor] = None, qt: Optional[F8Tensor] = None):
    """X [T, n] (bf16 or fp32) in 8-bit floating point, after a dropout if one is
    given.  ``form`` "rows": an F8Tensor [T, n] with a scale for 128 neighbours
    of a token, the operand of sg_linear_f8 and sg_linear_f8_grad_input;
    "columns": an F8Tensor [n, T] of the transposed matrix with a scale for 128
    tokens of a channel, what sg_linear_f8_grad_weight takes; "both": the two,
    from one reading of X.  ``q`` (not with "columns") and ``qt`` (not with "rows")
    are written if they are given."""
    lib = load_library()
    code = _f8_format(dtype)
    if form not in ("rows", "columns", "both"):
        raise ValueError('form must be "rows", "columns" or "both"')
    if (form == "columns" and q is not None) or (form == "rows" and qt is not None):
        raise ValueError(f'form "{form}" does not write the other one')
    if X.dim() != 2:
        raise ValueError("X must be [T, n]")
    T, n = X.shape
    x_dtype, ldx = _rows(X, "X", T, n)
    given = q, qt
    if q is None:
        q = None if form == "columns" else F8Tensor._unwritten(T, n, dtype, X)
    elif (q.rows, q.cols, q.format) != (T, n, code):
        raise ValueError(f"q must be [{T}, {n}] in {dtype}")
    if qt is None:
        qt = None if form == "rows" else F8Tensor._unwritten(n, T, dtype, X)
    elif (qt.rows, qt.cols, qt.format) != (n, T, code):
        raise ValueError(f"qt must be [{n}, {T}] in {dtype}")
    gpu = _one_gpu(_same_gpu(X, _drop_state(drop)), q, qt)
    _call("sg_quantize_f8", gpu, lib.sg_quantize_f8, *(_NO_F8 if q is None else q._args),
          *(_NO_F8 if qt is None else qt._args), code, X.data_ptr(), x_dtype, T, n, ldx, _drop_address(drop))
    for t in given:
        if t is not None:
            t._written()
    return q if qt is None else qt if q is None else (q, qt)


def sg_dequantize_f8(q: F8Tensor, dtype: torch.dtype = torch.bfloat16,
                     X_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The [rows, cols] tensor that an F8Tensor stands for, in ``dtype``
    (bfloat16 or float32)."""
    lib = load_library()
    given = X_out is not None
    X_out, x_dtype, ldx = _out_rows(X_out, "X_out", q.rows, q.cols, dtype, q._any())
    gpu = _one_gpu(_same_gpu(X_out), q)
    _call("sg_dequantize_f8", gpu, lib.sg_dequantize_f8, X_out.data_ptr(), x_dtype, ldx, *q._args, q.format, q.rows,
          q.cols)
    if given:
        _wrote(X_out)
    return X_out


def sg_pack_f8(W: torch.Tensor, transposed: bool = True, layer: Optional[F8Layer] = None) -> F8Layer:
    """The weights W [m, n] (bf16 or fp32; pruned ones 0) in e4m3 with a scale for
    every 128 x 128, for the calls below; ``transposed`` False leaves out what
    only the input gradient needs.  If ``layer`` is given it is written anew, in the
    forms that it has."""
    lib = load_library()
    if W.dim() != 2:
        raise ValueError("W must be [m, n]")
    m, n = W.shape
    w_dtype, ld = _rows(W, "W", m, n)
    again = layer is not None
    if layer is None:
        e4m3 = torch.float8_e4m3fn
        layer = F8Layer(F8Tensor._unwritten(m, n, e4m3, W),
                        F8Tensor._unwritten(n, m, e4m3, W) if transposed else None)
    elif (layer.m, layer.n) != (m, n):
        raise ValueError(f"layer must be [{m}, {n}]")
    w, wt = layer.w, layer.wt
    gpu = _one_gpu(_same_gpu(W), w, wt)
    _call("sg_pack_f8", gpu, lib.sg_pack_f8, *w._args, *(_NO_F8 if wt is None else wt._args), W.data_ptr(), w_dtype, m,
          n, ld)
    if again:
        w._written()
        if wt is not None:
            wt._written()
    return layer


def sg_linear_f8(q: F8Tensor, layer: F8Layer, dtype: torch.dtype = torch.bfloat16, Y: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y [T, m] = X_hat W_hat^T from the rows of sg_quantize_f8 and a packed
    layer; ``dtype`` bfloat16 or float32.  With float32 every product is exact and
    sums are in 32 bits, at half the rate.  With bfloat16 the matrix cores cut every
    eight products to 13 bits below the largest, toward zero: far below
    bfloat16's rounding unless products cancel to a small rest (include/sg.h has the
    bound).  Exact products in bfloat16: ask for float32 and round.  The same
    holds for the two gradients."""
    lib = load_library()
    w = layer.w
    m, n, T = layer.m, layer.n, q.rows
    if q.cols != n:
        raise ValueError(f"q must have {n} columns")
    given = Y is not None
    Y, y_dtype, ldy = _out_rows(Y, "Y", T, m, dtype, q._any())
    gpu = _one_gpu(_same_gpu(Y, workspace), q, w)
    _keep, ws, nb = _scratch(SG_OP_LINEAR_F8, m, n, T, Y.device, workspace)
    _call("sg_linear_f8", gpu, lib.sg_linear_f8, Y.data_ptr(), y_dtype, ldy, *q._args, q.format, T, *w._args, m, n, ws,
          nb)
    if given:
        _wrote(Y)
    return Y


def sg_linear_f8_grad_input(dy: F8Tensor, layer: F8Layer, dtype: torch.dtype = torch.bfloat16,
                            drop: Optional[Dropout] = None, dX: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dX [T, n] = drop(dY_hat W_hat) from the rows of sg_quantize_f8(dY) and a
    packed layer; ``drop`` is the dropout that the layer's input went through."""
    lib = load_library()
    wt = layer.wt
    if wt is None:
        raise ValueError("the layer was packed without its transposed form")
    m, n, T = layer.m, layer.n, dy.rows
    if dy.cols != m:
        raise ValueError(f"dy must have {m} columns")
    given = dX is not None
    dX, dx_dtype, lddx = _out_rows(dX, "dX", T, n, dtype, dy._any())
    gpu = _one_gpu(_same_gpu(dX, workspace, _drop_state(drop)), dy, wt)
    _keep, ws, nb = _scratch(SG_OP_F8_GRAD_INPUT, m, n, T, dX.device, workspace)
    _call("sg_linear_f8_grad_input", gpu, lib.sg_linear_f8_grad_input, dX.data_ptr(), dx_dtype, lddx, *dy._args,
          dy.format, T, *wt._args, m, n, _drop_address(drop), ws, nb)
    if given:
        _wrote(dX)
    return dX


def sg_linear_f8_grad_weight(dyt: F8Tensor, xt: F8Tensor, mask: Optional[torch.Tensor] = None,
                             dtype: torch.dtype = torch.bfloat16, dW: Optional[torch.Tensor] = None,
                             accumulate: bool = False, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dW [m, n] = dY_hat^T X_hat from the columns of sg_quantize_f8(dY) and of
    the layer's input (in e4m3), 0 where mask [m, n] uint8 is 1 (pruned).
    ``accumulate`` adds to ``dW``."""
    lib = load_library()
    m, n, T = dyt.rows, xt.rows, xt.cols
    if dyt.cols != T:
        raise ValueError(f"dyt must have {T} columns")
    if xt.format != SG_E4M3:
        raise ValueError("xt must be held in torch.float8_e4m3fn")
    if mask is not None:
        _shaped(mask, "mask", (m, n), torch.uint8)
    if dW is None and accumulate:
        raise ValueError("accumulate needs dW")
    given = dW is not None
    dW, dw_dtype, lddw = _out_rows(dW, "dW", m, n, dtype, xt._any())
    gpu = _one_gpu(_same_gpu(dW, mask, workspace), dyt, xt)
    _keep, ws, nb = _scratch(SG_OP_F8_GRAD_WEIGHT, m, n, T, dW.device, workspace)
    _call("sg_linear_f8_grad_weight", gpu, lib.sg_linear_f8_grad_weight, dW.data_ptr(), dw_dtype, lddw,
          1 if accumulate else 0, *dyt._args, dyt.format, *xt._args, T, None if mask is None else mask.data_ptr(), m, n,
          ws, nb)
    if given:
        _wrote(dW)
    return dW


def _same_state(drop, version):
    if drop is not None and drop._version() != version:
        raise RuntimeError("the dropout's state was changed between the forward and the backward pass")


def _f8_at(address, rows, cols):
    """The pointer and pitch arguments of such a matrix at an address."""
    pitch, size, scale_pitch, _ = _f8_room(rows, cols)
    return address, pitch, address + size, scale_pitch


class _LinearF8(torch.autograd.Function):
    # The calls of sg_quantize_f8, sg_pack_f8 and so on without their objects: the
    # matrices between them lie in one tensor that goes and one that is kept.
    @staticmethod
    def forward(ctx, X, W, layer, mask, drop, grad_dtype, grad):
        lib = load_library()
        # (needs_input_grad tells what requires a gradient under no_grad too)
        need_x, need_w = grad and ctx.needs_input_grad[0], grad and ctx.needs_input_grad[1]
        rows = _as_rows(X)
        T, n = rows.shape
        x_dtype, ldx = _rows(rows, "X", T, n)
        if layer is None:
            weights = _as_rows(W)
            m = weights.shape[0]
            w_dtype, ldw = _rows(weights, "W", m, n)
            gpu = _same_gpu(rows, weights, mask, _drop_state(drop))
        else:
            m = layer.m
            if need_x and layer.wt is None:
                raise ValueError("the layer was packed without its transposed form")
            gpu = _same_gpu(rows, W, layer.w.codes, mask, _drop_state(drop))
        size_q = _f8_room(T, n)[3]
        brief = torch.empty(size_q + (_f8_room(m, n)[3] if layer is None else 0), dtype=torch.uint8, device=X.device)
        at = brief.data_ptr()
        size_xt = _f8_room(n, T)[3] if need_w else 0
        own_wt = need_x and layer is None
        kept, xt, wt = None, _NO_F8, _NO_F8
        if need_w or own_wt:
            kept = torch.empty(size_xt + (_f8_room(n, m)[3] if own_wt else 0), dtype=torch.uint8, device=X.device)
            if need_w:
                xt = _f8_at(kept.data_ptr(), n, T)
            if own_wt:
                wt = _f8_at(kept.data_ptr() + size_xt, n, m)
        q = _f8_at(at, T, n)
        _call("sg_quantize_f8", gpu, lib.sg_quantize_f8, *q, *xt, SG_E4M3, rows.data_ptr(), x_dtype, T, n, ldx,
              _drop_address(drop))
        if layer is None:
            w = _f8_at(at + size_q, m, n)
            _call("sg_pack_f8", gpu, lib.sg_pack_f8, *w, *wt, weights.data_ptr(), w_dtype, m, n, ldw)
        else:
            w = layer.w._args
        Y = rows.new_empty((T, m))
        _keep, ws, nb = _scratch(SG_OP_LINEAR_F8, m, n, T, X.device, None)
        _call("sg_linear_f8", gpu, lib.sg_linear_f8, Y.data_ptr(), x_dtype, m, *q, SG_E4M3, T, *w, m, n, ws, nb)
        given = layer.wt._wide() if need_x and layer is not None else (None, None)
        ctx.save_for_backward(kept, mask, *given)
        ctx.sizes, ctx.gpu, ctx.x_shape, ctx.x_code = (T, m, n), gpu, X.shape, x_dtype
        ctx.w_dtype = None if W is None else W.dtype
        ctx.drop, ctx.version, ctx.grad_dtype = drop, None if drop is None else drop._version(), grad_dtype
        return Y if X.dim() == 2 else Y.view(*X.shape[:-1], m)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY):
        lib = load_library()
        kept, mask, wt_codes, wt_scale = ctx.saved_tensors
        _same_state(ctx.drop, ctx.version)
        (T, m, n), gpu = ctx.sizes, ctx.gpu
        need_x, need_w = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        rows = _as_rows(dY)
        dy_dtype, lddy = _rows(rows, "dY", T, m)
        if rows.get_device() != gpu:
            raise ValueError("tensors must live on one GPU")
        code, device = _F8_FORMATS[ctx.grad_dtype], rows.device
        size = _f8_room(T, m)[3] if need_x else 0
        brief = torch.empty(size + (_f8_room(m, T)[3] if need_w else 0), dtype=torch.uint8, device=device)
        dy = _f8_at(brief.data_ptr(), T, m) if need_x else _NO_F8
        dyt = _f8_at(brief.data_ptr() + size, m, T) if need_w else _NO_F8
        _call("sg_quantize_f8", gpu, lib.sg_quantize_f8, *dy, *dyt, code, rows.data_ptr(), dy_dtype, T, m, lddy, None)
        dX = dW = None
        size_xt = _f8_room(n, T)[3] if need_w else 0
        if need_x:
            # (hooks may have moved what was saved: addresses are taken anew)
            if wt_codes is not None:
                wt = F8Tensor._of(wt_codes, wt_scale, n, m)._args
            else:
                wt = _f8_at(kept.data_ptr() + size_xt, n, m)
            dX = torch.empty((T, n), dtype=_CODE_DTYPES[ctx.x_code], device=device)
            _keep, ws, nb = _scratch(SG_OP_F8_GRAD_INPUT, m, n, T, device, None)
            _call("sg_linear_f8_grad_input", gpu, lib.sg_linear_f8_grad_input, dX.data_ptr(), ctx.x_code, n, *dy, code, T,
                  *wt, m, n, _drop_address(ctx.drop), ws, nb)
            dX = dX.view(ctx.x_shape)
        if need_w:
            dW = torch.empty((m, n), dtype=ctx.w_dtype, device=device)
            _keep, ws, nb = _scratch(SG_OP_F8_GRAD_WEIGHT, m, n, T, device, None)
            _call("sg_linear_f8_grad_weight", gpu, lib.sg_linear_f8_grad_weight, dW.data_ptr(),
                  SG_F32 if ctx.w_dtype is torch.float32 else SG_BF16, n, 0, *dyt, code, *_f8_at(kept.data_ptr(), n, T), T,
                  None if mask is None else mask.data_ptr(), m, n, ws, nb)
        return dX, dW, None, None, None, None, None


def linear_f8(X: torch.Tensor, W: Optional[torch.Tensor], layer: Optional[F8Layer] = None,
              mask: Optional[torch.Tensor] = None, drop: Optional[Dropout] = None,
              grad_dtype: torch.dtype = torch.float8_e4m3fn) -> torch.Tensor:
    """The linear layer in 8-bit floating point for autograd: X [..., n], which
    goes through ``drop`` first, -> [..., m] in X's type.

    ``W`` [m, n] is the weight that is trained; ``layer`` is its packed form
    (sg_pack_f8), made here if it is not given, and then W may be None if no
    weight gradient is wanted.  The gradient of W is 0 where ``mask`` [m, n]
    uint8 is 1 (pruned); W itself has to hold zeros there.  Gradients are
    quantized to ``grad_dtype``.  What is kept for the backward pass is X in 8 bits, and the
    transposed weights in 8 bits; under torch.no_grad() neither is made.  There is no
    second derivative.

    Y and the gradient of X have X's type, the gradient of W has W's, and products go
    by that: exact for float32, cut for bfloat16 as sg_linear_f8 describes.

    A step can be captured in a graph with torch.autograd.grad; ``backward()``
    under capture needs that no eager graph of the same leaves is alive (torch
    would wait for the leaves' other stream, which a capture forbids)."""
    if W is None and layer is None:
        raise ValueError("W or its packed layer is needed")
    m, n = W.shape if layer is None else (layer.m, layer.n)
    if X.dim() < 1 or X.shape[-1] != n:
        raise ValueError(f"X must have {n} columns")
    if X.dtype not in _FLOATS:
        raise TypeError(f"unsupported dtype {X.dtype} (float32 or bfloat16)")
    if W is not None and (W.shape != (m, n) or W.dtype not in _FLOATS):
        raise ValueError(f"W must be [{m}, {n}] of float32 or bfloat16")
    if mask is not None:
        _shaped(mask, "mask", (m, n), torch.uint8)
    _f8_format(grad_dtype)
    return _LinearF8.apply(X, W, layer, mask, drop, grad_dtype, torch.is_grad_enabled())


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, drop, residual):
        ctx.drop, ctx.version = drop, drop._version()
        Y = sg_dropout(_as_rows(X), drop, None if residual is None else _as_rows(residual))
        return Y.view(X.shape)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY):
        _same_state(ctx.drop, ctx.version)
        dX = sg_dropout(_as_rows(dY), ctx.drop).view(dY.shape) if ctx.needs_input_grad[0] else None
        return dX, None, dY if ctx.needs_input_grad[2] else None


def dropout(X: torch.Tensor, drop: Dropout, residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """drop(X) (+ residual) for autograd: X [..., n] of any strides, its leading
    dimensions taken as rows.  No mask is stored: the backward pass makes it
    anew.  There is no second derivative."""
    if X.dim() < 1:
        raise ValueError("X must have at least one dimension")
    if X.dtype not in _FLOATS:
        raise TypeError(f"unsupported dtype {X.dtype} (float32 or bfloat16)")
    if residual is not None and (residual.shape != X.shape or residual.dtype != X.dtype):
        raise ValueError("the residual must have X's shape and type")
    return _Dropout.apply(X, drop, residual)


def solve_layer(W: torch.Tensor, x_chunks, pattern, blocksize: int = 128, damp: float = 0.01):
    """a1..a7 for one layer: Hessian over all chunks, factor, prune.  A chunk is
    a tensor [T, n], or an 8-bit checkpoint of one: the (q, scale) or
    (q, scale, total) of sg_quantize_tokens, or the rows of sg_quantize_f8, which
    read back in bf16."""
    n = W.shape[1]
    H = torch.zeros(n, n, dtype=torch.float32, device=W.device)
    for Xc in x_chunks:
        if isinstance(Xc, F8Tensor):
            wide = torch.empty(Xc.rows, -(-n // 8) * 8, dtype=torch.bfloat16, device=W.device)
            Xc = sg_dequantize_f8(Xc, X_out=wide[:, :n])
        elif isinstance(Xc, (tuple, list)):
            # rows of whole 16-byte pieces, as the Hessian reads them
            wide = torch.empty(Xc[0].shape[0], -(-n // 8) * 8, dtype=torch.bfloat16, device=W.device)
            Xc = sg_dequantize_tokens(Xc[0], Xc[1], X_out=wide[:, :n])
        sg_hessian_accumulate(H, Xc)
    Hinv, info = sg_prepare_hinv(H, damp)
    W_hat, mask = sg_prune_layer(W, Hinv, pattern, blocksize)
    return {"H": H, "Hinv": Hinv, "info": info, "W_hat": W_hat, "mask": mask}
