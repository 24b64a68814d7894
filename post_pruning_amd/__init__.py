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
"""

from __future__ import annotations

import ctypes
import functools
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
    return q, scale, total


def sg_dequantize_tokens(q: torch.Tensor, scale: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                         X_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The [T, n] tensor that the codes of sg_quantize_tokens stand for, in
    ``dtype`` (bfloat16 or float32)."""
    lib = load_library()
    gpu = _same_gpu(q, scale, X_out)
    T, n, ldq = _codes(q, "q")
    _shaped(scale, "scale", (T,), torch.float32)
    X_out, x_dtype, ldx = _out_rows(X_out, "X_out", T, n, dtype, q)
    _call("sg_dequantize_tokens", gpu, lib.sg_dequantize_tokens, X_out.data_ptr(), x_dtype, ldx,
          q.data_ptr(), ldq, scale.data_ptr(), T, n)
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
    Y, y_dtype, ldy = _out_rows(Y, "Y", T, m, dtype, q)
    _keep, ws, nb = _scratch(SG_OP_LINEAR_W8A8, m, n, T, q.device, workspace)
    _call("sg_linear_w8a8", gpu, lib.sg_linear_w8a8, Y.data_ptr(), y_dtype, ldy, q.data_ptr(), ldq,
          x_scale.data_ptr(), x_sum.data_ptr(), T, layer.codes.data_ptr(), layer.pitch, layer.offset.data_ptr(),
          layer.scale.data_ptr(), m, n, ws, nb)
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
    dX, dx_dtype, lddx = _out_rows(dX, "dX", T, n, dtype, dY)
    _keep, ws, nb = _scratch(SG_OP_GRAD_INPUT, m, n, T, dY.device, workspace)
    _call("sg_linear_w8_grad_input", gpu, lib.sg_linear_w8_grad_input, dX.data_ptr(), dx_dtype, lddx,
          dY.data_ptr(), dy_dtype, lddy, T, layer.codes.data_ptr(), layer.pitch, layer.offset.data_ptr(),
          layer.scale.data_ptr(), m, n, ws, nb)
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
    dW, dw_dtype, lddw = _out_rows(dW, "dW", m, n, dtype, dY)
    _keep, ws, nb = _scratch(SG_OP_GRAD_WEIGHT, m, n, T, dY.device, workspace)
    _call("sg_linear_w8_grad_weight", gpu, lib.sg_linear_w8_grad_weight, dW.data_ptr(), dw_dtype, lddw,
          1 if accumulate else 0, dY.data_ptr(), dy_dtype, lddy, q.data_ptr(), ldq, x_scale.data_ptr(), T,
          None if mask is None else mask.data_ptr(), m, n, ws, nb)
    return dW


def _as_rows(t):
    """[..., n] as row-major [rows, n], copied only where its strides need it
    (an expanded or transposed tensor, rows further apart than the library takes)."""
    if t.dim() != 2:
        t = t.reshape(-1, t.shape[-1])
    rows, n = t.shape
    if (n > 1 and t.stride(1) != 1) or \
            (rows > 1 and not n <= t.stride(0) <= SG_MAX_PITCH // t.element_size()):
        t = t.contiguous()
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


def solve_layer(W: torch.Tensor, x_chunks, pattern, blocksize: int = 128, damp: float = 0.01):
    """a1..a7 for one layer: Hessian over all chunks, factor, prune.  A chunk is
    a tensor [T, n], or an 8-bit checkpoint of one: the (q, scale) or
    (q, scale, total) of sg_quantize_tokens, which reads back in bf16."""
    n = W.shape[1]
    H = torch.zeros(n, n, dtype=torch.float32, device=W.device)
    for Xc in x_chunks:
        if isinstance(Xc, (tuple, list)):
            # rows of whole 16-byte pieces, as the Hessian reads them
            wide = torch.empty(Xc[0].shape[0], -(-n // 8) * 8, dtype=torch.bfloat16, device=W.device)
            Xc = sg_dequantize_tokens(Xc[0], Xc[1], X_out=wide[:, :n])
        sg_hessian_accumulate(H, Xc)
    Hinv, info = sg_prepare_hinv(H, damp)
    W_hat, mask = sg_prune_layer(W, Hinv, pattern, blocksize)
    return {"H": H, "Hinv": Hinv, "info": info, "W_hat": W_hat, "mask": mask}
