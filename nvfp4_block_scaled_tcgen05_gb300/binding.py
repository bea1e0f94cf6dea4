"""Thin Python binding over the C ABI in include/gb300gemm.h.

Argument marshalling only: every function checks dtypes/shapes/devices of
the torch tensors it is given, passes their device pointers and the current
CUDA stream to the C entry point of the same name, and raises GemmError on
a non-zero status.  All arithmetic runs in the library's CUDA kernels; there
is no fallback path.  A missing library raises immediately.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import NamedTuple

import torch

from . import build as _build

_lock = threading.Lock()
_lib = None

STATUS = {
    0: "GEMM_OK", 1: "GEMM_ERR_NULL", 2: "GEMM_ERR_SHAPE", 3: "GEMM_ERR_ALIGN",
    4: "GEMM_ERR_ALIAS", 5: "GEMM_ERR_ARCH", 6: "GEMM_ERR_LAUNCH", 7: "GEMM_ERR_TIMEOUT",
    8: "GEMM_ERR_NO_DEVICE", 9: "GEMM_ERR_CAPTURE",
}
EXPORTS = ("gemm_bf16_nt", "gemm_bf16_nn", "gemm_bf16_nt_scaled_acc", "gemm_bf16_nt_ordered", "gemm_nvfp4_bs",
           "gemm_bf16_nt_splitk", "gemm_bf16_nt_streamk", "gemm_nvfp4_bs_splitk", "gemm_w4a16", "gemm_w4a16_t", "gemm_w4a16_ws",
           "gemm_bf16_nt_xent", "gemm_bf16_nt_xent_backward", "router_topk", "router_topk_backward",
           "gemm_bf16_nt_gated", "gemm_bf16_nt_gated_backward", "gemm_bf16_tn",
           "residual_norm", "residual_norm_backward", "gemv_w4a16", "gemv_w4a16_gated",
           "bf16_scaled_add", "gemm_get_device_status", "gemm_selftest_wait_timeout",
           "gemm_testing_set_overrides", "gemm_status_string")


class GemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def library_path() -> str:
    return _build.LIB


def load() -> ctypes.CDLL:
    """Load libgb300gemm.so (built in-tree); raises if it is missing."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: build the CUDA library first "
                    "(python -c 'import __graft_entry__ as g; g.build()')")
            lib = ctypes.CDLL(path)
            vp, i, f, l = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_long
            lib.gemm_bf16_nt.argtypes = [vp, vp, vp, i, i, i, vp]
            lib.gemm_bf16_nn.argtypes = [vp, vp, vp, i, i, i, vp]
            lib.gemm_bf16_nt_scaled_acc.argtypes = [vp, vp, vp, i, i, i, f, vp]
            lib.gemm_bf16_nt_ordered.argtypes = [vp, vp, vp, i, i, i, vp]
            lib.gemm_nvfp4_bs.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, vp]
            lib.bf16_scaled_add.argtypes = [vp, vp, f, l, vp]
            lib.gemm_bf16_nt_splitk.argtypes = [vp, vp, vp, vp, ctypes.c_size_t, i, i, i, i, vp]
            lib.gemm_bf16_nt_splitk_workspace_bytes.argtypes = [i, i, i, i]
            lib.gemm_bf16_nt_splitk_workspace_bytes.restype = ctypes.c_size_t
            lib.gemm_bf16_nt_streamk.argtypes = [vp, vp, vp, vp, ctypes.c_size_t, i, i, i, vp]
            lib.gemm_w4a16.argtypes = [vp, vp, vp, f, vp, i, i, i, vp]
            lib.gemm_w4a16_t.argtypes = [vp, vp, vp, f, vp, i, i, i, i, vp]
            lib.gemm_w4a16_ws.argtypes = [vp, vp, vp, f, vp, vp, ctypes.c_size_t, i, i, i, vp]
            lib.gemm_w4a16_ws_workspace_bytes.argtypes = [i, i]
            lib.gemm_w4a16_ws_workspace_bytes.restype = ctypes.c_size_t
            lib.gemm_bf16_nt_streamk_workspace_bytes.argtypes = []
            lib.gemm_bf16_nt_streamk_workspace_bytes.restype = ctypes.c_size_t
            lib.gemm_nvfp4_bs_splitk.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.c_size_t,
                                                 i, i, i, i, i, vp]
            lib.gemm_nvfp4_bs_splitk_workspace_bytes.argtypes = [i, i, i, i]
            lib.gemm_nvfp4_bs_splitk_workspace_bytes.restype = ctypes.c_size_t
            lib.gemm_bf16_nt_xent.argtypes = [vp] * 6 + [ctypes.c_size_t] + [i] * 3 + [vp]
            lib.gemm_bf16_nt_xent_workspace_bytes.argtypes = [i, i]
            lib.gemm_bf16_nt_xent_workspace_bytes.restype = ctypes.c_size_t
            lib.gemm_bf16_nt_xent_backward.argtypes = [vp] * 8 + [ctypes.c_size_t] + [i] * 3 + [vp]
            lib.gemm_bf16_nt_xent_backward_workspace_bytes.argtypes = [i] * 3
            lib.gemm_bf16_nt_xent_backward_workspace_bytes.restype = ctypes.c_size_t
            lib.router_topk.argtypes = [vp] * 9 + [ctypes.c_size_t] + [i] * 5 + [vp]
            lib.router_topk_workspace_bytes.argtypes = [i, i]
            lib.router_topk_workspace_bytes.restype = ctypes.c_size_t
            lib.router_topk_backward.argtypes = [vp] * 7 + [i] * 6 + [vp]
            lib.gemm_bf16_nt_gated.argtypes = [vp] * 5 + [i] * 4 + [vp]
            lib.gemm_bf16_nt_gated_backward.argtypes = [vp] * 9 + [ctypes.c_size_t] + [i] * 4 + [vp]
            lib.gemm_bf16_nt_gated_backward_workspace_bytes.argtypes = [i] * 3
            lib.gemm_bf16_nt_gated_backward_workspace_bytes.restype = ctypes.c_size_t
            lib.gemm_bf16_tn.argtypes = [vp] * 4 + [ctypes.c_size_t] + [i] * 3 + [vp]
            lib.gemm_bf16_tn_workspace_bytes.argtypes = [i] * 3
            lib.gemm_bf16_tn_workspace_bytes.restype = ctypes.c_size_t
            lib.residual_norm.argtypes = [vp] * 9 + [f] * 2 + [i] * 4 + [vp]
            lib.residual_norm_backward.argtypes = [vp] * 15 + [ctypes.c_size_t, f] + [i] * 4 + [vp]
            lib.residual_norm_backward_workspace_bytes.argtypes = [i] * 5
            lib.residual_norm_backward_workspace_bytes.restype = ctypes.c_size_t
            lib.gemv_w4a16.argtypes = [vp, vp, vp, f, vp, i, i, i, vp]
            lib.gemv_w4a16_gated.argtypes = [vp, vp, vp, f, vp, vp, f, vp, i, i, i, i, vp]
            lib.gemm_get_device_status.argtypes = [vp]
            lib.gemm_selftest_wait_timeout.argtypes = [i, vp]
            lib.gemm_testing_set_overrides.argtypes = [i, i]
            lib.gemm_status_string.argtypes = [i]
            lib.gemm_status_string.restype = ctypes.c_char_p
            for name in EXPORTS[:-1]:
                getattr(lib, name).restype = i
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    try:
        return load().gemm_status_string(int(status)).decode()
    except RuntimeError:
        return STATUS.get(int(status), "unknown status")


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _check(rc: int, where: str) -> None:
    if rc != 0:
        raise GemmError(rc, where)


# The C ABI's sizes are 32-bit int, and ctypes passes the lower 32 bits of a
# larger number without a word.
_INT_MAX = (1 << 31) - 1


def _mat(t: torch.Tensor, dtype, name: str, ndim: int = 2) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")
    if t.numel() > _INT_MAX and max(t.shape) > _INT_MAX:
        raise ValueError(f"{name} has a dimension past 2^31 - 1: {tuple(t.shape)}")


def gemm_bf16_nt(A: torch.Tensor, B: torch.Tensor, C: torch.Tensor | None = None, stream=None):
    """C[M,N] = bf16(A[M,K] . B[N,K]^T), FP32 accumulation on tcgen05 tensor cores."""
    _mat(A, torch.bfloat16, "A")
    _mat(B, torch.bfloat16, "B")
    M, K = A.shape
    N, K2 = B.shape
    if K != K2:
        raise ValueError(f"K mismatch: A {tuple(A.shape)} vs B {tuple(B.shape)}")
    if C is None:
        C = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _mat(C, torch.bfloat16, "C")
    if tuple(C.shape) != (M, N):
        raise ValueError("C must be [M, N]")
    _check(load().gemm_bf16_nt(A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K,
                               _stream_ptr(stream)), "gemm_bf16_nt")
    return C


def gemm_bf16_nn(A: torch.Tensor, B: torch.Tensor, C: torch.Tensor | None = None, stream=None):
    """C[M,N] = bf16(A[M,K] . B[K,N]) (B row-major [K][N]), FP32 accumulation."""
    _mat(A, torch.bfloat16, "A")
    _mat(B, torch.bfloat16, "B")
    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise ValueError(f"K mismatch: A {tuple(A.shape)} vs B {tuple(B.shape)}")
    if C is None:
        C = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _mat(C, torch.bfloat16, "C")
    if tuple(C.shape) != (M, N):
        raise ValueError("C must be [M, N]")
    _check(load().gemm_bf16_nn(A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K,
                               _stream_ptr(stream)), "gemm_bf16_nn")
    return C


def gemm_bf16_nt_scaled_acc(A: torch.Tensor, B: torch.Tensor, C_inout: torch.Tensor, scale: float,
                            stream=None):
    """C_inout = bf16(C_inout + scale * bf16(A . B^T)) in place (fused LoRA fold)."""
    _mat(A, torch.bfloat16, "A")
    _mat(B, torch.bfloat16, "B")
    _mat(C_inout, torch.bfloat16, "C_inout")
    M, K = A.shape
    N, _ = B.shape
    if tuple(C_inout.shape) != (M, N) or B.shape[1] != K:
        raise ValueError("shape mismatch")
    _check(load().gemm_bf16_nt_scaled_acc(A.data_ptr(), B.data_ptr(), C_inout.data_ptr(), M, N, K,
                                          float(scale), _stream_ptr(stream)),
           "gemm_bf16_nt_scaled_acc")
    return C_inout


def gemm_bf16_nt_splitk_workspace_bytes(M: int, N: int, K: int, k_splits: int) -> int:
    return int(load().gemm_bf16_nt_splitk_workspace_bytes(M, N, K, k_splits))


def gemm_bf16_nt_splitk(A: torch.Tensor, B: torch.Tensor, k_splits: int,
                        workspace: torch.Tensor | None = None, C: torch.Tensor | None = None,
                        stream=None):
    """C = bf16(sum over K splits of FP32 partials), split-K with a caller workspace."""
    _mat(A, torch.bfloat16, "A")
    _mat(B, torch.bfloat16, "B")
    M, K = A.shape
    N, K2 = B.shape
    if K != K2:
        raise ValueError("K mismatch")
    need = gemm_bf16_nt_splitk_workspace_bytes(M, N, K, k_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=A.device)
    if not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    if C is None:
        C = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _mat(C, torch.bfloat16, "C")
    nbytes = workspace.numel() * workspace.element_size()
    _check(load().gemm_bf16_nt_splitk(A.data_ptr(), B.data_ptr(), C.data_ptr(),
                                      workspace.data_ptr(), nbytes, M, N, K, int(k_splits),
                                      _stream_ptr(stream)), "gemm_bf16_nt_splitk")
    return C


def gemm_bf16_nt_streamk_workspace_bytes() -> int:
    return int(load().gemm_bf16_nt_streamk_workspace_bytes())


def gemm_bf16_nt_streamk(A: torch.Tensor, B: torch.Tensor, workspace: torch.Tensor | None = None,
                         C: torch.Tensor | None = None, stream=None):
    """C = bf16(A . B^T) on the stream-K schedule, with a caller workspace."""
    _mat(A, torch.bfloat16, "A")
    _mat(B, torch.bfloat16, "B")
    M, K = A.shape
    N, K2 = B.shape
    if K != K2:
        raise ValueError("K mismatch")
    if workspace is None:
        need = gemm_bf16_nt_streamk_workspace_bytes()
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=A.device)
    if not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    if C is None:
        C = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _mat(C, torch.bfloat16, "C")
    nbytes = workspace.numel() * workspace.element_size()
    _check(load().gemm_bf16_nt_streamk(A.data_ptr(), B.data_ptr(), C.data_ptr(),
                                       workspace.data_ptr(), nbytes, M, N, K,
                                       _stream_ptr(stream)), "gemm_bf16_nt_streamk")
    return C


def gemm_w4a16(A: torch.Tensor, b: torch.Tensor, sfb: torch.Tensor, scale2: float,
               C: torch.Tensor | None = None, stream=None):
    """C = bf16(scale2 * (A . w^T)), w = e2m1(b) * e4m3(sfb) (exact in bf16).

    A bf16 [M,K]; b uint8 [N,K/2] packed e2m1 (low nibble = even k);
    sfb uint8 [N,K/16] e4m3 block scales; C bf16 [M,N].
    """
    _mat(A, torch.bfloat16, "A")
    _mat(b, torch.uint8, "b")
    _mat(sfb, torch.uint8, "sfb")
    M, K = A.shape
    N = b.shape[0]
    if tuple(b.shape) != (N, K // 2) or tuple(sfb.shape) != (N, K // 16):
        raise ValueError("shape mismatch")
    if C is None:
        C = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _mat(C, torch.bfloat16, "C")
    _check(load().gemm_w4a16(A.data_ptr(), b.data_ptr(), sfb.data_ptr(), float(scale2),
                             C.data_ptr(), M, N, K, _stream_ptr(stream)), "gemm_w4a16")
    return C


def gemm_w4a16_t(A: torch.Tensor, b_t: torch.Tensor, sfb_t: torch.Tensor, scale2: float, N: int,
                 C: torch.Tensor | None = None, stream=None):
    """gemm_w4a16 with the transposed weight layout.

    A bf16 [M,K]; b_t uint8 [K/2, ldb], byte (j, n) = elements 2j (low
    nibble) and 2j+1 (high nibble) of weight column n; sfb_t uint8 e4m3
    [K/16, ldb]; ldb >= N (columns >= N are padding); C bf16 [M,N].
    """
    _mat(A, torch.bfloat16, "A")
    _mat(b_t, torch.uint8, "b_t")
    _mat(sfb_t, torch.uint8, "sfb_t")
    M, K = A.shape
    ldb = b_t.shape[1]
    if tuple(b_t.shape) != (K // 2, ldb) or tuple(sfb_t.shape) != (K // 16, ldb):
        raise ValueError("shape mismatch")
    if C is None:
        C = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _mat(C, torch.bfloat16, "C")
    if tuple(C.shape) != (M, N):
        raise ValueError("C must be [M, N]")
    _check(load().gemm_w4a16_t(A.data_ptr(), b_t.data_ptr(), sfb_t.data_ptr(), float(scale2),
                               C.data_ptr(), M, N, K, ldb, _stream_ptr(stream)), "gemm_w4a16_t")
    return C


def gemm_w4a16_ws_workspace_bytes(N: int, K: int) -> int:
    return int(load().gemm_w4a16_ws_workspace_bytes(N, K))


def gemm_w4a16_ws(A: torch.Tensor, b: torch.Tensor, sfb: torch.Tensor, scale2: float,
                  workspace: torch.Tensor | None = None, C: torch.Tensor | None = None,
                  stream=None):
    """gemm_w4a16 in two passes (weights converted once into the workspace)."""
    _mat(A, torch.bfloat16, "A")
    _mat(b, torch.uint8, "b")
    _mat(sfb, torch.uint8, "sfb")
    M, K = A.shape
    N = b.shape[0]
    if tuple(b.shape) != (N, K // 2) or tuple(sfb.shape) != (N, K // 16):
        raise ValueError("shape mismatch")
    if workspace is None:
        workspace = torch.empty(max(gemm_w4a16_ws_workspace_bytes(N, K), 16), dtype=torch.uint8,
                                device=A.device)
    if not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    if C is None:
        C = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _mat(C, torch.bfloat16, "C")
    nbytes = workspace.numel() * workspace.element_size()
    _check(load().gemm_w4a16_ws(A.data_ptr(), b.data_ptr(), sfb.data_ptr(), float(scale2),
                                C.data_ptr(), workspace.data_ptr(), nbytes, M, N, K,
                                _stream_ptr(stream)), "gemm_w4a16_ws")
    return C


def gemm_bf16_nt_ordered(A: torch.Tensor, B: torch.Tensor, C: torch.Tensor | None = None,
                         stream=None):
    """FP32 C = strict-order, FMA-free A . B^T on CUDA cores (router GEMM)."""
    _mat(A, torch.bfloat16, "A")
    _mat(B, torch.bfloat16, "B")
    M, K = A.shape
    N, _ = B.shape
    if B.shape[1] != K:
        raise ValueError("K mismatch")
    if C is None:
        C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _mat(C, torch.float32, "C")
    _check(load().gemm_bf16_nt_ordered(A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K,
                                       _stream_ptr(stream)), "gemm_bf16_nt_ordered")
    return C


def gemm_nvfp4_bs(a: torch.Tensor, b: torch.Tensor, sfa: torch.Tensor, sfb: torch.Tensor,
                  L: int, M: int, N: int, K: int, c: torch.Tensor | None = None, stream=None):
    """fp16 c[L,M,N] for packed-e2m1 a[L,M,K/2], b[L,N,K/2] (uint8) with e4m3 scale
    bytes sfa (L*M*K/16), sfb (L*N*K/16) in the hardware scale layout."""
    for t, n in ((a, "a"), (b, "b"), (sfa, "sfa"), (sfb, "sfb")):
        if t.dtype not in (torch.uint8, torch.float8_e4m3fn) or not t.is_cuda or not t.is_contiguous():
            raise TypeError(f"{n} must be a contiguous CUDA uint8 tensor")
    if a.numel() != L * M * K // 2 or b.numel() != L * N * K // 2:
        raise ValueError("a/b size mismatch")
    if sfa.numel() != L * M * K // 16 or sfb.numel() != L * N * K // 16:
        raise ValueError("scale buffer size mismatch")
    if c is None:
        c = torch.empty((L, M, N), dtype=torch.float16, device=a.device)
    if c.dtype != torch.float16 or not c.is_contiguous() or c.numel() != L * M * N:
        raise ValueError("c must be a contiguous fp16 [L, M, N] tensor")
    _check(load().gemm_nvfp4_bs(a.data_ptr(), b.data_ptr(), sfa.data_ptr(), sfb.data_ptr(),
                                c.data_ptr(), L, M, N, K, _stream_ptr(stream)), "gemm_nvfp4_bs")
    return c


def gemm_nvfp4_bs_splitk_workspace_bytes(M: int, N: int, K: int, k_splits: int) -> int:
    return int(load().gemm_nvfp4_bs_splitk_workspace_bytes(M, N, K, k_splits))


def gemm_nvfp4_bs_splitk(a: torch.Tensor, b: torch.Tensor, sfa: torch.Tensor, sfb: torch.Tensor,
                         M: int, N: int, K: int, k_splits: int,
                         workspace: torch.Tensor | None = None, c: torch.Tensor | None = None,
                         stream=None, L: int = 1):
    """fp16 c[L,M,N] = gemm_nvfp4_bs with K split into k_splits chunks."""
    for t, n in ((a, "a"), (b, "b"), (sfa, "sfa"), (sfb, "sfb")):
        if t.dtype not in (torch.uint8, torch.float8_e4m3fn) or not t.is_cuda or not t.is_contiguous():
            raise TypeError(f"{n} must be a contiguous CUDA uint8 tensor")
    if a.numel() != L * M * K // 2 or b.numel() != L * N * K // 2:
        raise ValueError("a/b size mismatch")
    if sfa.numel() != L * M * K // 16 or sfb.numel() != L * N * K // 16:
        raise ValueError("scale buffer size mismatch")
    need = L * gemm_nvfp4_bs_splitk_workspace_bytes(M, N, K, k_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=a.device)
    if not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    if c is None:
        c = torch.empty((L, M, N), dtype=torch.float16, device=a.device)
    if c.dtype != torch.float16 or not c.is_contiguous() or c.numel() != L * M * N:
        raise ValueError("c must be a contiguous fp16 [L, M, N] tensor")
    nbytes = workspace.numel() * workspace.element_size()
    _check(load().gemm_nvfp4_bs_splitk(a.data_ptr(), b.data_ptr(), sfa.data_ptr(), sfb.data_ptr(),
                                       c.data_ptr(), workspace.data_ptr(), nbytes, L, M, N, K,
                                       int(k_splits), _stream_ptr(stream)), "gemm_nvfp4_bs_splitk")
    return c


def _on_device(name: str, device, t: torch.Tensor, dtype, shape) -> None:
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and
            t.device == device and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _context(device, stream):
    """The context that a call on tensors of `device` belongs in: the given
    stream (its allocations too, so that the caching allocator does not hand
    their memory out again before the call is done), or the tensors' device
    where another one is current.  None: it may run as it is."""
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(_stream_ptr(stream), device=device)
        return torch.cuda.stream(stream)
    if torch._C._cuda_getDevice() != device.index:
        return torch.cuda.device(device)
    return None


def _run(name: str, device, *args) -> None:
    """The C entry point `name` on the current stream."""
    rc = getattr(_lib or load(), name)(*args, torch._C._cuda_getCurrentRawStream(device.index))
    if rc:
        raise GemmError(rc, name)


def _workspace(given, need: int, device):
    """(pointer, bytes, tensor) of the caller's workspace, or of one allocated
    here (None where none is needed); the tensor has to live through the call."""
    if given is None:
        if not need:
            return None, 0, None
        given = torch.empty((need,), dtype=torch.uint8, device=device)
        return given.data_ptr(), need, given
    if not (given.device == device and given.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return given.data_ptr(), given.numel() * given.element_size(), given


def _ptr(t):
    return None if t is None else t.data_ptr()


def _xent_inputs(X, W, target):
    _mat(X, torch.bfloat16, "X")
    _mat(W, torch.bfloat16, "W")
    M, K = X.shape
    V, K2 = W.shape
    if K != K2:
        raise ValueError(f"K mismatch: X {tuple(X.shape)} vs W {tuple(W.shape)}")
    if W.device != X.device:
        raise ValueError("X and W must be on one device")
    if M > _INT_MAX or V > _INT_MAX or K > _INT_MAX:
        raise ValueError(f"sizes past 2^31 - 1: M {M}, V {V}, K {K}")
    _on_device("target", X.device, target, torch.int64, (M,))
    return M, V, K


def gemm_bf16_nt_xent_workspace_bytes(M: int, V: int) -> int:
    if not (0 <= M <= _INT_MAX and 0 <= V <= _INT_MAX):
        return 0
    return int((_lib or load()).gemm_bf16_nt_xent_workspace_bytes(M, V))


def gemm_bf16_nt_xent(X: torch.Tensor, W: torch.Tensor, target: torch.Tensor,
                      loss: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None):
    """(loss [M], lse [M]) of the softmax cross entropy of X W^T, FP32; the logits are not stored.

    X bf16 [M,K]; W bf16 [V,K]; target int64 [M], negative = the row has no
    loss.  Keep lse for gemm_bf16_nt_xent_backward.
    """
    M, V, K = _xent_inputs(X, W, target)
    device, f32 = X.device, torch.float32
    elsewhere = _context(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return gemm_bf16_nt_xent(X, W, target, loss, lse, workspace)
    if loss is None:
        loss = torch.empty((M,), dtype=f32, device=device)
    else:
        _on_device("loss", device, loss, f32, (M,))
    if lse is None:
        lse = torch.empty((M,), dtype=f32, device=device)
    else:
        _on_device("lse", device, lse, f32, (M,))
    ws, nbytes, _alive = _workspace(workspace, gemm_bf16_nt_xent_workspace_bytes(M, V), device)
    _run("gemm_bf16_nt_xent", device, X.data_ptr(), W.data_ptr(), target.data_ptr(),
         loss.data_ptr(), lse.data_ptr(), ws, nbytes, M, V, K)
    return loss, lse


def gemm_bf16_nt_xent_backward_workspace_bytes(M: int, V: int, K: int) -> int:
    if not (0 <= M <= _INT_MAX and 0 <= V <= _INT_MAX and 0 <= K <= _INT_MAX):
        return 0
    return int((_lib or load()).gemm_bf16_nt_xent_backward_workspace_bytes(M, V, K))


def gemm_bf16_nt_xent_backward(X: torch.Tensor, W: torch.Tensor, target: torch.Tensor,
                               lse: torch.Tensor, dloss: torch.Tensor,
                               dX: torch.Tensor | None = None, dW: torch.Tensor | None = None,
                               workspace: torch.Tensor | None = None, stream=None,
                               need_dx: bool = True, need_dw: bool = True):
    """(dX bf16 [M,K], dW bf16 [V,K]) of gemm_bf16_nt_xent; None for one that is not needed.

    lse: the forward call's; dloss float32 [M]: the rows' loss gradients.
    """
    M, V, K = _xent_inputs(X, W, target)
    device = X.device
    _on_device("lse", device, lse, torch.float32, (M,))
    _on_device("dloss", device, dloss, torch.float32, (M,))
    if not (need_dx or need_dw or dX is not None or dW is not None):
        raise ValueError("neither dX nor dW is needed")
    elsewhere = _context(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return gemm_bf16_nt_xent_backward(X, W, target, lse, dloss, dX, dW, workspace,
                                              need_dx=need_dx, need_dw=need_dw)
    if dX is not None:
        _on_device("dX", device, dX, torch.bfloat16, (M, K))
    elif need_dx:
        dX = torch.empty((M, K), dtype=torch.bfloat16, device=device)
    if dW is not None:
        _on_device("dW", device, dW, torch.bfloat16, (V, K))
    elif need_dw:
        dW = torch.empty((V, K), dtype=torch.bfloat16, device=device)
    ws, nbytes, _alive = _workspace(workspace, gemm_bf16_nt_xent_backward_workspace_bytes(M, V, K), device)
    _run("gemm_bf16_nt_xent_backward", device, X.data_ptr(), W.data_ptr(), target.data_ptr(),
         lse.data_ptr(), dloss.data_ptr(), _ptr(dX), _ptr(dW), ws, nbytes, M, V, K)
    return dX, dW


class RouterTopk(NamedTuple):
    """What router_topk returns (counts[E] is the number of rows that take part)."""
    weights: torch.Tensor
    experts: torch.Tensor
    lse: torch.Tensor
    counts: torch.Tensor
    probs: torch.Tensor
    losses: torch.Tensor


def _logit_rows(logits):
    """(M, E, ld) of FP32 logits whose rows may lie apart in a wider matrix."""
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if logits.dtype != torch.float32:
        raise TypeError(f"logits must be torch.float32, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError(f"logits must be 2-D, got shape {tuple(logits.shape)}")
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    M, E = logits.shape
    ld, inner = logits.stride()
    if E > 1 and inner != 1:
        raise ValueError("logits must have unit stride within a row")
    if M <= 1:
        ld = E
    if ld < E:
        raise ValueError("rows of logits overlap")
    if ld > _INT_MAX or M > _INT_MAX:
        raise ValueError(f"logits {M} x {E} with row stride {ld}: past 2^31 - 1")
    return M, E, ld


def router_topk_workspace_bytes(M: int, E: int) -> int:
    if not (0 <= M <= _INT_MAX and 0 <= E <= _INT_MAX):
        return 0
    return int((_lib or load()).router_topk_workspace_bytes(M, E))


def router_topk(logits: torch.Tensor, k: int, valid: torch.Tensor | None = None,
                normalize: bool = False, workspace: torch.Tensor | None = None,
                stream=None) -> RouterTopk:
    """Softmax, top-k experts, per-expert counts, balance loss and z-loss of FP32 router logits.

    logits float32 [M,E] (row stride >= E); valid uint8 or bool [M], zero = a
    padding row.  losses = [balance, z].
    """
    M, E, ld = _logit_rows(logits)
    device, empty, f32, i32 = logits.device, torch.empty, torch.float32, torch.int32
    if valid is not None:
        valid = valid.view(torch.uint8) if valid.dtype == torch.bool else valid
        _on_device("valid", device, valid, torch.uint8, (M,))
    if not 1 <= k <= E:
        raise ValueError(f"k must be in 1..{E}, got {k}")
    elsewhere = _context(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return router_topk(logits, k, valid, normalize, workspace)
    weights = empty((M, k), dtype=f32, device=device)
    experts = empty((M, k), dtype=i32, device=device)
    lse = empty((M,), dtype=f32, device=device)
    counts = empty((E + 1,), dtype=i32, device=device)
    probs = empty((E,), dtype=f32, device=device)
    losses = empty((2,), dtype=f32, device=device)
    ws, nbytes, _alive = _workspace(workspace, router_topk_workspace_bytes(M, E), device)
    _run("router_topk", device, logits.data_ptr(), _ptr(valid), weights.data_ptr(),
         experts.data_ptr(), lse.data_ptr(), counts.data_ptr(), probs.data_ptr(),
         losses.data_ptr(), ws, nbytes, M, E, ld, k,
         1 if normalize else 0)
    return RouterTopk(weights, experts, lse, counts, probs, losses)


def router_topk_backward(logits: torch.Tensor, experts: torch.Tensor, lse: torch.Tensor,
                         counts: torch.Tensor, dweights: torch.Tensor | None = None,
                         dlosses: torch.Tensor | None = None, normalize: bool = False,
                         dtype=torch.float32, dlogits: torch.Tensor | None = None, stream=None):
    """Gradient of router_topk's weights and losses with respect to its logits.

    experts, lse, counts: the forward call's.  dweights float32 [M,k] and
    dlosses float32 [2] may be None (zero).  dtype: float32, or bfloat16 for a
    gradient that goes into a BF16 product.
    """
    M, E, ld = _logit_rows(logits)
    device = logits.device
    if experts.dim() != 2:
        raise ValueError("experts must be [M, k]")
    k = experts.shape[1]
    _on_device("experts", device, experts, torch.int32, (M, k))
    _on_device("lse", device, lse, torch.float32, (M,))
    _on_device("counts", device, counts, torch.int32, (E + 1,))
    if dweights is not None:
        _on_device("dweights", device, dweights, torch.float32, (M, k))
    if dlosses is not None:
        _on_device("dlosses", device, dlosses, torch.float32, (2,))
    if dlogits is not None:
        dtype = dlogits.dtype
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"dlogits must be float32 or bfloat16, got {dtype}")
    elsewhere = _context(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return router_topk_backward(logits, experts, lse, counts, dweights, dlosses, normalize,
                                        dtype, dlogits)
    if dlogits is None:
        dlogits = torch.empty((M, E), dtype=dtype, device=device)
    else:
        _on_device("dlogits", device, dlogits, dtype, (M, E))
    _run("router_topk_backward", device, logits.data_ptr(), experts.data_ptr(), lse.data_ptr(),
         counts.data_ptr(), _ptr(dweights), _ptr(dlosses), dlogits.data_ptr(),
         1 if dtype == torch.bfloat16 else 0, M, E, ld, k, 1 if normalize else 0)
    return dlogits


ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}


def _activation(act: str) -> int:
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}")
    return ACTIVATIONS[act]


def _gated_inputs(X, Wg, Wu):
    _mat(X, torch.bfloat16, "X")
    _mat(Wg, torch.bfloat16, "Wg")
    M, K = X.shape
    F, K2 = Wg.shape
    if K != K2:
        raise ValueError(f"K mismatch: X {tuple(X.shape)} vs Wg {tuple(Wg.shape)}")
    if Wg.device != X.device:
        raise ValueError("X and Wg must be on one device")
    if M > _INT_MAX or F > _INT_MAX or K > _INT_MAX:
        raise ValueError(f"sizes past 2^31 - 1: M {M}, F {F}, K {K}")
    _on_device("Wu", X.device, Wu, torch.bfloat16, (F, K))
    return M, F, K


def gemm_bf16_nt_gated(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, act: str = "silu",
                       H: torch.Tensor | None = None, gates: torch.Tensor | None = None,
                       stream=None, save_gates: bool = False):
    """(H bf16 [M,F], gates): H = act(X Wg^T) * (X Wu^T) in one kernel.

    X bf16 [M,K]; Wg, Wu bf16 [F,K]; act "silu" or "gelu_tanh".  gates is
    None, or with save_gates (or a tensor given for it) both products as bf16
    [2,M,F], which gemm_bf16_nt_gated_backward reads.
    """
    M, F, K = _gated_inputs(X, Wg, Wu)
    kind, device, bf16 = _activation(act), X.device, torch.bfloat16
    elsewhere = _context(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return gemm_bf16_nt_gated(X, Wg, Wu, act, H, gates, save_gates=save_gates)
    if H is None:
        H = torch.empty((M, F), dtype=bf16, device=device)
    else:
        _on_device("H", device, H, bf16, (M, F))
    if gates is not None:
        _on_device("gates", device, gates, bf16, (2, M, F))
    elif save_gates:
        gates = torch.empty((2, M, F), dtype=bf16, device=device)
    _run("gemm_bf16_nt_gated", device, X.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), H.data_ptr(),
         _ptr(gates), kind, M, F, K)
    return H, gates


@functools.lru_cache(maxsize=1024)  # a size is asked for with every call
def gemm_bf16_nt_gated_backward_workspace_bytes(M: int, F: int, K: int) -> int:
    if not (0 <= M <= _INT_MAX and 0 <= F <= _INT_MAX and 0 <= K <= _INT_MAX):
        return 0
    return int((_lib or load()).gemm_bf16_nt_gated_backward_workspace_bytes(M, F, K))


def gemm_bf16_nt_gated_backward(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor,
                                dH: torch.Tensor, act: str = "silu",
                                gates: torch.Tensor | None = None,
                                dX: torch.Tensor | None = None, dWg: torch.Tensor | None = None,
                                dWu: torch.Tensor | None = None,
                                workspace: torch.Tensor | None = None, stream=None,
                                need_dx: bool = True, need_dw: bool = True):
    """(dX bf16 [M,K], dWg, dWu bf16 [F,K]) of gemm_bf16_nt_gated; None for what is not needed.

    dH bf16 [M,F]; gates: the forward call's, or None to form them again from X.
    """
    M, F, K = _gated_inputs(X, Wg, Wu)
    kind, device, bf16 = _activation(act), X.device, torch.bfloat16
    _on_device("dH", device, dH, bf16, (M, F))
    if gates is not None:
        _on_device("gates", device, gates, bf16, (2, M, F))
    if (dWg is None) != (dWu is None):
        raise ValueError("give both of dWg and dWu, or neither")
    if not (need_dx or need_dw or dX is not None or dWg is not None):
        raise ValueError("neither dX nor the weight gradients are needed")
    elsewhere = _context(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return gemm_bf16_nt_gated_backward(X, Wg, Wu, dH, act, gates, dX, dWg, dWu, workspace,
                                               need_dx=need_dx, need_dw=need_dw)
    if dX is not None:
        _on_device("dX", device, dX, bf16, (M, K))
    elif need_dx:
        dX = torch.empty((M, K), dtype=bf16, device=device)
    if dWg is not None:
        _on_device("dWg", device, dWg, bf16, (F, K))
        _on_device("dWu", device, dWu, bf16, (F, K))
    elif need_dw:
        dWg = torch.empty((F, K), dtype=bf16, device=device)
        dWu = torch.empty((F, K), dtype=bf16, device=device)
    ws, nbytes, _alive = _workspace(workspace, gemm_bf16_nt_gated_backward_workspace_bytes(M, F, K),
                                    device)
    _run("gemm_bf16_nt_gated_backward", device, X.data_ptr(), Wg.data_ptr(), Wu.data_ptr(),
         dH.data_ptr(), _ptr(gates), _ptr(dX), _ptr(dWg), _ptr(dWu), ws, nbytes, kind, M, F, K)
    return dX, dWg, dWu


@functools.lru_cache(maxsize=1024)  # a size is asked for with every call
def gemm_bf16_tn_workspace_bytes(M: int, N: int, K: int) -> int:
    if not (0 <= M <= _INT_MAX and 0 <= N <= _INT_MAX and 0 <= K <= _INT_MAX):
        return 0
    return int((_lib or load()).gemm_bf16_tn_workspace_bytes(M, N, K))


def gemm_bf16_tn(A: torch.Tensor, B: torch.Tensor, C: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None):
    """C[M,N] = bf16(A[K,M]^T . B[K,N]), FP32 accumulation: a weight gradient dY^T X."""
    _mat(A, torch.bfloat16, "A")
    _mat(B, torch.bfloat16, "B")
    K, M = A.shape
    K2, N = B.shape
    if K != K2:
        raise ValueError(f"K mismatch: A {tuple(A.shape)} vs B {tuple(B.shape)}")
    device = A.device
    if B.device != device:
        raise ValueError("A and B must be on one device")
    if M > _INT_MAX or N > _INT_MAX or K > _INT_MAX:
        raise ValueError(f"sizes past 2^31 - 1: M {M}, N {N}, K {K}")
    elsewhere = _context(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return gemm_bf16_tn(A, B, C, workspace)
    if C is None:
        C = torch.empty((M, N), dtype=torch.bfloat16, device=device)
    else:
        _on_device("C", device, C, torch.bfloat16, (M, N))
    ws, nbytes, _alive = _workspace(workspace, gemm_bf16_tn_workspace_bytes(M, N, K), device)
    _run("gemm_bf16_tn", device, A.data_ptr(), B.data_ptr(), C.data_ptr(), ws, nbytes, M, N, K)
    return C


class ResidualNorm(NamedTuple):
    """What residual_norm returns; None for what the call has no use for."""
    y: torch.Tensor
    n: torch.Tensor | None
    rstd_post: torch.Tensor | None
    rstd_pre: torch.Tensor | None


class ResidualNormGrads(NamedTuple):
    """What residual_norm_backward returns; None for what it was not asked for."""
    dx: torch.Tensor
    dblock: torch.Tensor | None
    dw_pre: torch.Tensor | None
    dw_post: torch.Tensor | None
    dgate: torch.Tensor | None


def _stream_rows(t, name: str):
    """(M, D, 1 if FP32) of the residual stream or its gradient."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dtype, shape = t.dtype, t.shape
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError(f"{name} must be bfloat16 or float32, got {dtype}")
    if len(shape) != 2 or not (t.is_cuda and t.is_contiguous()):
        _mat(t, dtype, name)
    M, D = shape
    if M > _INT_MAX or D > _INT_MAX:
        raise ValueError(f"sizes past 2^31 - 1: M {M}, D {D}")
    return M, D, 1 if dtype is torch.float32 else 0


def _norm_inputs(M, D, device, block, w_post, gate, w_pre):
    """Checks what residual_norm and its gradient share; rows per gate (M without one)."""
    bf16, row = torch.bfloat16, (D,)
    if block is not None:
        _on_device("block", device, block, bf16, (M, D))
    elif w_post is not None or gate is not None:
        raise ValueError("w_post and gate belong to a block: give block")
    elif w_pre is None:
        raise ValueError("neither a block nor w_pre: nothing to do")
    if w_post is not None:
        _on_device("w_post", device, w_post, bf16, row)
    if w_pre is not None:
        _on_device("w_pre", device, w_pre, bf16, row)
    if gate is None:
        return M
    if isinstance(gate, torch.Tensor) and gate.dim() == 1:
        _on_device("gate", device, gate, bf16, row)
        return M
    groups = gate.shape[0] if isinstance(gate, torch.Tensor) and gate.dim() == 2 else 1
    if groups == 0 or M % groups:
        raise ValueError(f"gate has {groups} rows, which do not divide {M}")
    _on_device("gate", device, gate, bf16, (groups, D))
    return M // groups


def residual_norm(x: torch.Tensor, block: torch.Tensor | None = None,
                  w_post: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                  w_pre: torch.Tensor | None = None, scale: float = 1.0, eps: float = 1e-6,
                  y: torch.Tensor | None = None, n: torch.Tensor | None = None,
                  stream=None, need_rstd: bool = True) -> ResidualNorm:
    """The residual step between two blocks: y = x + scale * gate * norm(block, w_post) and
    n = norm(y, w_pre), root-mean-square norms, in one pass.

    x [M,D], the stream, bf16 or float32; block bf16 [M,D], or None: no block
    yet (y is x); gate bf16 [D], or [G,D] with G a divisor of M: row m has gate
    row m // (M // G); w_post, w_pre bf16 [D], or None: no such norm.  y may be
    x: the stream is updated in place.  need_rstd False leaves out what only the
    gradient needs (one token: a quarter of the host's time).
    """
    M, D, f32 = _stream_rows(x, "x")
    device = x.device
    rows = _norm_inputs(M, D, device, block, w_post, gate, w_pre)
    if y is not None:
        if block is None:
            raise ValueError("without a block there is no y to write")
        _on_device("y", device, y, x.dtype, (M, D))
    if n is not None:
        if w_pre is None:
            raise ValueError("n needs w_pre")
        _on_device("n", device, n, torch.bfloat16, (M, D))
    elsewhere = _context(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return residual_norm(x, block, w_post, gate, w_pre, scale, eps, y, n, need_rstd=need_rstd)
    # (pointers without a call to _ptr each: the host's time is what a few rows take)
    empty, F32, like, post, pre = torch.empty, torch.float32, torch.empty_like, None, None
    if block is not None:
        if y is None:
            y = like(x)
        y_ptr, block_ptr = y.data_ptr(), block.data_ptr()
    else:
        y_ptr = block_ptr = None
    rstd_post = rstd_pre = n_ptr = post_ptr = pre_ptr = None
    if w_post is not None:
        post = w_post.data_ptr()
        if need_rstd:
            rstd_post = empty((M,), dtype=F32, device=device)
            post_ptr = rstd_post.data_ptr()
    if w_pre is not None:
        if n is None:
            n = like(x) if f32 == 0 else empty((M, D), dtype=torch.bfloat16, device=device)
        pre, n_ptr = w_pre.data_ptr(), n.data_ptr()
        if need_rstd:
            rstd_pre = empty((M,), dtype=F32, device=device)
            pre_ptr = rstd_pre.data_ptr()
    _run("residual_norm", device, x.data_ptr(), block_ptr, post,
         None if gate is None else gate.data_ptr(), pre, y_ptr, n_ptr, post_ptr, pre_ptr,
         float(scale), float(eps), f32, M, D, rows)
    return ResidualNorm(x if block is None else y, n, rstd_post, rstd_pre)


@functools.lru_cache(maxsize=1024)  # a size is asked for with every call
def residual_norm_backward_workspace_bytes(M: int, D: int, rows_per_gate: int, weights: int,
                                           gates: int) -> int:
    if not (0 <= M <= _INT_MAX and 0 <= D <= _INT_MAX and 0 <= rows_per_gate <= _INT_MAX):
        return 0
    return int((_lib or load()).residual_norm_backward_workspace_bytes(M, D, rows_per_gate, weights,
                                                                       gates))


def residual_norm_backward(dy: torch.Tensor | None, dn: torch.Tensor | None,
                           y: torch.Tensor | None, block: torch.Tensor | None = None,
                           rstd_post: torch.Tensor | None = None,
                           rstd_pre: torch.Tensor | None = None,
                           w_post: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                           w_pre: torch.Tensor | None = None, scale: float = 1.0,
                           dx: torch.Tensor | None = None, dblock: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None, stream=None,
                           need_dw: bool = True) -> ResidualNormGrads:
    """Gradients of residual_norm from those of y (dy, None: zero) and n (dn, with w_pre).

    y, rstd_post, rstd_pre: the forward call's; block, w_post, gate, w_pre and
    scale as there.  The gradients of the weights and the gate are float32 of
    the weights' and the gate's shape (need_dw False: none).  dx may be dy.
    """
    first = dy if dy is not None else y
    M, D, f32 = _stream_rows(first, "dy" if dy is not None else "y")
    device, bf16, F32 = first.device, torch.bfloat16, torch.float32
    rows = _norm_inputs(M, D, device, block, w_post, gate, w_pre)
    if (dn is None) != (w_pre is None):
        raise ValueError("dn and w_pre belong together")
    if dy is None and dn is None:
        raise ValueError("neither dy nor dn: nothing to do")
    if w_pre is not None:
        _on_device("dn", device, dn, bf16, (M, D))
        _on_device("y", device, y, first.dtype, (M, D))
        _on_device("rstd_pre", device, rstd_pre, F32, (M,))
    if w_post is not None:
        _on_device("rstd_post", device, rstd_post, F32, (M,))
    if dx is not None:
        _on_device("dx", device, dx, first.dtype, (M, D))
    if dblock is not None:
        if block is None:
            raise ValueError("without a block there is no dblock")
        _on_device("dblock", device, dblock, bf16, (M, D))
    elsewhere = _context(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return residual_norm_backward(dy, dn, y, block, rstd_post, rstd_pre, w_post, gate, w_pre,
                                          scale, dx, dblock, workspace, need_dw=need_dw)
    empty = torch.empty
    if dx is None:
        dx = empty((M, D), dtype=first.dtype, device=device)
    if dblock is None and block is not None:
        dblock = empty((M, D), dtype=bf16, device=device)
    dw_post = empty((D,), dtype=F32, device=device) if need_dw and w_post is not None else None
    dw_pre = empty((D,), dtype=F32, device=device) if need_dw and w_pre is not None else None
    dgate = empty(gate.shape, dtype=F32, device=device) if need_dw and gate is not None else None
    need = residual_norm_backward_workspace_bytes(M, D, rows, (dw_post is not None) + (dw_pre is not None),
                                                  1 if dgate is not None else 0)
    ws, nbytes, _alive = _workspace(workspace, need, device)
    _run("residual_norm_backward", device, _ptr(dy), _ptr(dn), _ptr(y), _ptr(block),
         _ptr(rstd_post) if w_post is not None else None, _ptr(rstd_pre) if w_pre is not None else None,
         _ptr(w_post), _ptr(gate), _ptr(w_pre), dx.data_ptr(), _ptr(dblock), _ptr(dw_post),
         _ptr(dgate), _ptr(dw_pre), ws, nbytes, float(scale), f32, M, D, rows)
    return ResidualNormGrads(dx, dblock, dw_pre, dw_post, dgate)


def _gemv_inputs(A, *weights):
    """(M, N, K) of few tokens A and NVFP4 weight matrices of one shape: (b, sfb, names)."""
    _mat(A, torch.bfloat16, "A")
    M, K = A.shape
    b, _, name_b, _ = weights[0]
    if not isinstance(b, torch.Tensor) or b.dim() != 2:
        _mat(b, torch.uint8, name_b)
    N = b.shape[0]
    if M > _INT_MAX or N > _INT_MAX or K > _INT_MAX:
        raise ValueError(f"sizes past 2^31 - 1: M {M}, N {N}, K {K}")
    if K % 256:
        raise ValueError(f"K must be a multiple of 256, got {K}")
    if not 1 <= M <= 16:
        raise ValueError(f"1 to 16 tokens, got {M}: gemm_w4a16 takes more")
    device, u8, codes, scales = A.device, torch.uint8, (N, K // 2), (N, K // 16)
    for b, sf, name_b, name_sf in weights:
        _on_device(name_b, device, b, u8, codes)
        _on_device(name_sf, device, sf, u8, scales)
    return M, N, K


def gemv_w4a16(A: torch.Tensor, b: torch.Tensor, sfb: torch.Tensor, scale2: float,
               C: torch.Tensor | None = None, stream=None):
    """gemm_w4a16 for 1 to 16 tokens: C = bf16(scale2 * (A . w^T)), w = e2m1(b) * e4m3(sfb).

    A bf16 [M,K]; b uint8 [N,K/2] (low nibble = even k); sfb uint8 [N,K/16]; K a
    multiple of 256, any N.
    """
    M, N, K = _gemv_inputs(A, (b, sfb, "b", "sfb"))
    device = A.device
    elsewhere = _context(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return gemv_w4a16(A, b, sfb, scale2, C)
    if C is None:
        C = torch.empty((M, N), dtype=torch.bfloat16, device=device)
    else:
        _on_device("C", device, C, torch.bfloat16, (M, N))
    _run("gemv_w4a16", device, A.data_ptr(), b.data_ptr(), sfb.data_ptr(), float(scale2),
         C.data_ptr(), M, N, K)
    return C


def gemv_w4a16_gated(A: torch.Tensor, bg: torch.Tensor, sfg: torch.Tensor, scale2_g: float,
                     bu: torch.Tensor, sfu: torch.Tensor, scale2_u: float, act: str = "silu",
                     H: torch.Tensor | None = None, stream=None):
    """The gated projection of 1 to 16 tokens with NVFP4 weights, in one kernel:
    H = bf16(act(scale2_g * (A . wg^T)) * (scale2_u * (A . wu^T))).

    Both matrices as for gemv_w4a16, of one shape; act "silu" or "gelu_tanh".
    """
    M, F, K = _gemv_inputs(A, (bg, sfg, "bg", "sfg"), (bu, sfu, "bu", "sfu"))
    kind, device = _activation(act), A.device
    elsewhere = _context(device, stream)
    if elsewhere is not None:
        with elsewhere:
            return gemv_w4a16_gated(A, bg, sfg, scale2_g, bu, sfu, scale2_u, act, H)
    if H is None:
        H = torch.empty((M, F), dtype=torch.bfloat16, device=device)
    else:
        _on_device("H", device, H, torch.bfloat16, (M, F))
    _run("gemv_w4a16_gated", device, A.data_ptr(), bg.data_ptr(), sfg.data_ptr(), float(scale2_g),
         bu.data_ptr(), sfu.data_ptr(), float(scale2_u), H.data_ptr(), kind, M, F, K)
    return H


def bf16_scaled_add(out: torch.Tensor, d: torch.Tensor, scale: float, stream=None):
    """out = bf16(out + scale * d) elementwise (the unfused pair's second step)."""
    if out.dtype != torch.bfloat16 or d.dtype != torch.bfloat16 or out.numel() != d.numel():
        raise ValueError("out and d must be bf16 tensors of the same size")
    if not (out.is_cuda and d.is_cuda and out.is_contiguous() and d.is_contiguous()):
        raise ValueError("out and d must be contiguous CUDA tensors")
    _check(load().bf16_scaled_add(out.data_ptr(), d.data_ptr(), float(scale), out.numel(),
                                  _stream_ptr(stream)), "bf16_scaled_add")
    return out


def gemm_selftest_wait_timeout(timeout_ms: int = 50, stream=None) -> None:
    """Launch the failure-path self test (a wait that must run out)."""
    _check(load().gemm_selftest_wait_timeout(int(timeout_ms), _stream_ptr(stream)),
           "gemm_selftest_wait_timeout")


def gemm_testing_set_overrides(cta_group: int = 0, streamk_clusters: int = 0) -> None:
    """Testing hook: force the CTA group of the BF16 launchers (1 or 2) and the
    CTA pairs sharing a stream-K tail; 0 restores the shape's own choice."""
    _check(load().gemm_testing_set_overrides(int(cta_group), int(streamk_clusters)),
           "gemm_testing_set_overrides")


def gemm_get_device_status(stream=None) -> int:
    """Synchronise the stream; return (and clear) the device status word."""
    return int(load().gemm_get_device_status(_stream_ptr(stream)))
