"""MI355X (gfx950) block-scaled GEMM: thin Python binding of libdbs.so.

    D = bf16(alpha * (sA . A) @ (sB . B)^T),  fp32 accumulation

The functions take torch tensors that already live on the GPU and only
marshal pointers, sizes and the current stream into the C ABI of
``include/dbs.h``; every step of the computation runs in the HIP kernels.
There is no CPU fallback: if ``libdbs.so`` is missing, or a call reports an
error, these functions raise.

Operand encodings (contiguous; K-major unless la / lb say MN_MAJOR):
  gemm_bf16(A, B)                     A: (M, K) bfloat16/uint16, B: (N, K)
  gemm_bf16_decoupled(A, B)           the same on the decoupled-ring kernel (K-major, K > 64)
  gemm_mx(elem, A, sA, B, sB)         elem 'e4m3': A (M, K) uint8;
                                      elem 'e2m1': A (M, K/2) uint8, 2 per byte
                                      sA: (M, K/32) uint8 E8M0 codes
  gemm_nvfp4(A, sA, tA, B, sB, tB)    A: (M, K/2) uint8 packed E2M1,
                                      sA: (M, K/16) uint8 E4M3 codes, tA float
MN-major operands (gemm_bf16, gemm_mx) are stored transposed: A (K, M), B
(K, N), E2M1 packing two consecutive M (N) per byte, (K, M/2); scales keep
their (M, K/32) layout.
The mixture-of-experts operators (moe_route ... moe_combine_backward) and those
in 8-bit integers (quant_i8 ... gemm_moe_swiglu_i8) are described at their
functions.
Each GEMM returns D: (M, N) torch.bfloat16 (or writes into ``out``).
"""
from __future__ import annotations

import contextlib
import ctypes
import operator
from pathlib import Path
from typing import NamedTuple

import torch

__all__ = ["gemm_bf16", "gemm_bf16_decoupled", "gemm_mx", "gemm_mx_mixed", "gemm_nvfp4", "gemm_nvfp4_fp8", "gemm_nvfp4_fp8_noalloc", "nvfp4_fp8_workspace_bytes", "gemm_nvfp4_fp6", "nvfp4_fp6_workspace_bytes", "gemm_grouped_bf16", "gemm_grouped_mx", "gemm_grouped_nvfp4", "quant_mx", "quant_nvfp4", "quant_bf16",
           "MoeRouting", "moe_route", "moe_route_backward", "gemm_moe_bf16", "gemm_moe_swiglu_bf16", "gemm_moe_dw_bf16",
           "moe_route_grouped", "moe_route_grouped_backward", "quant_i8", "gemm_i8", "gemm_moe_i8", "gemm_moe_swiglu_i8",
           "swiglu", "swiglu_backward", "moe_combine", "moe_combine_backward", "lib", "LIB_PATH", "DbsError", "load_poison_library", "using_library",
           "DBS_OK", "DBS_EINVAL", "DBS_EUNSUPPORTED", "DBS_EHIP", "K_MAJOR", "MN_MAJOR",
           "E4M3", "E5M2", "E2M3", "E3M2", "E2M1", "status_str"]

LIB_PATH = Path(__file__).resolve().parent / "libdbs.so"

DBS_OK, DBS_EINVAL, DBS_EUNSUPPORTED, DBS_EHIP = 0, 1, 2, 3
K_MAJOR, MN_MAJOR = 0, 1
E4M3, E5M2, E2M3, E3M2, E2M1 = 0, 1, 2, 3, 4
_ELEM = {"e4m3": E4M3, "e5m2": E5M2, "e2m3": E2M3, "e3m2": E3M2, "e2m1": E2M1}


class DbsError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{msg} (status {status})")
        self.status = status


_lib = None


def _load(path: Path) -> ctypes.CDLL:
    if not path.exists():
        raise ImportError(f"{path} is missing: build it with "
                          "`python -m dense_block_scaled_amd.build` (or __graft_entry__.build())")
    L = ctypes.CDLL(str(path))
    _declare(L)
    return L


def lib() -> ctypes.CDLL:
    """The loaded C-ABI library; raises if it has not been built."""
    global _lib
    if _lib is None:
        _lib = _load(LIB_PATH)
    return _lib


def load_poison_library() -> ctypes.CDLL:
    """The LDS-poison debug build of the library (libdbs_poison.so: every
    direct-to-LDS load first fills its destination with 0xFF), for the
    race-detection tests; raises if it has not been built."""
    return _load(LIB_PATH.with_name("libdbs_poison.so"))


@contextlib.contextmanager
def using_library(L: ctypes.CDLL):
    """Route this module's calls through library L (e.g. the poison build)
    inside the block."""
    global _lib
    prev = lib()
    _lib = L
    try:
        yield L
    finally:
        _lib = prev


def _declare(L: ctypes.CDLL) -> None:
    """Argument and result types of the C ABI's entry points."""
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.gemm_bf16.argtypes = [P, P, P, I64, I64, I64, I, I, P]
    L.gemm_bf16.restype = I
    L.gemm_bf16_decoupled.argtypes = [P, P, P, I64, I64, I64, I, P]
    L.gemm_bf16_decoupled.restype = I
    L.gemm_mx.argtypes = [I, P, P, P, P, P, I64, I64, I64, I, I, P]
    L.gemm_mx.restype = I
    L.gemm_mx_mixed.argtypes = [I, I, P, P, P, P, P, I64, I64, I64, I, I, P]
    L.gemm_mx_mixed.restype = I
    L.gemm_nvfp4.argtypes = [P, P, ctypes.c_float, P, P, ctypes.c_float, P, I64, I64, I64, I, I, P]
    L.gemm_nvfp4.restype = I
    L.gemm_nvfp4_fp8_workspace.argtypes = [I64, I64, I64]
    L.gemm_nvfp4_fp8_workspace.restype = ctypes.c_size_t
    L.gemm_nvfp4_fp8.argtypes = [P, P, ctypes.c_float, P, P, ctypes.c_float, P, I64, I64, I64, I, I, P,
                                 ctypes.c_size_t, P]
    L.gemm_nvfp4_fp8.restype = I
    L.gemm_nvfp4_fp6_workspace.argtypes = [I64, I64, I64]
    L.gemm_nvfp4_fp6_workspace.restype = ctypes.c_size_t
    L.gemm_nvfp4_fp6.argtypes = [P, P, ctypes.c_float, P, P, ctypes.c_float, P, I64, I64, I64, I, I, P,
                                 ctypes.c_size_t, P]
    L.gemm_nvfp4_fp6.restype = I
    L.gemm_nvfp4_fp8_noalloc.argtypes = [P, P, ctypes.c_float, P, P, ctypes.c_float, P, I64, I64, I64, I, I, P]
    L.gemm_nvfp4_fp8_noalloc.restype = I
    L.gemm_grouped_bf16.argtypes = [P, P, P, P, I64, I64, I64, P]
    L.gemm_grouped_bf16.restype = I
    L.gemm_grouped_mx.argtypes = [I, P, P, P, P, P, P, I64, I64, I64, P]
    L.gemm_grouped_mx.restype = I
    L.gemm_grouped_nvfp4.argtypes = [P, P, ctypes.c_float, P, P, P, P, P, I64, I64, I64, P]
    L.gemm_grouped_nvfp4.restype = I
    L.quant_mx.argtypes = [I, P, I64, I64, P, P, P]
    L.quant_mx.restype = I
    L.quant_nvfp4.argtypes = [P, I64, I64, P, P, P, P]
    L.quant_nvfp4.restype = I
    L.quant_bf16.argtypes = [P, I64, P, P]
    L.quant_bf16.restype = I
    SZ = ctypes.c_size_t
    L.moe_route_workspace.argtypes = [I64, I64, I64]
    L.moe_route_workspace.restype = SZ
    L.moe_route.argtypes = [I, P, I64, I64, I64, I, P, P, P, P, P, P, SZ, P]
    L.moe_route.restype = I
    L.moe_route_bwd.argtypes = [I, P, I64, I64, I64, I, P, P, P, P]
    L.moe_route_bwd.restype = I
    L.gemm_moe_bf16.argtypes = [P, P, P, P, P, I64, I64, I64, I64, I64, I, P]
    L.gemm_moe_bf16.restype = I
    L.gemm_moe_swiglu_bf16.argtypes = [P, P, P, P, P, I64, I64, I64, I64, I64, P]
    L.gemm_moe_swiglu_bf16.restype = I
    L.gemm_moe_dw_bf16.argtypes = [I, P, P, P, P, P, I64, I64, I64, I64, I64, I, P]
    L.gemm_moe_dw_bf16.restype = I
    L.swiglu_bf16.argtypes = [P, P, I64, I64, P]
    L.swiglu_bf16.restype = I
    L.swiglu_bwd_bf16.argtypes = [P, P, P, I64, I64, P]
    L.swiglu_bwd_bf16.restype = I
    L.moe_combine_bf16.argtypes = [P, P, P, P, I64, I64, I64, I64, P]
    L.moe_combine_bf16.restype = I
    L.moe_combine_bwd_bf16.argtypes = [P, P, P, P, P, I64, P, P, I64, I64, I64, P]
    L.moe_combine_bwd_bf16.restype = I
    F = ctypes.c_float
    L.moe_route_grouped_workspace.argtypes = [I64, I64, I64]
    L.moe_route_grouped_workspace.restype = SZ
    L.moe_route_grouped.argtypes = [I, P, P, I64, I64, I64, I, I64, I64, I64, I, F, P, P, P, P, P, P, SZ, P]
    L.moe_route_grouped.restype = I
    L.moe_route_grouped_bwd.argtypes = [I, P, I64, I64, I64, I, I, F, P, P, P, P]
    L.moe_route_grouped_bwd.restype = I
    L.quant_i8.argtypes = [I, P, I64, I64, P, P, P]
    L.quant_i8.restype = I
    L.gemm_i8.argtypes = [I, P, P, P, P, P, I64, I64, I64, P]
    L.gemm_i8.restype = I
    L.gemm_moe_i8.argtypes = [P, P, P, P, P, P, P, I64, I64, I64, I64, I64, P]
    L.gemm_moe_i8.restype = I
    L.gemm_moe_swiglu_i8.argtypes = [P, P, P, P, P, P, P, I64, I64, I64, I64, I64, P]
    L.gemm_moe_swiglu_i8.restype = I
    L.dbs_status_str.argtypes = [I]
    L.dbs_status_str.restype = ctypes.c_char_p
    L.dbs_last_error.argtypes = []
    L.dbs_last_error.restype = ctypes.c_char_p
    L.dbs_version.restype = I


def status_str(st: int) -> str:
    return lib().dbs_status_str(st).decode()


def _check(st: int) -> None:
    if st != DBS_OK:
        raise DbsError(st, f"{status_str(st)}: {lib().dbs_last_error().decode()}")


def _dev(t: torch.Tensor, name: str, dtypes, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _out(out, M, N, like):
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=like.device)
    _dev(out, "out", (torch.bfloat16, torch.int16, torch.uint16), (M, N))
    return out


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _layout(l: int, name: str) -> int:
    if l not in (K_MAJOR, MN_MAJOR):
        raise ValueError(f"{name}: layout must be K_MAJOR or MN_MAJOR")
    return l


def _rows(t: torch.Tensor, l: int, per_byte: int = 1) -> int:
    """M (or N) of an operand: its row count, or (MN-major) its columns."""
    return t.shape[0] if l == K_MAJOR else t.shape[1] * per_byte


def _shape(rows: int, kcols: int, l: int, per_byte: int = 1) -> tuple:
    """Expected tensor shape of an operand with `rows` rows (M or N) and K
    of kcols elements (per_byte elements per stored byte)."""
    return (rows, kcols // per_byte) if l == K_MAJOR else (kcols, rows // per_byte)


def gemm_bf16(A: torch.Tensor, B: torch.Tensor, out: torch.Tensor | None = None,
              la: int = K_MAJOR, lb: int = K_MAJOR) -> torch.Tensor:
    """D = A @ B^T for bf16 A (M, K), B (N, K) (MN-major: (K, M), (K, N));
    fp32 accumulate, bf16 out."""
    la, lb = _layout(la, "la"), _layout(lb, "lb")
    M, N = _rows(A, la), _rows(B, lb)
    K = A.shape[1] if la == K_MAJOR else A.shape[0]
    dt = (torch.bfloat16, torch.int16, torch.uint16)
    pa = _dev(A, "A", dt, _shape(M, K, la))
    pb = _dev(B, "B", dt, _shape(N, K, lb))
    out = _out(out, M, N, A)
    _check(lib().gemm_bf16(pa, pb, ctypes.c_void_p(out.data_ptr()), M, N, K, la, lb, _stream(A)))
    return out


def gemm_bf16_decoupled(A: torch.Tensor, B: torch.Tensor, out: torch.Tensor | None = None,
                        early_release_a: bool = True) -> torch.Tensor:
    """gemm_bf16 (K-major A (M, K), B (N, K)) on the kernel with decoupled A
    and B rings, A's slot released early (or at the stage's end); K > 64."""
    M, K = A.shape
    N = B.shape[0]
    dt = (torch.bfloat16, torch.int16, torch.uint16)
    pa = _dev(A, "A", dt, (M, K))
    pb = _dev(B, "B", dt, (N, K))
    out = _out(out, M, N, A)
    _check(lib().gemm_bf16_decoupled(pa, pb, ctypes.c_void_p(out.data_ptr()), M, N, K, int(bool(early_release_a)),
                                     _stream(A)))
    return out


def gemm_mx(elem: str, A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor, sB: torch.Tensor,
            K: int | None = None, out: torch.Tensor | None = None,
            la: int = K_MAJOR, lb: int = K_MAJOR) -> torch.Tensor:
    """MXFP8 (elem='e4m3' or 'e5m2'), MXFP6 (elem='e2m3' or 'e3m2', K-major)
    or MXFP4 (elem='e2m1') GEMM with E8M0 scales per 32."""
    return gemm_mx_mixed(elem, elem, A, sA, B, sB, K=K, out=out, la=la, lb=lb)


def gemm_mx_mixed(elem_a: str, elem_b: str, A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor,
                  sB: torch.Tensor, K: int | None = None, out: torch.Tensor | None = None,
                  la: int = K_MAJOR, lb: int = K_MAJOR) -> torch.Tensor:
    """MX GEMM with A's elements in elem_a and B's in elem_b ('e4m3', 'e5m2',
    'e2m1', or the FP6 'e2m3' / 'e3m2', four elements per three bytes; the
    library takes every pairing except FP6 with E2M1, FP6 K-major only)."""
    code_a, code_b = _ELEM[elem_a], _ELEM[elem_b]
    la, lb = _layout(la, "la"), _layout(lb, "lb")
    fp6 = ("e2m3", "e3m2")
    if (elem_a in fp6 and la != K_MAJOR) or (elem_b in fp6 and lb != K_MAJOR):
        raise ValueError("FP6 operands are K-major only")
    pa_ = 2 if elem_a == "e2m1" else 1   # elements per byte (FP6: 4 per 3, K-major)
    pb_ = 2 if elem_b == "e2m1" else 1
    M, N = _rows(A, la, pa_), _rows(B, lb, pb_)
    if K is None:
        K = (A.shape[1] * 4 // 3 if elem_a in fp6 else A.shape[1] * pa_) if la == K_MAJOR else A.shape[0]
    u8 = (torch.uint8,)
    pa = _dev(A, "A", u8, (M, K // 4 * 3) if elem_a in fp6 else _shape(M, K, la, pa_))
    pb = _dev(B, "B", u8, (N, K // 4 * 3) if elem_b in fp6 else _shape(N, K, lb, pb_))
    psa = _dev(sA, "sA", u8, (M, K // 32))
    psb = _dev(sB, "sB", u8, (N, K // 32))
    out = _out(out, M, N, A)
    _check(lib().gemm_mx_mixed(code_a, code_b, pa, psa, pb, psb, ctypes.c_void_p(out.data_ptr()), M, N, K,
                               la, lb, _stream(A)))
    return out


def gemm_nvfp4(A: torch.Tensor, sA: torch.Tensor, tA: float, B: torch.Tensor, sB: torch.Tensor, tB: float,
               out: torch.Tensor | None = None, la: int = K_MAJOR, lb: int = K_MAJOR) -> torch.Tensor:
    """NVFP4 GEMM: packed E2M1 with E4M3 scales per 16 and fp32 tensor scales
    (MN-major operands: (K, M / 2), (K, N / 2) bytes; scales stay (rows, K / 16))."""
    la, lb = _layout(la, "la"), _layout(lb, "lb")
    M, N = _rows(A, la, 2), _rows(B, lb, 2)
    K = A.shape[1] * 2 if la == K_MAJOR else A.shape[0]
    u8 = (torch.uint8,)
    pa = _dev(A, "A", u8, _shape(M, K, la, 2))
    pb = _dev(B, "B", u8, _shape(N, K, lb, 2))
    psa = _dev(sA, "sA", u8, (M, K // 16))
    psb = _dev(sB, "sB", u8, (N, K // 16))
    out = _out(out, M, N, A)
    _check(lib().gemm_nvfp4(pa, psa, float(tA), pb, psb, float(tB), ctypes.c_void_p(out.data_ptr()),
                            M, N, K, la, lb, _stream(A)))
    return out


def nvfp4_fp8_workspace_bytes(M: int, N: int, K: int) -> int:
    """Device workspace gemm_nvfp4_fp8 needs for an M x N x K problem (0 if
    the sizes are invalid)."""
    return int(lib().gemm_nvfp4_fp8_workspace(M, N, K))


def gemm_nvfp4_fp8(A: torch.Tensor, sA: torch.Tensor, tA: float, B: torch.Tensor, sB: torch.Tensor, tB: float,
                   out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """FP8-rate NVFP4 GEMM (opt-in, lossy; see include/dbs.h): the NVFP4
    operands of gemm_nvfp4 are requantised to MXFP8 in ``workspace`` (a uint8
    GPU tensor of at least nvfp4_fp8_workspace_bytes(M, N, K) bytes, allocated
    here if not given) and multiplied at the 8-bit MFMA rate."""
    M, N = A.shape[0], B.shape[0]
    K = A.shape[1] * 2
    u8 = (torch.uint8,)
    pa = _dev(A, "A", u8, (M, K // 2))
    pb = _dev(B, "B", u8, (N, K // 2))
    psa = _dev(sA, "sA", u8, (M, K // 16))
    psb = _dev(sB, "sB", u8, (N, K // 16))
    out = _out(out, M, N, A)
    need = nvfp4_fp8_workspace_bytes(M, N, K)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=A.device)
    _dev(workspace, "workspace", u8, (workspace.numel(),))
    _check(lib().gemm_nvfp4_fp8(pa, psa, float(tA), pb, psb, float(tB), ctypes.c_void_p(out.data_ptr()),
                                M, N, K, K_MAJOR, K_MAJOR, ctypes.c_void_p(workspace.data_ptr()),
                                workspace.numel(), _stream(A)))
    return out


# ---- quantisers (fp32 -> GEMM input formats, on the GPU) ----------------------

def quant_mx(elem: str, x: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """fp32 x (rows, K) -> (codes, E8M0 scales per 32): codes (rows, K) uint8
    for elem='e4m3' or 'e5m2', (rows, K/2) packed for elem='e2m1', (rows,
    3K/4) packed for the FP6 'e2m3' / 'e3m2'; scales (rows, K/32)."""
    code = _ELEM[elem]
    rows, K = x.shape
    px = _dev(x, "x", (torch.float32,), (rows, K))
    width = {"e2m1": K // 2, "e2m3": K // 4 * 3, "e3m2": K // 4 * 3}.get(elem, K)
    codes = torch.empty((rows, width), dtype=torch.uint8, device=x.device)
    scales = torch.empty((rows, K // 32), dtype=torch.uint8, device=x.device)
    _check(lib().quant_mx(code, px, rows, K, ctypes.c_void_p(codes.data_ptr()), ctypes.c_void_p(scales.data_ptr()),
                          _stream(x)))
    return codes, scales


def quant_nvfp4(x: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """fp32 x (rows, K) -> (packed E2M1 codes (rows, K/2), E4M3 scales per 16
    (rows, K/16), tensor scale t as a one-element fp32 GPU tensor)."""
    rows, K = x.shape
    px = _dev(x, "x", (torch.float32,), (rows, K))
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device=x.device)
    scales = torch.empty((rows, K // 16), dtype=torch.uint8, device=x.device)
    t = torch.empty((1,), dtype=torch.float32, device=x.device)
    _check(lib().quant_nvfp4(px, rows, K, ctypes.c_void_p(codes.data_ptr()), ctypes.c_void_p(scales.data_ptr()),
                             ctypes.c_void_p(t.data_ptr()), _stream(x)))
    return codes, scales, t


def quant_bf16(x: torch.Tensor) -> torch.Tensor:
    """fp32 x -> bf16 (round to nearest even), same shape."""
    px = _dev(x, "x", (torch.float32,), tuple(x.shape))
    out = torch.empty(tuple(x.shape), dtype=torch.bfloat16, device=x.device)
    _check(lib().quant_bf16(px, x.numel(), ctypes.c_void_p(out.data_ptr()), _stream(x)))
    return out


# ---- grouped GEMMs (mixture-of-experts layout) ----------------------------------

def _offsets(offsets) -> tuple[ctypes.Array, int]:
    off = [int(v) for v in offsets]
    return (ctypes.c_int64 * len(off))(*off), len(off) - 1


def gemm_grouped_bf16(A: torch.Tensor, B: torch.Tensor, offsets, out: torch.Tensor | None = None) -> torch.Tensor:
    """Group g: D[off[g]:off[g+1]] = A[off[g]:off[g+1]] @ B[g]^T; A (M, K) and
    B (G, N, K) bf16, offsets a host sequence of G + 1 row offsets."""
    off, G = _offsets(offsets)
    M, K = A.shape
    N = B.shape[1]
    dt = (torch.bfloat16, torch.int16, torch.uint16)
    pa = _dev(A, "A", dt, (M, K))
    pb = _dev(B, "B", dt, (G, N, K))
    out = _out(out, M, N, A)
    _check(lib().gemm_grouped_bf16(pa, pb, ctypes.c_void_p(out.data_ptr()), off, G, N, K, _stream(A)))
    return out


def gemm_grouped_mx(elem: str, A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor, sB: torch.Tensor, offsets,
                    K: int | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Grouped MXFP8 / MXFP4 GEMM: A (M, K bytes) with sA (M, K/32); B (G, N, K
    bytes) with sB (G, N, K/32); offsets as for gemm_grouped_bf16."""
    code = _ELEM[elem]
    off, G = _offsets(offsets)
    M, N = A.shape[0], B.shape[1]
    if K is None:
        K = A.shape[1] * (2 if elem == "e2m1" else 1)
    kb = K // 2 if elem == "e2m1" else K
    u8 = (torch.uint8,)
    pa = _dev(A, "A", u8, (M, kb))
    pb = _dev(B, "B", u8, (G, N, kb))
    psa = _dev(sA, "sA", u8, (M, K // 32))
    psb = _dev(sB, "sB", u8, (G, N, K // 32))
    out = _out(out, M, N, A)
    _check(lib().gemm_grouped_mx(code, pa, psa, pb, psb, ctypes.c_void_p(out.data_ptr()), off, G, N, K, _stream(A)))
    return out


def gemm_grouped_nvfp4(A: torch.Tensor, sA: torch.Tensor, tA: float, B: torch.Tensor, sB: torch.Tensor, tB,
                       offsets, out: torch.Tensor | None = None) -> torch.Tensor:
    """Grouped NVFP4 GEMM: one tensor scale tA for A, one tB[g] per group of B."""
    off, G = _offsets(offsets)
    M, N = A.shape[0], B.shape[1]
    K = A.shape[1] * 2
    u8 = (torch.uint8,)
    pa = _dev(A, "A", u8, (M, K // 2))
    pb = _dev(B, "B", u8, (G, N, K // 2))
    psa = _dev(sA, "sA", u8, (M, K // 16))
    psb = _dev(sB, "sB", u8, (G, N, K // 16))
    tb = (ctypes.c_float * G)(*[float(v) for v in tB])
    out = _out(out, M, N, A)
    _check(lib().gemm_grouped_nvfp4(pa, psa, float(tA), pb, psb, tb, ctypes.c_void_p(out.data_ptr()), off, G, N, K,
                                    _stream(A)))
    return out


def gemm_nvfp4_fp8_noalloc(A: torch.Tensor, sA: torch.Tensor, tA: float, B: torch.Tensor, sB: torch.Tensor,
                           tB: float, out: torch.Tensor) -> torch.Tensor:
    """gemm_nvfp4_fp8 without any allocation: the library's static 64 MiB
    device workspace replaces the caller's (see include/dbs.h; problems whose
    workspace would be larger raise DbsError with DBS_EINVAL).  ``out`` (M x N
    bfloat16 on the GPU) is required, since allocating it would defeat the
    purpose."""
    M, N = A.shape[0], B.shape[0]
    K = A.shape[1] * 2
    u8 = (torch.uint8,)
    pa = _dev(A, "A", u8, (M, K // 2))
    pb = _dev(B, "B", u8, (N, K // 2))
    psa = _dev(sA, "sA", u8, (M, K // 16))
    psb = _dev(sB, "sB", u8, (N, K // 16))
    po = _dev(out, "out", (torch.bfloat16,), (M, N))
    _check(lib().gemm_nvfp4_fp8_noalloc(pa, psa, float(tA), pb, psb, float(tB), po, M, N, K, K_MAJOR, K_MAJOR,
                                        _stream(A)))
    return out


def nvfp4_fp6_workspace_bytes(M: int, N: int, K: int) -> int:
    """Device workspace gemm_nvfp4_fp6 needs for an M x N x K problem (0 if
    the sizes are invalid)."""
    return int(lib().gemm_nvfp4_fp6_workspace(M, N, K))


def gemm_nvfp4_fp6(A: torch.Tensor, sA: torch.Tensor, tA: float, B: torch.Tensor, sB: torch.Tensor, tB: float,
                   out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """FP4-rate NVFP4 GEMM (opt-in, lossy; see include/dbs.h): the NVFP4
    operands are requantised to MXFP6 E2M3 in ``workspace`` (a uint8 GPU
    tensor of at least nvfp4_fp6_workspace_bytes(M, N, K) bytes, allocated
    here if not given) and multiplied at the FP6 (= FP4) MFMA rate."""
    M, N = A.shape[0], B.shape[0]
    K = A.shape[1] * 2
    u8 = (torch.uint8,)
    pa = _dev(A, "A", u8, (M, K // 2))
    pb = _dev(B, "B", u8, (N, K // 2))
    psa = _dev(sA, "sA", u8, (M, K // 16))
    psb = _dev(sB, "sB", u8, (N, K // 16))
    out = _out(out, M, N, A)
    need = nvfp4_fp6_workspace_bytes(M, N, K)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=A.device)
    _dev(workspace, "workspace", u8, (workspace.numel(),))
    _check(lib().gemm_nvfp4_fp6(pa, psa, float(tA), pb, psb, float(tB), ctypes.c_void_p(out.data_ptr()),
                                M, N, K, K_MAJOR, K_MAJOR, ctypes.c_void_p(workspace.data_ptr()),
                                workspace.numel(), _stream(A)))
    return out


# ---- mixture-of-experts operators ------------------------------------------------
#
# A routed layer, with W13 (E, 2F, H) the experts' gate and up matrices and W2
# (E, H, F) their way back:
#
#     r = moe_route(logits, k)
#     a = gemm_moe_swiglu_bf16(x, W13, r.offsets, r.rows)       serving
#     h = gemm_moe_bf16(x, W13, r.offsets, r.rows)              training: h is kept
#     a = swiglu(h)
#     y = gemm_moe_bf16(a, W2, r.offsets)
#     out = moe_combine(y, r.slots, r.weights)
#
# Offsets, rows and slots stay on the GPU: no call synchronises.

_REAL = {torch.float32: 0, torch.bfloat16: 1}
_BF16 = (torch.bfloat16,)
_I32 = (torch.int32,)
_F32 = (torch.float32,)


class MoeRouting(NamedTuple):
    """What moe_route returns: experts (T, k) int32 (-1: none), weights (T, k)
    fp32, offsets (E + 1) int32 (expert e's sorted rows), rows (T k) int32
    (token of a sorted row, -1 past the last), slots (T, k) int32 (sorted row
    of a pair, -1: none)."""
    experts: torch.Tensor
    weights: torch.Tensor
    offsets: torch.Tensor
    rows: torch.Tensor
    slots: torch.Tensor


def _dims(t: torch.Tensor, name: str, n: int) -> torch.Size:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != n:
        raise ValueError(f"{name}: {t.dim()} dimensions, expected {n}")
    return t.shape


def _arg(t: torch.Tensor, name: str, dtypes, shape, device: torch.device) -> int:
    """The address of a checked argument (a decoding step makes these calls
    by the dozen: one pass over what is right, _dev for what is not)."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.device == device \
            and device.type == "cuda" and t.is_contiguous():
        return t.data_ptr()
    _dev(t, name, dtypes, shape)
    raise ValueError(f"{name} is on {t.device}, expected {device}")


def _raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# (the same handle without the Stream object around it: 2 us less a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _call(name: str, device: torch.device, *args) -> None:
    """Library call on the current stream of the device, with that device
    current: kernels are launched, and compute units counted, there."""
    f = getattr(lib(), name)
    if device.index == torch.cuda.current_device():
        st = f(*args, _raw_stream(device.index))
    else:
        with torch.cuda.device(device):
            st = f(*args, _raw_stream(device.index))
    if st:
        _check(st)


# An allocation on the current device without the parsing of torch.empty's arguments (moe_route_grouped's five: 13.3 us
# a call, 15.4 with it; quant_i8's two: 8.1, 8.7) and past its dispatcher, so that a profiler has no entry for it.  None
# where torch lacks what it takes to see who else would.
_empty_strided = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)
_WATCHES = tuple(getattr(torch._C, n, None) for n in ("_len_torch_dispatch_stack", "_len_torch_function_stack",
                                                      "_get_deterministic_algorithms"))
if None in _WATCHES:
    _empty_strided = None
else:
    _dispatch_modes, _function_modes, _deterministic = _WATCHES


def _new(shape: tuple, dtype: torch.dtype, device: torch.device) -> torch.Tensor:
    """An uninitialised contiguous tensor of one or two dimensions: torch.empty's
    where a dispatch or function mode sees allocations, or deterministic
    algorithms fill them."""
    if (_empty_strided is None or _dispatch_modes() or _function_modes() or _deterministic()
            or device.index != torch.cuda.current_device()):
        return torch.empty(shape, dtype=dtype, device=device)
    return _empty_strided(shape, (1,) if len(shape) == 1 else (max(shape[1], 1), 1), dtype)


def _given(out: torch.Tensor | None, shape, dtype, device: torch.device) -> torch.Tensor:
    if out is None:
        return _new(shape, dtype, device) if len(shape) <= 2 else torch.empty(shape, dtype=dtype, device=device)
    _arg(out, "out", (dtype,), shape, device)
    return out


_NO_WORKSPACE_TOKENS = 64                     # tokens up to which the library's routers need none


def _routing(T: int, E: int, k: int, device: torch.device, workspace):
    """Outputs of a router, and its workspace (bytes, tensor or None)."""
    kk = min(max(k, 0), E)                    # (the library refuses other k; nothing is sized by them)
    need = int(workspace(T, E, kk)) if T > _NO_WORKSPACE_TOKENS else 0
    r = MoeRouting(_new((T, kk), torch.int32, device), _new((T, kk), torch.float32, device),
                   _new((E + 1,), torch.int32, device), _new((T * kk,), torch.int32, device),
                   _new((T, kk), torch.int32, device))
    return r, need, _new((need,), torch.uint8, device) if need else None


def moe_route(logits: torch.Tensor, k: int, renormalize: bool = True) -> MoeRouting:
    """Router: the k best of E experts for each of T tokens from logits (T, E)
    fp32 or bf16, their softmax weights (over the chosen experts, or over all
    with renormalize=False) and the stable order of the pairs by expert.
    Logits of -inf or NaN close an expert to the token; ties go to the lower
    expert."""
    k = operator.index(k)
    T, E = _dims(logits, "logits", 2)
    dev = logits.device
    pl = _arg(logits, "logits", _REAL, (T, E), dev)
    r, need, ws = _routing(T, E, k, dev, lib().moe_route_workspace)
    _call("moe_route", dev, _REAL[logits.dtype], pl, T, E, k, int(bool(renormalize)), r.experts.data_ptr(),
          r.weights.data_ptr(), r.offsets.data_ptr(), r.rows.data_ptr(), r.slots.data_ptr(),
          None if ws is None else ws.data_ptr(), need)
    return r


_SCORE = {"softmax": 0, "sigmoid": 1}


def _score(scores: str) -> int:
    if scores not in _SCORE:
        raise ValueError(f"scores: {scores!r} not in {tuple(_SCORE)}")
    return _SCORE[scores]


def moe_route_grouped(logits: torch.Tensor, k: int, bias: torch.Tensor | None = None, groups: int = 1,
                      kept_groups: int | None = None, group_best: int = 2, scores: str = "sigmoid",
                      renormalize: bool = True, scale: float = 1.0) -> MoeRouting:
    """Router by groups of experts: scores of the logits (T, E) fp32 or bf16 by
    'sigmoid' or 'softmax'; by score plus ``bias`` (E,) fp32 the best
    ``kept_groups`` (default: all) of ``groups`` runs of E / groups experts are
    kept, by the sum of their ``group_best`` (1 or 2) largest, and the k best
    experts of those chosen.  Weights are ``scale`` times the chosen scores,
    divided by their sum with renormalize=True; the bias is not in them.
    Logits (or biases) of -inf or NaN close an expert.  Equal logits and biases go
    by index; scores with bias that differ by less than 2**-39 of the larger of
    score and |bias| (groups' sums: 2**-37) may come in either order."""
    k, groups = operator.index(k), operator.index(groups)
    kept = groups if kept_groups is None else operator.index(kept_groups)
    T, E = _dims(logits, "logits", 2)
    dev = logits.device
    pl = _arg(logits, "logits", _REAL, (T, E), dev)
    pb = None if bias is None else _arg(bias, "bias", _F32, (E,), dev)
    code = _score(scores)
    r, need, ws = _routing(T, E, k, dev, lib().moe_route_grouped_workspace)
    _call("moe_route_grouped", dev, _REAL[logits.dtype], pl, pb, T, E, k, code, groups, kept, operator.index(group_best),
          int(bool(renormalize)), float(scale), r.experts.data_ptr(), r.weights.data_ptr(), r.offsets.data_ptr(),
          r.rows.data_ptr(), r.slots.data_ptr(), None if ws is None else ws.data_ptr(), need)
    return r


def moe_route_grouped_backward(logits: torch.Tensor, experts: torch.Tensor, dweights: torch.Tensor,
                               scores: str = "sigmoid", renormalize: bool = True, scale: float = 1.0) -> torch.Tensor:
    """Gradient of moe_route_grouped's weights with respect to its logits (T, E):
    experts (T, k) as moe_route_grouped gave them, dweights (T, k) fp32.  (The
    choice, and with it the bias, has none.)"""
    T, E = _dims(logits, "logits", 2)
    k = _dims(experts, "experts", 2)[1]
    dev = logits.device
    pl = _arg(logits, "logits", _REAL, (T, E), dev)
    pe = _arg(experts, "experts", _I32, (T, k), dev)
    pw = _arg(dweights, "dweights", _F32, (T, k), dev)
    code = _score(scores)
    out = torch.empty_like(logits)
    _call("moe_route_grouped_bwd", dev, _REAL[logits.dtype], pl, T, E, k, code, int(bool(renormalize)), float(scale), pe,
          pw, out.data_ptr())
    return out


def moe_route_backward(logits: torch.Tensor, experts: torch.Tensor, dweights: torch.Tensor,
                       renormalize: bool = True) -> torch.Tensor:
    """Gradient of moe_route's weights with respect to its logits (T, E):
    experts (T, k) as moe_route gave them, dweights (T, k) fp32."""
    T, E = _dims(logits, "logits", 2)
    k = _dims(experts, "experts", 2)[1]
    dev = logits.device
    pl = _arg(logits, "logits", _REAL, (T, E), dev)
    pe = _arg(experts, "experts", _I32, (T, k), dev)
    pw = _arg(dweights, "dweights", _F32, (T, k), dev)
    out = torch.empty_like(logits)
    _call("moe_route_bwd", dev, _REAL[logits.dtype], pl, T, E, k, int(bool(renormalize)), pe, pw, out.data_ptr())
    return out


def _sorted(X, offsets, rows, E):
    """Checked addresses of X, offsets and rows, with T, M and K."""
    T, K = _dims(X, "X", 2)
    dev = X.device
    px = _arg(X, "X", _BF16, (T, K), dev)
    po = _arg(offsets, "offsets", _I32, (E + 1,), dev)
    if rows is None:
        return px, po, None, T, T, K
    M = _dims(rows, "rows", 1)[0]
    return px, po, _arg(rows, "rows", _I32, (M,), dev), T, M, K


def gemm_moe_bf16(X: torch.Tensor, W: torch.Tensor, offsets: torch.Tensor, rows: torch.Tensor | None = None,
                  out: torch.Tensor | None = None, lw: int = K_MAJOR) -> torch.Tensor:
    """Experts' products: D[i] = X[rows[i]] @ W[g].T for the sorted rows i of
    expert g (offsets (E + 1) int32 on the GPU).  X (T, K) bf16, gathered
    through rows (M,) int32, or sorted already (rows=None); W (E, N, K), or
    with lw=MN_MAJOR (E, K, N): D[i] = X[rows[i]] @ W[g], the gradient with
    respect to the rows.  Rows of D past offsets[E] are zero."""
    lw = _layout(lw, "lw")
    E, a, b = _dims(W, "W", 3)
    px, po, pr, T, M, K = _sorted(X, offsets, rows, E)
    N = a if lw == K_MAJOR else b
    pw = _arg(W, "W", _BF16, (E, N, K) if lw == K_MAJOR else (E, K, N), X.device)
    out = _given(out, (M, N), torch.bfloat16, X.device)
    _call("gemm_moe_bf16", X.device, px, pw, out.data_ptr(), po, pr, T, M, E, N, K, lw)
    return out


def gemm_moe_swiglu_bf16(X: torch.Tensor, W: torch.Tensor, offsets: torch.Tensor, rows: torch.Tensor | None = None,
                         out: torch.Tensor | None = None) -> torch.Tensor:
    """gemm_moe_bf16 with the gate applied on the way out: W (E, 2F, K) holds
    every expert's gate matrix (first F rows) and up matrix; returns
    silu(gate) * up, (M, F)."""
    E, N, _ = _dims(W, "W", 3)
    if N % 2:
        raise ValueError(f"W: {N} rows per expert, expected an even number (gate and up matrices)")
    px, po, pr, T, M, K = _sorted(X, offsets, rows, E)
    pw = _arg(W, "W", _BF16, (E, N, K), X.device)
    out = _given(out, (M, N // 2), torch.bfloat16, X.device)
    _call("gemm_moe_swiglu_bf16", X.device, px, pw, out.data_ptr(), po, pr, T, M, E, N // 2, K)
    return out


def gemm_moe_dw_bf16(dY: torch.Tensor, X: torch.Tensor, offsets: torch.Tensor, rows: torch.Tensor | None = None,
                     out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
                     accumulate: bool = False) -> torch.Tensor:
    """Gradient with respect to the experts' matrices: dW[g] = dY_g.T @ X_g
    over the sorted rows of expert g; dY (M, N), X (T, K) gathered through rows
    or (M, K); dW (E, N, K) bf16 or fp32.  accumulate=True adds to the fp32
    ``out``; otherwise an expert without rows gets zeros."""
    if out_dtype not in _REAL:
        raise TypeError(f"out_dtype: {out_dtype} not in {tuple(_REAL)}")
    E = _dims(offsets, "offsets", 1)[0] - 1
    px, po, pr, T, M, K = _sorted(X, offsets, rows, E)
    N = _dims(dY, "dY", 2)[1]
    py = _arg(dY, "dY", _BF16, (M, N), X.device)
    if out is not None:
        out_dtype = out.dtype if out.dtype in _REAL else out_dtype
    elif accumulate:
        raise ValueError("accumulate needs out")
    out = _given(out, (E, N, K), out_dtype, X.device)
    _call("gemm_moe_dw_bf16", X.device, _REAL[out_dtype], py, px, out.data_ptr(), po, pr, T, M, E, N, K,
          int(bool(accumulate)))
    return out


def swiglu(H: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """silu(H[:, :F]) * H[:, F:] for H (M, 2F) bf16."""
    M, N = _dims(H, "H", 2)
    if N % 2:
        raise ValueError(f"H: {N} columns, expected an even number")
    ph = _arg(H, "H", _BF16, (M, N), H.device)
    out = _given(out, (M, N // 2), torch.bfloat16, H.device)
    _call("swiglu_bf16", H.device, ph, out.data_ptr(), M, N // 2)
    return out


def swiglu_backward(dA: torch.Tensor, H: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of swiglu with respect to H (M, 2F) from dA (M, F)."""
    M, N = _dims(H, "H", 2)
    if N % 2:
        raise ValueError(f"H: {N} columns, expected an even number")
    ph = _arg(H, "H", _BF16, (M, N), H.device)
    pa = _arg(dA, "dA", _BF16, (M, N // 2), H.device)
    out = _given(out, (M, N), torch.bfloat16, H.device)
    _call("swiglu_bwd_bf16", H.device, pa, ph, out.data_ptr(), M, N // 2)
    return out


def moe_combine(Y: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None = None,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """Back to token order: out[t] = sum over j of weights[t, j] * Y[slots[t, j]]
    (weights=None: ones; slots of -1 add nothing); Y (M, H) bf16, slots (T, k)
    int32, weights (T, k) fp32."""
    M, H = _dims(Y, "Y", 2)
    T, k = _dims(slots, "slots", 2)
    py = _arg(Y, "Y", _BF16, (M, H), Y.device)
    ps = _arg(slots, "slots", _I32, (T, k), Y.device)
    pw = None if weights is None else _arg(weights, "weights", _F32, (T, k), Y.device)
    out = _given(out, (T, H), torch.bfloat16, Y.device)
    _call("moe_combine_bf16", Y.device, py, ps, pw, out.data_ptr(), T, M, k, H)
    return out


def moe_combine_backward(dO: torch.Tensor, Y: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor,
                         offsets: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradients of moe_combine with respect to Y (T k, H) and weights (T, k)
    from dO (T, H); rows of dY past offsets[E] are zero."""
    T, H = _dims(dO, "dO", 2)
    k = _dims(slots, "slots", 2)[1]
    E = _dims(offsets, "offsets", 1)[0] - 1
    dev = dO.device
    pd = _arg(dO, "dO", _BF16, (T, H), dev)
    py = _arg(Y, "Y", _BF16, (T * k, H), dev)
    ps = _arg(slots, "slots", _I32, (T, k), dev)
    pw = _arg(weights, "weights", _F32, (T, k), dev)
    po = _arg(offsets, "offsets", _I32, (E + 1,), dev)
    dY = torch.empty_like(Y)
    dweights = torch.empty_like(weights)
    _call("moe_combine_bwd_bf16", dev, pd, py, ps, pw, po, E, dY.data_ptr(), dweights.data_ptr(), T, k, H)
    return dY, dweights


# ---- products in 8-bit integers ---------------------------------------------------
#
# A matrix product with int8 codes and a scale for each row (token) of A and each
# row (channel) of B, and a routed layer served that way:
#
#     qw, sw = quant_i8(W)                                    once
#     qx, sx = quant_i8(x)
#     y = gemm_i8(qx, sx, qw, sw)
#
#     r = moe_route_grouped(logits, k, bias, groups, kept_groups)
#     a = gemm_moe_swiglu_i8(qx, sx, q13, s13, r.offsets, r.rows)
#     qa, sa = quant_i8(a)
#     out = moe_combine(gemm_moe_i8(qa, sa, q2, s2, r.offsets), r.slots, r.weights)

_I8 = (torch.int8,)


def quant_i8(x: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """Rows x (M, K) fp32 or bf16 -> (codes (M, K) int8, scales (M,) fp32): scale =
    amax / 127, codes the nearest whole numbers to 127 x / amax (ties to even).
    A row of zeros has scale 0, one with an infinity or a NaN scale NaN."""
    M, K = _dims(x, "x", 2)
    dev = x.device
    px = _arg(x, "x", _REAL, (M, K), dev)
    codes, scales = _new((M, K), torch.int8, dev), _new((M,), torch.float32, dev)
    _call("quant_i8", dev, _REAL[x.dtype], px, M, K, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def gemm_i8(A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor, sB: torch.Tensor, out: torch.Tensor | None = None,
            out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """D[m, n] = sA[m] * sB[n] * sum over k of A[m, k] * B[n, k]: codes A (M, K) and B
    (N, K) int8, scales sA (M,) and sB (N,) fp32; the sum in whole numbers; D (M, N)
    bf16 or fp32 (or ``out``'s type)."""
    M, K = _dims(A, "A", 2)
    N = _dims(B, "B", 2)[0]
    dev = A.device
    pa, psa = _arg(A, "A", _I8, (M, K), dev), _arg(sA, "sA", _F32, (M,), dev)
    pb, psb = _arg(B, "B", _I8, (N, K), dev), _arg(sB, "sB", _F32, (N,), dev)
    if out is not None and isinstance(out, torch.Tensor):
        out_dtype = out.dtype if out.dtype in _REAL else out_dtype
    if out_dtype not in _REAL:
        raise TypeError(f"out_dtype: {out_dtype} not in {tuple(_REAL)}")
    out = _given(out, (M, N), out_dtype, dev)
    _call("gemm_i8", dev, _REAL[out_dtype], pa, psa, pb, psb, out.data_ptr(), M, N, K)
    return out


def _sorted_i8(X, sX, offsets, rows, E):
    """Checked addresses of X, sX, offsets and rows, with T, M and K."""
    T, K = _dims(X, "X", 2)
    dev = X.device
    px, ps = _arg(X, "X", _I8, (T, K), dev), _arg(sX, "sX", _F32, (T,), dev)
    po = _arg(offsets, "offsets", _I32, (E + 1,), dev)
    if rows is None:
        return px, ps, po, None, T, T, K
    M = _dims(rows, "rows", 1)[0]
    return px, ps, po, _arg(rows, "rows", _I32, (M,), dev), T, M, K


def gemm_moe_i8(X: torch.Tensor, sX: torch.Tensor, W: torch.Tensor, sW: torch.Tensor, offsets: torch.Tensor,
                rows: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """gemm_moe_bf16 in 8-bit integers: D[i] = sX[r] * sW[g] * (X[r] @ W[g].T), r =
    rows[i], for the sorted rows i of expert g.  X (T, K) int8 gathered through
    rows (M,) int32, or sorted already (rows=None), sX (T,) fp32; W (E, N, K)
    int8, sW (E, N) fp32; D (M, N) bf16.  Rows of D past offsets[E] are zero."""
    E, N, _ = _dims(W, "W", 3)
    px, ps, po, pr, T, M, K = _sorted_i8(X, sX, offsets, rows, E)
    dev = X.device
    pw, pt = _arg(W, "W", _I8, (E, N, K), dev), _arg(sW, "sW", _F32, (E, N), dev)
    out = _given(out, (M, N), torch.bfloat16, dev)
    _call("gemm_moe_i8", dev, px, ps, pw, pt, out.data_ptr(), po, pr, T, M, E, N, K)
    return out


def gemm_moe_swiglu_i8(X: torch.Tensor, sX: torch.Tensor, W: torch.Tensor, sW: torch.Tensor, offsets: torch.Tensor,
                       rows: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """gemm_moe_i8 with the gate applied on the way out: W (E, 2F, K) holds every
    expert's gate matrix (first F rows) and up matrix; returns silu(gate) * up,
    (M, F) bf16."""
    E, N, _ = _dims(W, "W", 3)
    if N % 2:
        raise ValueError(f"W: {N} rows per expert, expected an even number (gate and up matrices)")
    px, ps, po, pr, T, M, K = _sorted_i8(X, sX, offsets, rows, E)
    dev = X.device
    pw, pt = _arg(W, "W", _I8, (E, N, K), dev), _arg(sW, "sW", _F32, (E, N), dev)
    out = _given(out, (M, N // 2), torch.bfloat16, dev)
    _call("gemm_moe_swiglu_i8", dev, px, ps, pw, pt, out.data_ptr(), po, pr, T, M, E, N // 2, K)
    return out
