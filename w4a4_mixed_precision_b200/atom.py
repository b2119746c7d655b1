"""Python binding of the C ABI in include/atom.h (argument marshalling only).

Every function here forwards to `libatom_b200.so`: the tensors' device
pointers, sizes and the current CUDA stream go in, a status code comes back,
and any status other than ATOM_OK raises AtomError. There is no fallback: if
the library is missing or the device is not an sm_100 part, the calls fail.

Layouts (see include/atom.h): for R rows of K channels with G = K/128,
  q4     uint8  [R, (K-128)/2]   two INT4 codes per byte, element 2i low nibble
  q8     int8   [R, 128]         INT8 codes of the outlier channels, list order
  scales float32 [G, R]          group-major scales (last row = outlier group)
"""
from __future__ import annotations

import ctypes as ct
import functools
import os
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libatom_b200.so")

STATUS = {
    0: "ATOM_OK",
    1: "ATOM_ERR_INVALID_ARG",
    2: "ATOM_ERR_SHAPE",
    3: "ATOM_ERR_ALIGN",
    4: "ATOM_ERR_UNSUPPORTED",
    5: "ATOM_ERR_CUDA",
    6: "ATOM_ERR_TIMEOUT",
}

N_OUTLIER = 128
GROUP = 128

#: every entry point include/atom.h declares, with its argument types
SIGNATURES = {
    "atom_reorder_quant": ([ct.c_void_p, ct.c_int64, ct.c_int64, ct.c_int64, ct.c_void_p,
                            ct.c_int32, ct.c_int32, ct.c_void_p, ct.c_void_p, ct.c_void_p,
                            ct.c_void_p], ct.c_int),
    "atom_reorder_quant_a8": ([ct.c_void_p, ct.c_int64, ct.c_int64, ct.c_int64, ct.c_void_p,
                               ct.c_int32, ct.c_int32, ct.c_void_p, ct.c_void_p, ct.c_void_p],
                              ct.c_int),
    "atom_w4a8_gemm": ([ct.c_void_p] * 6 + [ct.c_int64, ct.c_int64, ct.c_int64, ct.c_int32,
                                            ct.c_int32, ct.c_void_p], ct.c_int),
    "atom_w4a8_gemm_partials": ([ct.c_void_p] * 7 + [ct.c_int64, ct.c_int64, ct.c_int64,
                                                     ct.c_int32, ct.c_int32, ct.c_void_p],
                                ct.c_int),
    "atom_quant_weights": ([ct.c_void_p, ct.c_int64, ct.c_int64, ct.c_int64, ct.c_void_p,
                            ct.c_int32, ct.c_int32, ct.c_void_p, ct.c_void_p, ct.c_void_p,
                            ct.c_void_p], ct.c_int),
    "atom_w4a4_gemm": ([ct.c_void_p] * 7 + [ct.c_int64, ct.c_int64, ct.c_int64, ct.c_int32,
                                            ct.c_int32, ct.c_void_p, ct.c_size_t, ct.c_void_p],
                       ct.c_int),
    "atom_w4a4_gemm_partials": ([ct.c_void_p] * 8 + [ct.c_int64, ct.c_int64, ct.c_int64,
                                                     ct.c_int32, ct.c_int32, ct.c_void_p],
                                ct.c_int),
    "atom_w4a4_gemm_quant": ([ct.c_void_p] * 6 + [ct.c_int64, ct.c_int64, ct.c_int64, ct.c_int32,
                              ct.c_int32] + [ct.c_void_p] * 4, ct.c_int),
    "atom_gemm_workspace_bytes": ([ct.c_int64, ct.c_int64, ct.c_int64], ct.c_size_t),
    "atom_tiled_weights_bytes": ([ct.c_int64, ct.c_int64], ct.c_size_t),
    "atom_pack_weights_tiled": ([ct.c_void_p, ct.c_int64, ct.c_int64, ct.c_void_p, ct.c_void_p],
                                ct.c_int),
    "atom_unpack_weights_tiled": ([ct.c_void_p, ct.c_int64, ct.c_int64, ct.c_void_p, ct.c_void_p],
                                  ct.c_int),
    "atom_w4a4_gemm_tiled": ([ct.c_void_p] * 7 + [ct.c_int64, ct.c_int64, ct.c_int64, ct.c_int32,
                                                  ct.c_int32, ct.c_void_p, ct.c_size_t,
                                                  ct.c_void_p], ct.c_int),
    "atom_w4a4_gemm_noalloc": ([ct.c_void_p] * 7 + [ct.c_int64, ct.c_int64, ct.c_int64, ct.c_int32,
                                                    ct.c_int32, ct.c_void_p], ct.c_int),
    "atom_w8a8_gemm": ([ct.c_void_p] * 5 + [ct.c_int64, ct.c_int64, ct.c_int64, ct.c_void_p],
                       ct.c_int),
    "atom_kv_quant": ([ct.c_void_p, ct.c_int64, ct.c_void_p, ct.c_void_p, ct.c_void_p], ct.c_int),
    "atom_kv_dequant": ([ct.c_void_p, ct.c_void_p, ct.c_int64, ct.c_void_p, ct.c_void_p],
                        ct.c_int),
    "atom_kv4_append": ([ct.c_void_p, ct.c_int64, ct.c_int64] * 2 + [ct.c_int64] +
                        [ct.c_void_p] * 3, ct.c_int),
    "atom_kv4_gather": ([ct.c_void_p] * 2 + [ct.c_int64] + [ct.c_void_p] * 3, ct.c_int),
    "atom_kv4_attention_workspace_bytes": ([ct.c_int64] * 4, ct.c_size_t),
    "atom_kv4_attention": ([ct.c_void_p] + [ct.c_int64] * 4 + [ct.c_void_p] * 2 +
                           [ct.c_int32, ct.c_float] + [ct.c_void_p] * 3 +
                           [ct.c_size_t, ct.c_void_p], ct.c_int),
    "atom_kv4_attention_weights": ([ct.c_void_p] + [ct.c_int64] * 4 + [ct.c_void_p] * 3 +
                                   [ct.c_int32, ct.c_float] + [ct.c_void_p] * 2 +
                                   [ct.c_int64, ct.c_void_p], ct.c_int),
    "atom_kv4_evict": ([ct.c_void_p, ct.c_int64] + [ct.c_void_p] * 2 + [ct.c_int64] * 2 +
                       [ct.c_void_p] * 2 + [ct.c_int64] * 2 + [ct.c_void_p] * 3 +
                       [ct.c_int64, ct.c_void_p], ct.c_int),
    "atom_debug_wait_timeout": ([ct.c_uint64, ct.c_void_p], ct.c_int),
    "atom_probe_mma_i8": ([ct.c_int64, ct.POINTER(ct.c_int32), ct.c_void_p], ct.c_int),
    "atom_device_status": ([ct.c_int], ct.c_int),
    "atom_status_string": ([ct.c_int], ct.c_char_p),
    "atom_version": ([], ct.c_int),
}


class AtomError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")
        self.status = status


_lib: Optional[ct.CDLL] = None


def lib() -> ct.CDLL:
    """Load libatom_b200.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run `python -m w4a4_mixed_precision_b200.build`")
        handle = ct.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            f = getattr(handle, name)
            f.argtypes = args
            f.restype = res
        _lib = handle
    return _lib


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise AtomError(fn, status)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev(t: torch.Tensor, dtype: torch.dtype, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


MAX_K = 32768   # the largest K the library accepts (include/atom.h)


def _valid_k(K: int) -> bool:
    return K % GROUP == 0 and 2 * GROUP <= K <= MAX_K


def _expect_shape(t: torch.Tensor, shape, name: str) -> None:
    if t.shape != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _check_quantized(q, K: int, name: str, rows: Optional[int] = None) -> None:
    """Shapes of a quantized operand (Quantized) for K. Only checked for a K the
    library accepts: it reports any other K itself, with its own status."""
    if not _valid_k(K):
        return
    rows = q.q4.shape[0] if rows is None else rows
    _expect_shape(q.q4, (rows, (K - N_OUTLIER) // 2), name + ".q4")
    _expect_shape(q.q8, (rows, N_OUTLIER), name + ".q8")
    _expect_shape(q.scales, (K // GROUP, rows), name + ".scales")


def _check_quantized_a8(q, K: int, name: str, rows: Optional[int] = None) -> None:
    """Shapes of W4A8 activations (QuantizedA8) for K, as _check_quantized."""
    if not _valid_k(K):
        return
    rows = q.q8.shape[0] if rows is None else rows
    _expect_shape(q.q8, (rows, K), name + ".q8")
    _expect_shape(q.scales, (K // GROUP, rows), name + ".scales")


class Quantized(NamedTuple):
    """One quantized operand: INT4 codes, INT8 outlier codes, group-major scales."""
    q4: torch.Tensor
    q8: torch.Tensor
    scales: torch.Tensor

    @property
    def rows(self) -> int:
        return self.q4.shape[0]


def empty_quantized(rows: int, K: int, device) -> Quantized:
    return Quantized(torch.empty((rows, (K - N_OUTLIER) // 2), dtype=torch.uint8, device=device),
                     torch.empty((rows, N_OUTLIER), dtype=torch.int8, device=device),
                     torch.empty((K // GROUP, rows), dtype=torch.float32, device=device))


def _quant(fn: str, x: torch.Tensor, outlier_idx: torch.Tensor, out: Optional[Quantized], stream):
    if x.dim() != 2:
        raise ValueError("input must be 2-D [rows, K]")
    rows, K = x.shape
    if x.stride(1) != 1:
        raise ValueError("input rows must be contiguous")
    if out is None:
        out = empty_quantized(rows, K, x.device)
    _check_quantized(out, K, "out", rows)
    if not x.is_cuda or x.dtype != torch.float16:
        raise ValueError("input must be a CUDA float16 tensor")
    st = getattr(lib(), fn)(x.data_ptr(), rows, K, x.stride(0),
                            _dev(outlier_idx, torch.int32, "outlier_idx"), outlier_idx.numel(),
                            GROUP, _dev(out.q4, torch.uint8, "q4"), _dev(out.q8, torch.int8, "q8"),
                            _dev(out.scales, torch.float32, "scales"), _stream(stream))
    _check(fn, st)
    return out


def atom_reorder_quant(x: torch.Tensor, outlier_idx: torch.Tensor,
                       out: Optional[Quantized] = None, stream=None) -> Quantized:
    """Fused outlier reorder + INT4/INT8 quantization of fp16 activations [M, K]."""
    return _quant("atom_reorder_quant", x, outlier_idx, out, stream)


class QuantizedA8(NamedTuple):
    """W4A8 activations: INT8 codes [rows, K] in reordered order, scales [K/128, rows]."""
    q8: torch.Tensor
    scales: torch.Tensor

    @property
    def rows(self) -> int:
        return self.q8.shape[0]


def atom_reorder_quant_a8(x: torch.Tensor, outlier_idx: torch.Tensor,
                          out: Optional[QuantizedA8] = None, stream=None) -> QuantizedA8:
    """W4A8 activations: the outlier reorder, then INT8 in every group (see include/atom.h)."""
    if x.dim() != 2 or x.stride(1) != 1 or not x.is_cuda or x.dtype != torch.float16:
        raise ValueError("input must be a 2-D CUDA float16 tensor with contiguous rows")
    rows, K = x.shape
    if out is None:
        out = QuantizedA8(torch.empty((rows, K), dtype=torch.int8, device=x.device),
                          torch.empty((K // GROUP, rows), dtype=torch.float32, device=x.device))
    _check_quantized_a8(out, K, "out", rows)
    st = lib().atom_reorder_quant_a8(x.data_ptr(), rows, K, x.stride(0),
                                     _dev(outlier_idx, torch.int32, "outlier_idx"),
                                     outlier_idx.numel(), GROUP, _dev(out.q8, torch.int8, "q8"),
                                     _dev(out.scales, torch.float32, "scales"), _stream(stream))
    _check("atom_reorder_quant_a8", st)
    return out


def atom_w4a8_gemm(qa: QuantizedA8, qw: Quantized, K: int, y: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """W4A8: Y fp16 [M, N] from INT8 activations and the W4A4 weights (see include/atom.h)."""
    M, N = qa.rows, qw.rows
    _check_quantized_a8(qa, K, "qa")
    _check_quantized(qw, K, "qw")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=qa.q8.device)
    _expect_shape(y, (M, N), "y")
    st = lib().atom_w4a8_gemm(
        _dev(qa.q8, torch.int8, "qa8"), _dev(qa.scales, torch.float32, "sa"),
        _dev(qw.q4, torch.uint8, "qw4"), _dev(qw.q8, torch.int8, "qw8"),
        _dev(qw.scales, torch.float32, "sw"), _dev(y, torch.float16, "y"),
        M, N, K, N_OUTLIER, GROUP, _stream(stream))
    _check("atom_w4a8_gemm", st)
    return y


def atom_w4a8_gemm_partials(qa: QuantizedA8, qw: Quantized, K: int, stream=None):
    """Debug entry of the W4A8 GEMM: per-group int32 partial sums [G, M, N] and Y."""
    M, N = qa.rows, qw.rows
    dev = qa.q8.device
    _check_quantized_a8(qa, K, "qa")
    _check_quantized(qw, K, "qw")
    partials = torch.empty((K // GROUP, M, N), dtype=torch.int32, device=dev)
    y = torch.empty((M, N), dtype=torch.float16, device=dev)
    st = lib().atom_w4a8_gemm_partials(
        _dev(qa.q8, torch.int8, "qa8"), _dev(qa.scales, torch.float32, "sa"),
        _dev(qw.q4, torch.uint8, "qw4"), _dev(qw.q8, torch.int8, "qw8"),
        _dev(qw.scales, torch.float32, "sw"), _dev(partials, torch.int32, "partials"),
        _dev(y, torch.float16, "y"), M, N, K, N_OUTLIER, GROUP, _stream(stream))
    _check("atom_w4a8_gemm_partials", st)
    return partials, y


def atom_quant_weights(w: torch.Tensor, outlier_idx: torch.Tensor,
                       out: Optional[Quantized] = None, stream=None) -> Quantized:
    """Offline weight quantization of fp16 W [N, K] (same encoding as the activations)."""
    return _quant("atom_quant_weights", w, outlier_idx, out, stream)


def gemm_workspace(M: int, N: int, K: int, device) -> Optional[torch.Tensor]:
    """Scratch for atom_w4a4_gemm on this shape (None when it needs none)."""
    n = atom_gemm_workspace_bytes(M, N, K)
    return torch.empty(n, dtype=torch.uint8, device=device) if n > 0 else None


def atom_w4a4_gemm(qa: Quantized, qw: Quantized, K: int, y: Optional[torch.Tensor] = None,
                   stream=None, workspace: Optional[torch.Tensor] = None,
                   split: bool = True) -> torch.Tensor:
    """Y fp16 [M, N] = sum_g sa*sw*P_g (see include/atom.h).

    `workspace` (uint8 CUDA tensor) is the scratch a split-K launch uses; when it
    is None and `split` is true, one of atom_gemm_workspace_bytes() bytes is
    allocated here. `split=False` runs without a workspace (no K split)."""
    M, N = qa.rows, qw.rows
    dev = qa.q4.device
    _check_quantized(qa, K, "qa")
    _check_quantized(qw, K, "qw")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=dev)
    _expect_shape(y, (M, N), "y")
    if workspace is None and split:
        workspace = gemm_workspace(M, N, K, dev)
    ws_ptr, ws_bytes = (None, 0) if workspace is None or not split else (
        _dev(workspace, torch.uint8, "workspace"), workspace.numel())
    st = lib().atom_w4a4_gemm(
        _dev(qa.q4, torch.uint8, "qa4"), _dev(qa.q8, torch.int8, "qa8"),
        _dev(qa.scales, torch.float32, "sa"), _dev(qw.q4, torch.uint8, "qw4"),
        _dev(qw.q8, torch.int8, "qw8"), _dev(qw.scales, torch.float32, "sw"),
        _dev(y, torch.float16, "y"), M, N, K, N_OUTLIER, GROUP, ws_ptr, ws_bytes, _stream(stream))
    _check("atom_w4a4_gemm", st)
    return y


class TiledWeights(NamedTuple):
    """Quantized weights with the INT4 codes in the tiled layout (see
    include/atom.h): q4t uint8 [ceil(N/128), K/128 - 1, 128, 64]; q8 and scales as
    in Quantized."""
    q4t: torch.Tensor
    q8: torch.Tensor
    scales: torch.Tensor

    @property
    def rows(self) -> int:
        return self.q8.shape[0]


def _tiled_shape(N: int, K: int):
    return ((N + 127) // 128, K // GROUP - 1, 128, 64)


def atom_pack_weights_tiled(qw: Quantized, K: int, stream=None) -> TiledWeights:
    """One-off repack of quantized weights into the tiled layout."""
    N = qw.rows
    _check_quantized(qw, K, "qw")
    q4t = torch.empty(_tiled_shape(N, K), dtype=torch.uint8, device=qw.q4.device)
    st = lib().atom_pack_weights_tiled(_dev(qw.q4, torch.uint8, "qw4"), N, K,
                                       _dev(q4t, torch.uint8, "qw4t"), _stream(stream))
    _check("atom_pack_weights_tiled", st)
    return TiledWeights(q4t, qw.q8, qw.scales)


def atom_unpack_weights_tiled(qwt: TiledWeights, K: int, stream=None) -> torch.Tensor:
    """The row layout [N, (K-128)/2] of tiled INT4 weight codes (the inverse repack)."""
    N = qwt.rows
    if _valid_k(K):
        _expect_shape(qwt.q4t, _tiled_shape(N, K), "qw4t")
    q4 = torch.empty((N, (K - N_OUTLIER) // 2), dtype=torch.uint8, device=qwt.q4t.device)
    st = lib().atom_unpack_weights_tiled(_dev(qwt.q4t, torch.uint8, "qw4t"), N, K,
                                         _dev(q4, torch.uint8, "qw4"), _stream(stream))
    _check("atom_unpack_weights_tiled", st)
    return q4


def atom_w4a4_gemm_tiled(qa: Quantized, qwt: TiledWeights, K: int,
                         y: Optional[torch.Tensor] = None, stream=None,
                         workspace: Optional[torch.Tensor] = None,
                         split: bool = True) -> torch.Tensor:
    """atom_w4a4_gemm with the weights in the tiled layout (bit-identical Y)."""
    M, N = qa.rows, qwt.rows
    dev = qa.q4.device
    _check_quantized(qa, K, "qa")
    if _valid_k(K):
        _expect_shape(qwt.q4t, _tiled_shape(N, K), "qw4t")
        _expect_shape(qwt.q8, (N, N_OUTLIER), "qw.q8")
        _expect_shape(qwt.scales, (K // GROUP, N), "qw.scales")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=dev)
    _expect_shape(y, (M, N), "y")
    if workspace is None and split:
        workspace = gemm_workspace(M, N, K, dev)
    ws_ptr, ws_bytes = (None, 0) if workspace is None or not split else (
        _dev(workspace, torch.uint8, "workspace"), workspace.numel())
    st = lib().atom_w4a4_gemm_tiled(
        _dev(qa.q4, torch.uint8, "qa4"), _dev(qa.q8, torch.int8, "qa8"),
        _dev(qa.scales, torch.float32, "sa"), _dev(qwt.q4t, torch.uint8, "qw4t"),
        _dev(qwt.q8, torch.int8, "qw8"), _dev(qwt.scales, torch.float32, "sw"),
        _dev(y, torch.float16, "y"), M, N, K, N_OUTLIER, GROUP, ws_ptr, ws_bytes, _stream(stream))
    _check("atom_w4a4_gemm_tiled", st)
    return y


def atom_tiled_weights_bytes(N: int, K: int) -> int:
    return int(lib().atom_tiled_weights_bytes(N, K))


def atom_w4a4_gemm_noalloc(qa: Quantized, qw: Quantized, K: int,
                           y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """atom_w4a4_gemm for callers that cannot allocate device memory around the
    call (a runtime whose device memory all sits in a fixed pool, a C caller
    without an allocator): a split of K keeps its partials in the library's
    fixed 8 MiB device array (see include/atom.h). Pass `y` to keep this wrapper
    allocation-free as well."""
    M, N = qa.rows, qw.rows
    _check_quantized(qa, K, "qa")
    _check_quantized(qw, K, "qw")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=qa.q4.device)
    _expect_shape(y, (M, N), "y")
    st = lib().atom_w4a4_gemm_noalloc(
        _dev(qa.q4, torch.uint8, "qa4"), _dev(qa.q8, torch.int8, "qa8"),
        _dev(qa.scales, torch.float32, "sa"), _dev(qw.q4, torch.uint8, "qw4"),
        _dev(qw.q8, torch.int8, "qw8"), _dev(qw.scales, torch.float32, "sw"),
        _dev(y, torch.float16, "y"), M, N, K, N_OUTLIER, GROUP, _stream(stream))
    _check("atom_w4a4_gemm_noalloc", st)
    return y


def atom_w4a4_gemm_partials(qa: Quantized, qw: Quantized, K: int,
                            partials: Optional[torch.Tensor] = None,
                            y: Optional[torch.Tensor] = None, want_y: bool = True,
                            stream=None):
    """Debug entry: per-group int32 partial sums [G, M, N] (and Y unless want_y is False)."""
    M, N = qa.rows, qw.rows
    dev = qa.q4.device
    _check_quantized(qa, K, "qa")
    _check_quantized(qw, K, "qw")
    if partials is None:
        partials = torch.empty((K // GROUP, M, N), dtype=torch.int32, device=dev)
    if _valid_k(K):
        _expect_shape(partials, (K // GROUP, M, N), "partials")
    if want_y and y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=dev)
    if want_y:
        _expect_shape(y, (M, N), "y")
    st = lib().atom_w4a4_gemm_partials(
        _dev(qa.q4, torch.uint8, "qa4"), _dev(qa.q8, torch.int8, "qa8"),
        _dev(qa.scales, torch.float32, "sa"), _dev(qw.q4, torch.uint8, "qw4"),
        _dev(qw.q8, torch.int8, "qw8"), _dev(qw.scales, torch.float32, "sw"),
        _dev(partials, torch.int32, "partials"),
        _dev(y, torch.float16, "y") if want_y else None,
        M, N, K, N_OUTLIER, GROUP, _stream(stream))
    _check("atom_w4a4_gemm_partials", st)
    return partials, y


def atom_w4a4_gemm_quant(qa: Quantized, qw: Quantized, K: int, out: Optional[Quantized] = None,
                         stream=None) -> Quantized:
    """The GEMM with the next layer's activation quantization in its epilogue: the codes
    and scales atom_reorder_quant would write for Y (unsplit, fp16) with Y's last 128
    columns as the outlier channels (see include/atom.h). N must be a multiple of 128."""
    M, N = qa.rows, qw.rows
    _check_quantized(qa, K, "qa")
    _check_quantized(qw, K, "qw")
    if out is None:
        out = empty_quantized(M, N, qa.q4.device)
    _check_quantized(out, N, "out", M)   # Y's N is the next layer's K
    st = lib().atom_w4a4_gemm_quant(
        _dev(qa.q4, torch.uint8, "qa4"), _dev(qa.q8, torch.int8, "qa8"),
        _dev(qa.scales, torch.float32, "sa"), _dev(qw.q4, torch.uint8, "qw4"),
        _dev(qw.q8, torch.int8, "qw8"), _dev(qw.scales, torch.float32, "sw"),
        M, N, K, N_OUTLIER, GROUP,
        _dev(out.q4, torch.uint8, "qy4"), _dev(out.q8, torch.int8, "qy8"),
        _dev(out.scales, torch.float32, "sy"), _stream(stream))
    _check("atom_w4a4_gemm_quant", st)
    return out


def atom_w8a8_gemm(qa: torch.Tensor, sa: torch.Tensor, qw: torch.Tensor, sw: torch.Tensor,
                   y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """W8A8 comparator: y = fp16(float(qa @ qw^T) * sa[:, None] * sw[None, :]) with int8
    qa [M, K], qw [N, K] and fp32 scales sa [M], sw [N] (see include/atom.h)."""
    M, K = qa.shape
    N = qw.shape[0]
    if qw.shape[1] != K or sa.shape != (M,) or sw.shape != (N,):
        raise ValueError("atom_w8a8_gemm: shapes must be qa [M, K], qw [N, K], sa [M], sw [N]")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=qa.device)
    st = lib().atom_w8a8_gemm(
        _dev(qa, torch.int8, "qa"), _dev(sa, torch.float32, "sa"), _dev(qw, torch.int8, "qw"),
        _dev(sw, torch.float32, "sw"), _dev(y, torch.float16, "y"), M, N, K, _stream(stream))
    _check("atom_w8a8_gemm", st)
    return y


def atom_kv_quant(x: torch.Tensor, q4: Optional[torch.Tensor] = None,
                  scales: Optional[torch.Tensor] = None, stream=None):
    """INT4 KV-cache quantization of fp16 [..., 128] (one group per 128-vector):
    returns (q4 uint8 [..., 64], scales fp32 [...]) (see include/atom.h)."""
    if x.shape[-1] != 128:
        raise ValueError("atom_kv_quant: the last axis must be head_dim = 128")
    lead = tuple(x.shape[:-1])
    groups = x.numel() // 128
    if q4 is None:
        q4 = torch.empty(lead + (64,), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(lead, dtype=torch.float32, device=x.device)
    st = lib().atom_kv_quant(_dev(x, torch.float16, "x"), groups, _dev(q4, torch.uint8, "q4"),
                             _dev(scales, torch.float32, "scales"), _stream(stream))
    _check("atom_kv_quant", st)
    return q4, scales


def atom_kv_dequant(q4: torch.Tensor, scales: torch.Tensor, out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """fp16 [..., 128] from atom_kv_quant's codes and scales."""
    if q4.shape[-1] != 64 or tuple(scales.shape) != tuple(q4.shape[:-1]):
        raise ValueError("atom_kv_dequant: q4 [..., 64] and scales [...] must match")
    groups = scales.numel()
    if out is None:
        out = torch.empty(tuple(q4.shape[:-1]) + (128,), dtype=torch.float16, device=q4.device)
    st = lib().atom_kv_dequant(_dev(q4, torch.uint8, "q4"), _dev(scales, torch.float32, "scales"),
                               groups, _dev(out, torch.float16, "out"), _stream(stream))
    _check("atom_kv_dequant", st)
    return out


class _CacheStruct(ct.Structure):
    _fields_ = ([(n, ct.c_void_p) for n in ("k4", "ks", "v4", "vs")] +
                [(n, ct.c_int64) for n in ("pages", "page_size", "heads", "page_stride",
                                           "token_stride", "head_stride")])


class _BatchStruct(ct.Structure):
    _fields_ = [("block_table", ct.c_void_p), ("table_stride", ct.c_int64),
                ("max_pages", ct.c_int64), ("kv_lens", ct.c_void_p), ("cu_q", ct.c_void_p),
                ("batch", ct.c_int64), ("max_q", ct.c_int64)]


def _kv4_check(t: torch.Tensor, dtype: torch.dtype, name: str, device=None) -> torch.Tensor:
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return t


def _kv4_rows(t: torch.Tensor, heads: Optional[int], name: str, device):
    """Pointer, token stride and head stride of fp16 [rows, heads, 128]; a dimension of
    one has no stride of its own."""
    shape = t.shape
    if len(shape) != 3 or shape[2] != 128 or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must have shape (rows, {heads or 'heads'}, 128), got "
                         f"{tuple(shape)}")
    _kv4_check(t, torch.float16, name, device)
    a, b, c = t.stride()
    if c != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    return t.data_ptr(), a if shape[0] > 1 else 0, b if shape[1] > 1 else 0


def _kv4_contiguous(t: torch.Tensor, dtype: torch.dtype, shape, name: str, device) -> int:
    _expect_shape(t, shape, name)
    _kv4_check(t, dtype, name, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _kv4_output(t: Optional[torch.Tensor], like: torch.Tensor, dtype: torch.dtype, shape, name: str,
                device) -> torch.Tensor:
    """The caller's output tensor, checked, or a new one on `like`'s device."""
    if t is None:   # (naming a shape, then a type, costs from half a microsecond to some)
        if like.dtype != dtype:
            return like.new_empty(shape, dtype=dtype)
        same = like.is_contiguous() and like.shape == shape
        return torch.empty_like(like) if same else like.new_empty(shape)
    _kv4_contiguous(t, dtype, shape, name, device)
    return t


class KV4Cache:
    """A paged INT4 KV cache (see include/atom.h): codes k4, v4 uint8 [pages, page_size,
    heads, 64] and scales ks, vs float32 [pages, page_size, heads], all on one device, in
    any layout that keeps a vector's 64 bytes together and is the same for the four (views
    of [pages, heads, page_size, ...] storage, for example). The object holds the tensors'
    addresses: their storage must stay in place."""

    def __init__(self, k4: torch.Tensor, ks: torch.Tensor, v4: torch.Tensor, vs: torch.Tensor):
        if k4.dim() != 4 or k4.shape[3] != 64:
            raise ValueError(f"k4 must have shape (pages, page_size, heads, 64), got "
                             f"{tuple(k4.shape)}")
        lead = tuple(k4.shape[:3])
        _expect_shape(v4, lead + (64,), "v4")
        _expect_shape(ks, lead, "ks")
        _expect_shape(vs, lead, "vs")
        real = [i for i in range(3) if lead[i] > 1]   # dimensions whose stride counts
        for t, unit, name in ((k4, 64, "k4"), (v4, 64, "v4"), (vs, 1, "vs")):
            if any(t.stride(i) != unit * ks.stride(i) for i in real) or (
                    unit == 64 and t.stride(3) != 1):
                raise ValueError(f"{name} must have the layout of ks (strides, in vectors)")
        device = k4.device
        for t, dtype, name in ((k4, torch.uint8, "k4"), (ks, torch.float32, "ks"),
                               (v4, torch.uint8, "v4"), (vs, torch.float32, "vs")):
            _kv4_check(t, dtype, name, device)
        self.k4, self.ks, self.v4, self.vs = k4, ks, v4, vs
        self.pages, self.page_size, self.heads = lead
        self.device = device
        strides = [ks.stride(i) if i in real else 0 for i in range(3)]
        self.struct = _CacheStruct(k4.data_ptr(), ks.data_ptr(), v4.data_ptr(), vs.data_ptr(),
                                   *lead, *strides)
        self._ref = ct.addressof(self.struct)


def empty_kv4_cache(pages: int, page_size: int, heads: int, device,
                    token_major: bool = False) -> KV4Cache:
    """A KV4Cache in new storage: [pages, heads, page_size, ...] (a head's tokens of a page
    together) or, token_major, [pages, page_size, heads, ...] (atom_kv_quant's order). Its
    contents are undefined."""
    lead = (pages, page_size, heads) if token_major else (pages, heads, page_size)
    parts = []
    for _ in range(2):
        q4 = torch.empty(lead + (64,), dtype=torch.uint8, device=device)
        scales = torch.empty(lead, dtype=torch.float32, device=device)
        parts += [q4, scales] if token_major else [q4.transpose(1, 2), scales.transpose(1, 2)]
    return KV4Cache(*parts)


class KV4Batch:
    """The sequences of a call on a KV4Cache (see include/atom.h): block_table int32 [batch,
    max_pages] (a row's entries together), kv_lens int32 [batch] (the new tokens included)
    and cu_q int32 [batch + 1], on one device; max_q bounds the new tokens of a sequence
    (default: no bound but the call's rows). The object holds the tensors' addresses: a
    program updates their values in place from step to step."""

    def __init__(self, block_table: torch.Tensor, kv_lens: torch.Tensor, cu_q: torch.Tensor,
                 max_q: Optional[int] = None):
        if kv_lens.dim() != 1:
            raise ValueError(f"kv_lens must have shape (batch,), got {tuple(kv_lens.shape)}")
        batch = kv_lens.shape[0]
        if block_table.dim() != 2 or block_table.shape[0] != batch:
            raise ValueError(f"block_table must have shape ({batch}, max_pages), got "
                             f"{tuple(block_table.shape)}")
        _expect_shape(cu_q, (batch + 1,), "cu_q")
        if max_q is not None and max_q < 0:
            raise ValueError("max_q must not be negative")
        self.device = kv_lens.device
        for t, name in ((block_table, "block_table"), (kv_lens, "kv_lens"), (cu_q, "cu_q")):
            _kv4_check(t, torch.int32, name, self.device)
        width = block_table.shape[1]
        if (block_table.stride(1) != 1 and width > 1) or not kv_lens.is_contiguous() or (
                not cu_q.is_contiguous()):
            raise ValueError("block_table rows, kv_lens and cu_q must be contiguous")
        self.block_table, self.kv_lens, self.cu_q = block_table, kv_lens, cu_q
        self.batch = batch
        self.max_q = 2 ** 31 - 1 if max_q is None else max_q
        stride = block_table.stride(0) if batch > 1 else width
        self.struct = _BatchStruct(block_table.data_ptr(), stride, width, kv_lens.data_ptr(),
                                   cu_q.data_ptr(), batch, self.max_q)
        self._ref = ct.addressof(self.struct)


def _kv4_run(device: torch.device, stream, call):
    """call(stream handle) with `device` current and the call's stream (default: the device's
    current one) the one whose memory new tensors come from."""
    if stream is None and torch._C._cuda_getDevice() == device.index:
        # the same handle as torch.cuda.current_stream()'s, without the 3 us of its object: a
        # third of what a call for a few tokens takes
        return call(torch._C._cuda_getCurrentRawStream(device.index))
    with torch.cuda.device(device):
        if stream is None:
            return call(torch.cuda.current_stream().cuda_stream)
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)


def _kv4_same_device(cache: KV4Cache, batch: KV4Batch) -> torch.device:
    if batch.device != cache.device:
        raise ValueError(f"the batch must be on {cache.device}, got {batch.device}")
    return cache.device


def atom_kv4_append(k: torch.Tensor, v: torch.Tensor, cache: KV4Cache, batch: KV4Batch,
                    stream=None) -> None:
    """Quantizes new keys and values, fp16 [rows, heads, 128] (strided views are taken),
    into their slots of the cache: the last positions of their sequences."""
    device = _kv4_same_device(cache, batch)
    if k.shape[0] != v.shape[0]:
        raise ValueError("k and v must have the same rows")
    kp, vp = _kv4_rows(k, cache.heads, "k", device), _kv4_rows(v, cache.heads, "v", device)
    fn = lib().atom_kv4_append
    _check("atom_kv4_append", _kv4_run(device, stream, lambda s: fn(
        *kp, *vp, k.shape[0], cache._ref, batch._ref, s)))


def atom_kv4_gather(cache: KV4Cache, batch: KV4Batch, rows: int,
                    k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
                    stream=None):
    """Reads the tokens that atom_kv4_append wrote back as fp16 (k, v), each [rows, heads,
    128] with atom_kv_dequant's values. Rows that no sequence has are not written."""
    device = _kv4_same_device(cache, batch)
    shape = (rows, cache.heads, 128)

    def call(s):
        to_k = _kv4_output(k, cache.k4, torch.float16, shape, "k", device)
        to_v = _kv4_output(v, to_k, torch.float16, shape, "v", device)
        _check("atom_kv4_gather", lib().atom_kv4_gather(
            cache._ref, batch._ref, rows, to_k.data_ptr(), to_v.data_ptr(), s))
        return to_k, to_v

    return _kv4_run(device, stream, call)


def atom_kv4_attention_workspace_bytes(rows: int, q_heads: int, heads: int, max_q: int) -> int:
    return int(lib().atom_kv4_attention_workspace_bytes(rows, q_heads, heads, max_q))


@functools.lru_cache(maxsize=64)
def _kv4_workspace_bytes(device_index: int, rows: int, q_heads: int, heads: int,
                         max_q: int) -> int:
    """Of the current device, device_index. 0 says that there is no work, sizes that the call
    refuses, or a failed CUDA call: that one raises, and is not kept."""
    n = atom_kv4_attention_workspace_bytes(rows, q_heads, heads, max_q)
    if n == 0 and min(rows, q_heads, heads, max_q) > 0 and q_heads % heads == 0:
        _check("atom_kv4_attention_workspace_bytes", 5)   # ATOM_ERR_CUDA
    return n


def atom_kv4_attention(q: torch.Tensor, cache: KV4Cache, batch: KV4Batch, causal: bool = True,
                       scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                       lse: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, split: bool = True,
                       stream=None):
    """Attention of new tokens over the INT4 cache (their own keys and values already
    appended): q fp16 [rows, q_heads, 128] (strided views are taken) -> (out fp16 [rows,
    q_heads, 128], lse float32 [rows, q_heads]). `scale` defaults to 1/sqrt(128).

    `workspace` (uint8) is the scratch with which a sequence's cached tokens are shared
    between CTAs; when it is None and `split` is true, one of
    atom_kv4_attention_workspace_bytes() bytes is allocated here."""
    device = _kv4_same_device(cache, batch)
    qp = _kv4_rows(q, None, "q", device)
    rows, q_heads = q.shape[0], q.shape[1]
    if workspace is not None and split:
        _kv4_check(workspace, torch.uint8, "workspace", device)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")

    def call(s):
        o = _kv4_output(out, q, torch.float16, (rows, q_heads, 128), "out", device)
        z = _kv4_output(lse, cache.ks, torch.float32, (rows, q_heads), "lse", device)
        ws, ws_bytes = workspace, 0
        if split:
            if ws is None:
                ws_bytes = _kv4_workspace_bytes(device.index, rows, q_heads, cache.heads,
                                                batch.max_q)
                ws = cache.k4.new_empty(ws_bytes) if ws_bytes else None
            else:
                ws_bytes = ws.numel()
        _check("atom_kv4_attention", lib().atom_kv4_attention(
            *qp, rows, q_heads, cache._ref, batch._ref, 1 if causal else 0,
            128.0 ** -0.5 if scale is None else scale,
            o.data_ptr(), z.data_ptr(), ws.data_ptr() if ws_bytes else None, ws_bytes, s))
        return o, z

    return _kv4_run(device, stream, call)


def atom_kv4_attention_weights(q: torch.Tensor, lse: torch.Tensor, cache: KV4Cache,
                               batch: KV4Batch, sums: torch.Tensor,
                               prev: Optional[torch.Tensor] = None, causal: bool = True,
                               scale: Optional[float] = None, stream=None) -> torch.Tensor:
    """The attention weight that each cached token received from the call's queries, summed
    over a KV head's query heads: float32 [batch, heads, width], written to `sums` (added to
    `prev`, which may be `sums` itself) for the tokens of each sequence. q, causal and scale
    as given to atom_kv4_attention, lse as it returned."""
    device = _kv4_same_device(cache, batch)
    qp = _kv4_rows(q, None, "q", device)
    rows, q_heads = q.shape[0], q.shape[1]
    if sums.dim() != 3:
        raise ValueError("sums must have shape (batch, heads, width)")
    width = sums.shape[2]
    shape = (batch.batch, cache.heads, width)
    sums_ptr = _kv4_contiguous(sums, torch.float32, shape, "sums", device)
    prev_ptr = None
    if prev is not None:
        prev_ptr = _kv4_contiguous(prev, torch.float32, shape, "prev", device)
    lse_ptr = _kv4_contiguous(lse, torch.float32, (rows, q_heads), "lse", device)
    fn = lib().atom_kv4_attention_weights
    _check("atom_kv4_attention_weights", _kv4_run(device, stream, lambda s: fn(
        *qp, rows, q_heads, lse_ptr, cache._ref, batch._ref, 1 if causal else 0,
        128.0 ** -0.5 if scale is None else scale, prev_ptr, sums_ptr, width, s)))
    return sums


def atom_kv4_evict(weights: torch.Tensor, cache: KV4Cache, batch: KV4Batch, budget: int,
                   recent: int, dst: KV4Cache, to_table: torch.Tensor, new_lens: torch.Tensor,
                   kept: Optional[torch.Tensor] = None,
                   new_weights: Optional[torch.Tensor] = None, stream=None):
    """Keeps `budget` tokens of each sequence and KV head: the last `recent` ones and those
    with the largest `weights` (float32 [batch, heads, width]), moved in their order to the
    first positions of `dst` (pages to_table int32 [batch, pages]); `dst` and `to_table` may
    be the cache and its own table. Writes new_lens int32 [batch] (not batch.kv_lens) and
    returns (kept int32 [batch, heads, budget], new_weights float32 [batch, heads,
    new_width]); elements of new_weights behind a sequence's new length are not written."""
    device = _kv4_same_device(cache, batch)
    if dst.device != device:
        raise ValueError(f"dst must be on {device}, got {dst.device}")
    n, heads = batch.batch, cache.heads
    if weights.dim() != 3:
        raise ValueError("weights must have shape (batch, heads, width)")
    width = weights.shape[2]
    weights_ptr = _kv4_contiguous(weights, torch.float32, (n, heads, width), "weights", device)
    if to_table.dim() != 2 or to_table.shape[0] != n:
        raise ValueError(f"to_table must have shape ({n}, pages), got {tuple(to_table.shape)}")
    _kv4_check(to_table, torch.int32, "to_table", device)
    to_pages = to_table.shape[1]
    if to_pages > 1 and to_table.stride(1) != 1:
        raise ValueError("to_table rows must be contiguous")
    lens_ptr = _kv4_contiguous(new_lens, torch.int32, (n,), "new_lens", device)

    def call(s):
        at = _kv4_output(kept, weights, torch.int32, (n, heads, budget), "kept", device)
        new_width = budget if new_weights is None else new_weights.shape[-1]
        w = _kv4_output(new_weights, weights, torch.float32, (n, heads, new_width), "new_weights",
                        device)
        _check("atom_kv4_evict", lib().atom_kv4_evict(
            weights_ptr, width, cache._ref, batch._ref, budget, recent, dst._ref,
            to_table.data_ptr(), to_table.stride(0) if n > 1 else to_pages, to_pages, lens_ptr,
            at.data_ptr(), w.data_ptr(), new_width, s))
        return at, w

    return _kv4_run(device, stream, call)


def atom_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().atom_gemm_workspace_bytes(M, N, K))


def atom_probe_mma_i8(groups: int, stream=None) -> int:
    """Measurement aid: launches the INT8 tensor-core peak loop (see
    include/atom.h) and returns the integer operations it performs."""
    pairs = ct.c_int32(0)
    _check("atom_probe_mma_i8", lib().atom_probe_mma_i8(groups, ct.byref(pairs), _stream(stream)))
    return 2 * 256 * 256 * 128 * groups * pairs.value


def atom_debug_wait_timeout(limit_ns: int, stream=None) -> None:
    """Test aid: runs the library's bounded mbarrier wait on a barrier nothing
    arrives on, with a limit of `limit_ns`; the wait gives up and the device
    status becomes ATOM_ERR_TIMEOUT (see include/atom.h)."""
    _check("atom_debug_wait_timeout", lib().atom_debug_wait_timeout(limit_ns, _stream(stream)))


def atom_device_status(clear: bool = True) -> int:
    """First device-detected error since the last clear (0 = none); synchronises."""
    return int(lib().atom_device_status(1 if clear else 0))


def atom_status_string(status: int) -> str:
    return lib().atom_status_string(status).decode()


def atom_version() -> int:
    return int(lib().atom_version())
