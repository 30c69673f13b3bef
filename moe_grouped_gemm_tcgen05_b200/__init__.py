"""FP8 block-scaled GEMMs (dense, contiguous and masked M-grouped; UE8M0 or fp32
scales), the UE8M0 pack and the calls of a layer of routed experts (routing,
rows, dispatch, combine and their gradients) for B200, as a thin Python binding
over libdgb200.so.

Every function here only checks shapes/dtypes/devices on the host and passes
raw pointers to the C ABI declared in ``include/dgb200.h``; all arithmetic runs
in the library's CUDA kernels. There is no fallback: if the shared library is
missing or cannot run on the current device, calls raise.

Tensors are torch tensors used as device memory; work is queued on torch's
current CUDA stream. No call synchronises or allocates (except the
convenience allocations of ``pack_ue8m0`` / ``empty_*`` / ``moe_*`` when no
output is given), so the calls of the method can be captured in a CUDA Graph (no claim
is made for ``fp8_gemm_nt_noalloc``).
"""

from __future__ import annotations

import ctypes
import os
import threading

import torch

__all__ = [
    "BLOCK", "lib_path", "load", "init", "device_error", "last_device_error", "set_block_n", "block_n_supported",
    "fp8_gemm_nt", "m_grouped_fp8_gemm_nt_contiguous", "m_grouped_fp8_gemm_nt_masked",
    "pack_ue8m0", "pack_ue8m0_validate", "DgError", "set_test_hooks", "set_cta_group", "set_splits",
    "fp8_gemm_nt_noalloc", "m_grouped_bf16_gemm_nt_masked", "fp8_gemm_nt_acc", "quantize_fp8_1x128",
    "fp8_gemm_nn", "fp8_gemm_tn", "fp8_gemm_tt",
    "fp8_gemm_nt_sfb_gran", "m_grouped_fp8_gemm_nt_contiguous_sfb_gran", "m_grouped_fp8_gemm_nt_masked_sfb_gran",
    "m_grouped_fp8_gemm_nt_psum",
    "moe_route", "moe_route_backward", "moe_rows_bound", "moe_rows_contiguous", "moe_rows_masked", "moe_dispatch_fp8",
    "moe_combine", "moe_combine_backward", "quantize_fp8_1x128_sf_f32",
    "fp8_gemm_nt_sf_f32", "m_grouped_fp8_gemm_nt_contiguous_sf_f32", "m_grouped_fp8_gemm_nt_masked_sf_f32",
    "DEVERR_TIMEOUT", "DEVERR_MIXED_EXPERT_BLOCK",
]

BLOCK = 128
DEVERR_TIMEOUT = 1
DEVERR_MIXED_EXPERT_BLOCK = 2

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libdgb200.so"
_lib = None
_lock = threading.Lock()

_STATUS = {
    0: "DG_OK", 1: "DG_ERR_INVALID_ARG", 2: "DG_ERR_ALIGNMENT", 3: "DG_ERR_UNSUPPORTED",
    4: "DG_ERR_NOT_INITIALIZED", 5: "DG_ERR_CUDA", 6: "DG_ERR_SCRATCH_TOO_SMALL",
}


class DgError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {_STATUS.get(status, status)}")


def lib_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


def load():
    """Load libdgb200.so (built in-tree) and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m moe_grouped_gemm_tcgen05_b200.build`")
        L = ctypes.CDLL(path)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        L.dgb200_status_string.restype = ctypes.c_char_p
        L.dgb200_status_string.argtypes = [i32]
        L.dgb200_init.restype = i32
        L.dgb200_init.argtypes = [i32]
        L.dgb200_last_device_error.restype = i32
        L.dgb200_last_device_error.argtypes = [ctypes.POINTER(ctypes.c_int)]
        L.dgb200_device_error.restype = i32
        L.dgb200_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32), i32]
        L.dgb200_set_block_n.restype = i32
        L.dgb200_set_block_n.argtypes = [i32]
        L.dgb200_block_n_supported.restype = i32
        L.dgb200_block_n_supported.argtypes = [i32]
        L.dgb200_set_cta_group.restype = i32
        L.dgb200_set_cta_group.argtypes = [i32]
        L.dgb200_set_splits.restype = i32
        L.dgb200_set_splits.argtypes = [i32]
        L.dgb200_set_test_hooks.restype = i32
        L.dgb200_set_test_hooks.argtypes = [i32, i32]
        L.fp8_gemm_nt.restype = i32
        L.fp8_gemm_nt.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, vp]
        L.m_grouped_bf16_gemm_nt_masked.restype = i32
        L.m_grouped_bf16_gemm_nt_masked.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp]
        L.quantize_fp8_1x128.restype = i32
        L.quantize_fp8_1x128.argtypes = [vp, i32, vp, vp, vp, ctypes.c_int64, i32, vp]
        for name in ("fp8_gemm_nn", "fp8_gemm_tn", "fp8_gemm_tt"):
            getattr(L, name).restype = i32
            getattr(L, name).argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, vp]
        L.fp8_gemm_nt_acc.restype = i32
        L.fp8_gemm_nt_acc.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, vp]
        L.fp8_gemm_nt_noalloc.restype = i32
        L.fp8_gemm_nt_noalloc.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp]
        L.m_grouped_fp8_gemm_nt_contiguous.restype = i32
        L.m_grouped_fp8_gemm_nt_contiguous.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, vp]
        L.m_grouped_fp8_gemm_nt_masked.restype = i32
        L.m_grouped_fp8_gemm_nt_masked.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, vp]
        L.m_grouped_fp8_gemm_nt_psum.restype = i32
        L.m_grouped_fp8_gemm_nt_psum.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, vp]
        L.fp8_gemm_nt_sfb_gran.restype = i32
        L.fp8_gemm_nt_sfb_gran.argtypes = [vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, vp]
        L.m_grouped_fp8_gemm_nt_contiguous_sfb_gran.restype = i32
        L.m_grouped_fp8_gemm_nt_contiguous_sfb_gran.argtypes = [vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, vp]
        L.m_grouped_fp8_gemm_nt_masked_sfb_gran.restype = i32
        L.m_grouped_fp8_gemm_nt_masked_sfb_gran.argtypes = [vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, vp]
        L.pack_ue8m0.restype = i32
        L.pack_ue8m0.argtypes = [vp, vp, i64, i32, vp]
        L.pack_ue8m0_validate.restype = i32
        L.pack_ue8m0_validate.argtypes = [vp, i64, i32, vp, vp]
        for name, args in (
                ("moe_route", [vp, i32, vp, vp, vp] + [i32] * 8 + [ctypes.c_float, vp]),
                ("moe_route_backward", [vp, i32, vp, vp, vp] + [i32] * 5 + [ctypes.c_float, vp]),
                ("moe_rows_contiguous", [vp] * 4 + [i32] * 3 + [i64, vp]),
                ("moe_rows_masked", [vp] * 4 + [i32] * 4 + [vp]),
                ("moe_dispatch_fp8", [vp, i32, vp, vp, vp, i32, i64] + [i32] * 3 + [vp]),
                ("quantize_fp8_1x128_sf_f32", [vp, i32, vp, vp, i64, i32, vp]),
                ("fp8_gemm_nt_sf_f32", [vp] * 4 + [i32, vp, vp] + [i32] * 4 + [vp]),
                ("m_grouped_fp8_gemm_nt_contiguous_sf_f32", [vp] * 6 + [i32] * 4 + [vp]),
                ("m_grouped_fp8_gemm_nt_masked_sf_f32", [vp] * 6 + [i32] * 4 + [vp]),
                ("moe_combine", [vp] * 4 + [i64] + [i32] * 3 + [vp]),
                ("moe_combine_backward", [vp] * 6 + [i64] + [i32] * 3 + [vp])):
            getattr(L, name).restype = i32
            getattr(L, name).argtypes = args
        L.moe_rows_bound.restype = i64
        L.moe_rows_bound.argtypes = [i32, i32, i32]
        _lib = L
        return L


def _check(fn: str, status: int):
    if status != 0:
        raise DgError(fn, status)


# The handle of torch's current stream as a number. (current_stream() builds a
# Stream object around it on every call: ~1.5 us of a call's ~10.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device=None):
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device() if device is None else device)
    return torch.cuda.current_stream().cuda_stream


def _ptr(t: torch.Tensor):
    return t.data_ptr()  # ctypes turns it into the void* that the signatures declare


def _need(t: torch.Tensor, name: str, dtypes, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:  # a torch.Size compares as the tuple it is
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


_FP8 = (torch.float8_e4m3fn, torch.uint8)
_I32 = (torch.int32,)
_BF16 = (torch.bfloat16,)


def init(device=None):
    """Configure the kernels for a CUDA device (default: torch's current one);
    do it before graph capture."""
    if device is None:
        device = torch.cuda.current_device()
    elif isinstance(device, torch.device):
        device = device.index if device.index is not None else torch.cuda.current_device()
    _check("dgb200_init", load().dgb200_init(int(device)))


def last_device_error() -> int:
    """Device status bits (DEVERR_*) of the current device, then reset to 0;
    synchronises the device."""
    v = ctypes.c_int(0)
    _check("dgb200_last_device_error", load().dgb200_last_device_error(ctypes.byref(v)))
    return int(v.value)


def device_error(clear: bool = True) -> int:
    """Device status bits (DEVERR_*); synchronises the device."""
    v = ctypes.c_uint32(0)
    _check("dgb200_device_error", load().dgb200_device_error(ctypes.byref(v), 1 if clear else 0))
    return int(v.value)


def set_block_n(block_n: int):
    """Force the N tile width (0 = heuristic). For tests and tuning."""
    _check("dgb200_set_block_n", load().dgb200_set_block_n(int(block_n)))


def set_cta_group(cta_group: int):
    """Force single CTAs (1) or CTA pairs (2) for the dense GEMM (0 = heuristic)."""
    _check("dgb200_set_cta_group", load().dgb200_set_cta_group(int(cta_group)))


def set_splits(splits: int):
    """Split-K for the dense GEMM: 0 = heuristic, 1 = never, s >= 2 = s ranges of K."""
    _check("dgb200_set_splits", load().dgb200_set_splits(int(splits)))


def set_test_hooks(mode: int = 0, wait_limit_ms: int = 0):
    """Test hooks: mode 1 makes CTA 0 withhold the arrive of its first group of
    scale words so that a bounded wait runs out, mode 2 launches moe_rows_* on
    clusters of at most 8 CTAs (see include/dgb200.h). mode 0 = normal."""
    _check("dgb200_set_test_hooks", load().dgb200_set_test_hooks(int(mode), int(wait_limit_ms)))


def block_n_supported(block_n: int) -> bool:
    return bool(load().dgb200_block_n_supported(int(block_n)))


def _kp(K: int) -> int:
    return (K // BLOCK + 3) // 4


def fp8_gemm_nt(a, sfa, b, sfb, d):
    """d[M, N] (bf16) = (a . sfa) @ (b . sfb)^T for E4M3 a [M, K], b [N, K]."""
    _need(a, "a", _FP8)
    M, K = a.shape
    _need(b, "b", _FP8)
    N = b.shape[0]
    _need(b, "b", _FP8, (N, K))
    _need(sfa, "sfa", _I32, (M, _kp(K)))
    _need(sfb, "sfb", _I32, ((N + BLOCK - 1) // BLOCK, _kp(K)))
    _need(d, "d", _BF16, (M, N))
    _check("fp8_gemm_nt", load().fp8_gemm_nt(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d), M, N, K, _stream()))
    return d


def _fp8_gemm_layout(name, a, sfa, b, sfb, d, a_mk: bool, b_nk: bool):
    _need(a, "a", _FP8)
    _need(b, "b", _FP8)
    if a_mk:
        M, K = a.shape
    else:
        K, M = a.shape
    N = b.shape[0] if b_nk else b.shape[1]
    _need(a, "a", _FP8, (M, K) if a_mk else (K, M))
    _need(b, "b", _FP8, (N, K) if b_nk else (K, N))
    _need(sfa, "sfa", _I32, (M, _kp(K)))
    _need(sfb, "sfb", _I32, ((N + BLOCK - 1) // BLOCK, _kp(K)))
    _need(d, "d", _BF16, (M, N))
    _check(name, getattr(load(), name)(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d), M, N, K, _stream()))
    return d


def fp8_gemm_nn(a, sfa, b, sfb, d):
    """d[M, N] = (a . sfa) @ (b . sfb) for E4M3 a [M, K], b [K, N]."""
    return _fp8_gemm_layout("fp8_gemm_nn", a, sfa, b, sfb, d, True, False)


def fp8_gemm_tn(a, sfa, b, sfb, d):
    """d[M, N] = (a . sfa)^T @ (b . sfb) for E4M3 a [K, M], b [K, N]."""
    return _fp8_gemm_layout("fp8_gemm_tn", a, sfa, b, sfb, d, False, False)


def fp8_gemm_tt(a, sfa, b, sfb, d):
    """d[M, N] = (a . sfa)^T @ (b . sfb)^T for E4M3 a [K, M], b [N, K]."""
    return _fp8_gemm_layout("fp8_gemm_tt", a, sfa, b, sfb, d, False, True)


def fp8_gemm_nt_acc(a, sfa, b, sfb, d, c=None):
    """d[M, N] = c + (a . sfa) @ (b . sfb)^T; d is bf16 or fp32, c (optional) has d's
    dtype and may be d itself (in-place accumulation)."""
    _need(a, "a", _FP8)
    M, K = a.shape
    _need(b, "b", _FP8)
    N = b.shape[0]
    _need(b, "b", _FP8, (N, K))
    _need(sfa, "sfa", _I32, (M, _kp(K)))
    _need(sfb, "sfb", _I32, ((N + BLOCK - 1) // BLOCK, _kp(K)))
    _need(d, "d", (torch.bfloat16, torch.float32), (M, N))
    if c is not None:
        _need(c, "c", (d.dtype,), (M, N))
    _check("fp8_gemm_nt_acc", load().fp8_gemm_nt_acc(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb),
                                                     None if c is None else _ptr(c), _ptr(d), M, N, K,
                                                     1 if d.dtype == torch.float32 else 0, _stream()))
    return d


def fp8_gemm_nt_noalloc(a, sfa, b, sfb, d, splits: int = 0):
    """fp8_gemm_nt that allocates no device memory: split-K scratch comes from
    static arrays of the library (8 MiB of partials, 1024 tiles). splits: 0 =
    model's choice within that scratch, 1 = none, s >= 2 = exactly s. Calls that
    overlap in time on one device race on the scratch (see include/dgb200.h)."""
    _need(a, "a", _FP8)
    M, K = a.shape
    _need(b, "b", _FP8)
    N = b.shape[0]
    _need(b, "b", _FP8, (N, K))
    _need(sfa, "sfa", _I32, (M, _kp(K)))
    _need(sfb, "sfb", _I32, ((N + BLOCK - 1) // BLOCK, _kp(K)))
    _need(d, "d", _BF16, (M, N))
    _check("fp8_gemm_nt_noalloc", load().fp8_gemm_nt_noalloc(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d), M, N, K,
                                                             int(splits), _stream()))
    return d


def m_grouped_fp8_gemm_nt_contiguous(a, sfa, b, sfb, d, m_indices):
    """Contiguous M-grouped GEMM; rows tagged by expert in m_indices (-1 = padding)."""
    _need(a, "a", _FP8)
    M_total, K = a.shape
    _need(b, "b", _FP8)
    G, N = b.shape[0], b.shape[1]
    _need(b, "b", _FP8, (G, N, K))
    _need(sfa, "sfa", _I32, (M_total, _kp(K)))
    _need(sfb, "sfb", _I32, (G, (N + BLOCK - 1) // BLOCK, _kp(K)))
    _need(d, "d", _BF16, (M_total, N))
    _need(m_indices, "m_indices", _I32, (M_total,))
    _check("m_grouped_fp8_gemm_nt_contiguous",
           load().m_grouped_fp8_gemm_nt_contiguous(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d), _ptr(m_indices),
                                                   M_total, N, K, G, _stream()))
    return d


def m_grouped_fp8_gemm_nt_masked(a, sfa, b, sfb, d, masked_m, max_m=None):
    """Masked M-grouped GEMM; group g uses its first masked_m[g] rows (device tensor)."""
    _need(a, "a", _FP8)
    G, mm, K = a.shape
    if max_m is None:
        max_m = mm
    if max_m != mm:
        raise ValueError(f"max_m={max_m} does not match a.shape[1]={mm}")
    _need(b, "b", _FP8)
    N = b.shape[1]
    _need(b, "b", _FP8, (G, N, K))
    _need(sfa, "sfa", _I32, (G, max_m, _kp(K)))
    _need(sfb, "sfb", _I32, (G, (N + BLOCK - 1) // BLOCK, _kp(K)))
    _need(d, "d", _BF16, (G, max_m, N))
    _need(masked_m, "masked_m", _I32, (G,))
    _check("m_grouped_fp8_gemm_nt_masked",
           load().m_grouped_fp8_gemm_nt_masked(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d), _ptr(masked_m),
                                               G, max_m, N, K, _stream()))
    return d


def m_grouped_fp8_gemm_nt_psum(a, sfa, b, sfb, d, psum_m):
    """M-grouped GEMM with groups given by psum_m (device int32 [G]): group g owns
    rows [psum_m[g-1], psum_m[g]) of a [M_total, K]; rows in no group are not written."""
    _need(a, "a", _FP8)
    M_total, K = a.shape
    _need(b, "b", _FP8)
    G, N = b.shape[0], b.shape[1]
    _need(b, "b", _FP8, (G, N, K))
    _need(sfa, "sfa", _I32, (M_total, _kp(K)))
    _need(sfb, "sfb", _I32, (G, (N + BLOCK - 1) // BLOCK, _kp(K)))
    _need(d, "d", _BF16, (M_total, N))
    _need(psum_m, "psum_m", _I32, (G,))
    _check("m_grouped_fp8_gemm_nt_psum",
           load().m_grouped_fp8_gemm_nt_psum(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d), _ptr(psum_m),
                                             M_total, N, K, G, _stream()))
    return d


def _sfb_rows(N: int, sfb_gran_n: int) -> int:
    if sfb_gran_n not in (1, BLOCK):
        raise ValueError(f"sfb_gran_n={sfb_gran_n}: B scale rows cover 1 or {BLOCK} rows of B")
    return N if sfb_gran_n == 1 else (N + BLOCK - 1) // BLOCK


def fp8_gemm_nt_sfb_gran(a, sfa, b, sfb, d, sfb_gran_n: int, c=None):
    """fp8_gemm_nt_acc with the B-scale granularity given: sfb [N, KP] (sfb_gran_n=1,
    one scale row per row of b) or [ceil(N/128), KP] (sfb_gran_n=128)."""
    _need(a, "a", _FP8)
    M, K = a.shape
    _need(b, "b", _FP8)
    N = b.shape[0]
    _need(b, "b", _FP8, (N, K))
    _need(sfa, "sfa", _I32, (M, _kp(K)))
    _need(sfb, "sfb", _I32, (_sfb_rows(N, sfb_gran_n), _kp(K)))
    _need(d, "d", (torch.bfloat16, torch.float32), (M, N))
    if c is not None:
        _need(c, "c", (d.dtype,), (M, N))
    _check("fp8_gemm_nt_sfb_gran",
           load().fp8_gemm_nt_sfb_gran(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), int(sfb_gran_n),
                                       None if c is None else _ptr(c), _ptr(d), M, N, K,
                                       1 if d.dtype == torch.float32 else 0, _stream()))
    return d


def m_grouped_fp8_gemm_nt_contiguous_sfb_gran(a, sfa, b, sfb, d, m_indices, sfb_gran_n: int):
    """m_grouped_fp8_gemm_nt_contiguous with sfb [G, N, KP] (sfb_gran_n=1) or
    [G, ceil(N/128), KP] (sfb_gran_n=128)."""
    _need(a, "a", _FP8)
    M_total, K = a.shape
    _need(b, "b", _FP8)
    G, N = b.shape[0], b.shape[1]
    _need(b, "b", _FP8, (G, N, K))
    _need(sfa, "sfa", _I32, (M_total, _kp(K)))
    _need(sfb, "sfb", _I32, (G, _sfb_rows(N, sfb_gran_n), _kp(K)))
    _need(d, "d", _BF16, (M_total, N))
    _need(m_indices, "m_indices", _I32, (M_total,))
    _check("m_grouped_fp8_gemm_nt_contiguous_sfb_gran",
           load().m_grouped_fp8_gemm_nt_contiguous_sfb_gran(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), int(sfb_gran_n),
                                                            _ptr(d), _ptr(m_indices), M_total, N, K, G, _stream()))
    return d


def m_grouped_fp8_gemm_nt_masked_sfb_gran(a, sfa, b, sfb, d, masked_m, sfb_gran_n: int):
    """m_grouped_fp8_gemm_nt_masked with sfb [G, N, KP] (sfb_gran_n=1) or
    [G, ceil(N/128), KP] (sfb_gran_n=128)."""
    _need(a, "a", _FP8)
    G, max_m, K = a.shape
    _need(b, "b", _FP8)
    N = b.shape[1]
    _need(b, "b", _FP8, (G, N, K))
    _need(sfa, "sfa", _I32, (G, max_m, _kp(K)))
    _need(sfb, "sfb", _I32, (G, _sfb_rows(N, sfb_gran_n), _kp(K)))
    _need(d, "d", _BF16, (G, max_m, N))
    _need(masked_m, "masked_m", _I32, (G,))
    _check("m_grouped_fp8_gemm_nt_masked_sfb_gran",
           load().m_grouped_fp8_gemm_nt_masked_sfb_gran(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), int(sfb_gran_n),
                                                        _ptr(d), _ptr(masked_m), G, max_m, N, K, _stream()))
    return d


_BF16_OPERAND = (torch.bfloat16, torch.int16, torch.uint16)  # bf16 values or their bit patterns


def m_grouped_bf16_gemm_nt_masked(a, b, d, masked_m):
    """Masked M-grouped BF16 GEMM: d[g, :m_g] = a[g, :m_g] @ b[g]^T, m_g = masked_m[g] (device)."""
    _need(a, "a", _BF16_OPERAND)
    G, max_m, K = a.shape
    _need(b, "b", _BF16_OPERAND)
    N = b.shape[1]
    _need(b, "b", _BF16_OPERAND, (G, N, K))
    _need(d, "d", _BF16, (G, max_m, N))
    _need(masked_m, "masked_m", _I32, (G,))
    _check("m_grouped_bf16_gemm_nt_masked",
           load().m_grouped_bf16_gemm_nt_masked(_ptr(a), _ptr(b), _ptr(d), _ptr(masked_m), G, max_m, N, K,
                                                _stream()))
    return d


def pack_ue8m0(sf, out=None):
    """Pack fp32 scales [..., cols] into int32 [..., ceil(cols/4)] (UE8M0, 4 per word)."""
    _need(sf, "sf", (torch.float32,))
    if sf.dim() < 1:
        raise ValueError("sf must have at least one dimension")
    cols = sf.shape[-1]
    rows = sf.numel() // cols if cols else 0
    kp = (cols + 3) // 4
    if out is None:
        out = torch.empty((*sf.shape[:-1], kp), dtype=torch.int32, device=sf.device)
    _need(out, "out", _I32, (*sf.shape[:-1], kp))
    _check("pack_ue8m0", load().pack_ue8m0(_ptr(sf), _ptr(out), rows, cols, _stream()))
    return out


def quantize_fp8_1x128(x, q=None, sf_packed=None, sf_f32=None):
    """x [rows, K] bf16/fp32 -> (q E4M3 as uint8 [rows, K], packed UE8M0 scales
    int32 [rows, ceil(K/512)], fp32 scales [rows, K/128] or None)."""
    _need(x, "x", (torch.bfloat16, torch.float32))
    rows, K = x.shape
    if q is None:
        q = torch.empty((rows, K), dtype=torch.uint8, device=x.device)
    if sf_packed is None:
        sf_packed = torch.empty((rows, _kp(K)), dtype=torch.int32, device=x.device)
    _need(q, "q", _FP8, (rows, K))
    _need(sf_packed, "sf_packed", _I32, (rows, _kp(K)))
    if sf_f32 is not None:
        _need(sf_f32, "sf_f32", (torch.float32,), (rows, K // BLOCK))
    _check("quantize_fp8_1x128",
           load().quantize_fp8_1x128(_ptr(x), 1 if x.dtype == torch.float32 else 0, _ptr(q), _ptr(sf_packed),
                                     None if sf_f32 is None else _ptr(sf_f32), rows, K, _stream()))
    return q, sf_packed, sf_f32


def pack_ue8m0_validate(sf, bad_count):
    """Write to bad_count (device int32 [1]) the number of scales with sign set or mantissa != 0."""
    _need(sf, "sf", (torch.float32,))
    _need(bad_count, "bad_count", _I32, (1,))
    cols = sf.shape[-1]
    rows = sf.numel() // cols if cols else 0
    _check("pack_ue8m0_validate", load().pack_ue8m0_validate(_ptr(sf), rows, cols, _ptr(bad_count), _stream()))
    return bad_count


# ------------------------------------------------- around the experts' products

_F32 = (torch.float32,)
_LOGITS = (torch.float32, torch.bfloat16)
_SCORES = {"softmax": 0, "sigmoid": 1}


def _new(shape, dtype, device):
    """torch.empty of a matrix or vector, a third quicker (a decode step's calls are bound by such things)."""
    return torch.empty_strided(shape, (shape[1], 1) if len(shape) == 2 else (1,), dtype=dtype, device=device)


def _here(*tensors):
    """The handle of the current device's current stream; all tensors live on that device."""
    device = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"a tensor is on {t.device}, but the current device is cuda:{device}")
    return _stream(device)


def _fits(fn, *sizes):
    """Sizes that a C int holds: ctypes would cut larger ones down to their lowest 32 bits.
    (Callers ask only where a size has a bit above the lowest 31: 0.4 us a call otherwise.)"""
    if max(sizes) > 0x7FFFFFFF or min(sizes) < -0x80000000:
        raise DgError(fn, 3)


def _score(score):
    if score not in _SCORES:
        raise ValueError(f"score={score!r}: one of {tuple(_SCORES)}")
    return _SCORES[score]


def _opt(t):
    return None if t is None else _ptr(t)


def moe_route(logits, k, *, bias=None, score="softmax", n_groups=1, top_groups=1, group_top=2, renormalize=True,
              scale=1.0, ids=None, weights=None):
    """Choose k of E experts for each token: logits [T, E] bf16/fp32 -> (ids int32 [T, k]
    by falling score + bias, weights fp32 [T, k] = scale * score, divided by their sum
    when renormalize). The choice stays within the top_groups best of n_groups equal
    groups of experts, ranked by their group_top (1 or 2) best keys."""
    _need(logits, "logits", _LOGITS)
    T, E = logits.shape
    k, n_groups, top_groups, group_top = int(k), int(n_groups), int(top_groups), int(group_top)
    if (T | E | k | n_groups | top_groups | group_top) >> 31:
        _fits("moe_route", T, E, k, n_groups, top_groups, group_top)
    if bias is not None:
        _need(bias, "bias", _F32, (E,))
    if ids is None:
        ids = _new((T, max(k, 0)), torch.int32, logits.device)
    else:
        _need(ids, "ids", _I32, (T, k))
    if weights is None:
        weights = _new((T, max(k, 0)), torch.float32, logits.device)
    else:
        _need(weights, "weights", _F32, (T, k))
    stream = _here(logits, bias, ids, weights)
    _check("moe_route",
           load().moe_route(_ptr(logits), int(logits.dtype == torch.float32), _opt(bias), _ptr(ids), _ptr(weights), T, E,
                            k, _score(score), n_groups, top_groups, group_top, int(bool(renormalize)),
                            float(scale), stream))
    return ids, weights


def moe_route_backward(logits, ids, d_weights, *, score="softmax", renormalize=True, scale=1.0, d_logits=None):
    """Gradient of moe_route's weights: d_weights fp32 [T, k] -> d_logits [T, E] in the
    logits' type, for the ids that moe_route chose."""
    _need(logits, "logits", _LOGITS)
    T, E = logits.shape
    _need(ids, "ids", _I32)
    if ids.dim() != 2 or ids.shape[0] != T:
        raise ValueError(f"ids has shape {tuple(ids.shape)}, expected ({T}, k)")
    k = ids.shape[1]
    if (T | E | k) >> 31:
        _fits("moe_route_backward", T, E, k)
    _need(d_weights, "d_weights", _F32, (T, k))
    if d_logits is None:
        d_logits = torch.empty_like(logits)
    else:
        _need(d_logits, "d_logits", (logits.dtype,), (T, E))
    stream = _here(logits, ids, d_weights, d_logits)
    _check("moe_route_backward",
           load().moe_route_backward(_ptr(logits), int(logits.dtype == torch.float32), _ptr(ids), _ptr(d_weights),
                                     _ptr(d_logits), T, E, k, _score(score), int(bool(renormalize)), float(scale),
                                     stream))
    return d_logits


def moe_rows_bound(T: int, k: int, G: int) -> int:
    """Rows that T*k choices of G experts can take in whole 128-row blocks, however they fall."""
    T, k, G = int(T), int(k), int(G)
    if (T | k | G) >> 31:
        _fits("moe_rows_bound", T, k, G)
    return load().moe_rows_bound(T, k, G)


def _rows_args(fn, ids, G, max_m, row_of, counts):
    _need(ids, "ids", _I32)
    if ids.dim() != 2:
        raise ValueError(f"ids has shape {tuple(ids.shape)}, expected (T, k)")
    T, k = ids.shape
    if (T | k | G | max_m) >> 31:
        _fits(fn, T, k, G, max_m)
    if row_of is None:
        row_of = _new(ids.shape, torch.int32, ids.device)
    else:
        _need(row_of, "row_of", _I32, ids.shape)
    if counts is None:
        counts = _new((max(G, 0),), torch.int32, ids.device)
    else:
        _need(counts, "counts", _I32, (G,))
    return row_of, counts


def moe_rows_contiguous(ids, G, *, row_of=None, m_indices=None, counts=None):
    """Rows of the contiguous layout for the choices ids int32 [T, k] of G experts ->
    (row_of int32 [T, k], m_indices int32 [m_rows], counts int32 [G]); m_rows is
    moe_rows_bound(T, k, G) unless m_indices is given."""
    G = int(G)
    row_of, counts = _rows_args("moe_rows_contiguous", ids, G, 0, row_of, counts)
    T, k = ids.shape
    if m_indices is None:
        m_indices = _new((moe_rows_bound(T, k, G),), torch.int32, ids.device)
    else:
        _need(m_indices, "m_indices", _I32, (m_indices.numel(),))
    stream = _here(ids, row_of, m_indices, counts)
    _check("moe_rows_contiguous",
           load().moe_rows_contiguous(_ptr(ids), _ptr(row_of), _ptr(m_indices), _ptr(counts), T, k, G,
                                      m_indices.numel(), stream))
    return row_of, m_indices, counts


def moe_rows_masked(ids, G, max_m, *, row_of=None, masked_m=None, counts=None):
    """Rows of the masked layout [G, max_m] for the choices ids int32 [T, k] ->
    (row_of int32 [T, k], -1 past max_m; masked_m int32 [G]; counts int32 [G])."""
    G, max_m = int(G), int(max_m)
    row_of, counts = _rows_args("moe_rows_masked", ids, G, max_m, row_of, counts)
    T, k = ids.shape
    if masked_m is None:
        masked_m = _new((max(G, 0),), torch.int32, ids.device)
    else:
        _need(masked_m, "masked_m", _I32, (G,))
    stream = _here(ids, row_of, masked_m, counts)
    _check("moe_rows_masked",
           load().moe_rows_masked(_ptr(ids), _ptr(row_of), _ptr(masked_m), _ptr(counts), T, k, G, max_m, stream))
    return row_of, masked_m, counts


def _row_count(t, H, name):
    """Rows of [rows, H] or of the masked layout [G, max_m, H]."""
    if t.dim() not in (2, 3) or t.shape[-1] != H:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected (rows, {H}) or (G, max_m, {H})")
    return t.shape[0] if t.dim() == 2 else t.shape[0] * t.shape[1]


def moe_dispatch_fp8(x, row_of, q, sf):
    """Write token t of x [T, H] bf16/fp32, cast to E4M3, to the rows row_of[t] of q
    ([rows, H] or [G, max_m, H]) and its scales to sf: int32 [..., ceil(H/512)] packed
    UE8M0, or fp32 [..., H/128]. Other rows are left as they were."""
    _need(x, "x", _LOGITS)
    T, H = x.shape
    _need(row_of, "row_of", _I32)
    if row_of.dim() != 2 or row_of.shape[0] != T:
        raise ValueError(f"row_of has shape {tuple(row_of.shape)}, expected ({T}, k)")
    if (T | H | row_of.shape[1]) >> 31:
        _fits("moe_dispatch_fp8", T, H, row_of.shape[1])
    _need(q, "q", _FP8)
    rows = _row_count(q, H, "q")
    _need(sf, "sf", (torch.int32, torch.float32))
    sf_f32 = sf.dtype == torch.float32
    _need(sf, "sf", (sf.dtype,), (*q.shape[:-1], H // BLOCK if sf_f32 else _kp(H)))
    stream = _here(x, row_of, q, sf)
    _check("moe_dispatch_fp8",
           load().moe_dispatch_fp8(_ptr(x), int(x.dtype == torch.float32), _ptr(row_of), _ptr(q), _ptr(sf), int(sf_f32),
                                   rows, T, row_of.shape[1], H, stream))
    return q, sf


def quantize_fp8_1x128_sf_f32(x, q=None, sf=None):
    """x [rows, K] bf16/fp32 -> (q E4M3 as uint8 [rows, K], sf fp32 [rows, K/128] = amax / 448)."""
    _need(x, "x", _LOGITS)
    rows, K = x.shape
    if K >> 31:
        _fits("quantize_fp8_1x128_sf_f32", K)
    if q is None:
        q = _new((rows, K), torch.uint8, x.device)
    if sf is None:
        sf = _new((rows, K // BLOCK), torch.float32, x.device)
    _need(q, "q", _FP8, (rows, K))
    _need(sf, "sf", _F32, (rows, K // BLOCK))
    stream = _here(x, q, sf)
    _check("quantize_fp8_1x128_sf_f32",
           load().quantize_fp8_1x128_sf_f32(_ptr(x), int(x.dtype == torch.float32), _ptr(q), _ptr(sf), rows, K,
                                            stream))
    return q, sf


def _combine_args(fn, y, row_of, weights):
    _need(y, "y", _BF16)
    if y.dim() not in (2, 3):
        raise ValueError(f"y has shape {tuple(y.shape)}, expected (rows, H) or (G, max_m, H)")
    H = y.shape[-1]
    _need(row_of, "row_of", _I32)
    if row_of.dim() != 2:
        raise ValueError(f"row_of has shape {tuple(row_of.shape)}, expected (T, k)")
    T, k = row_of.shape
    if (T | k | H) >> 31:
        _fits(fn, T, k, H)
    if weights is not None:
        _need(weights, "weights", _F32, row_of.shape)
    return _row_count(y, H, "y"), T, k, H


def moe_combine(y, row_of, weights=None, out=None):
    """out [T, H] bf16 = sum over j of weights[t, j] * y[row_of[t, j]] for y [rows, H] or
    [G, max_m, H] bf16; slots with row -1 add nothing; weights None means ones."""
    rows, T, k, H = _combine_args("moe_combine", y, row_of, weights)
    if out is None:
        out = _new((T, H), torch.bfloat16, y.device)
    else:
        _need(out, "out", _BF16, (T, H))
    stream = _here(y, row_of, weights, out)
    _check("moe_combine", load().moe_combine(_ptr(y), _ptr(row_of), _opt(weights), _ptr(out), rows, T, k, H, stream))
    return out


def moe_combine_backward(y, row_of, weights, d_out, d_y, d_weights=None):
    """Gradients of moe_combine: d_y[row_of[t, j]] = weights[t, j] * d_out[t] (other rows are
    left as they were) and d_weights[t, j] = <y[row_of[t, j]], d_out[t]> fp32."""
    rows, T, k, H = _combine_args("moe_combine_backward", y, row_of, weights)
    _need(d_out, "d_out", _BF16, (T, H))
    _need(d_y, "d_y", _BF16, y.shape)
    if d_weights is None:
        d_weights = _new((T, k), torch.float32, y.device)
    else:
        _need(d_weights, "d_weights", _F32, (T, k))
    stream = _here(y, row_of, weights, d_out, d_y, d_weights)
    _check("moe_combine_backward",
           load().moe_combine_backward(_ptr(y), _ptr(row_of), _opt(weights), _ptr(d_out), _ptr(d_y), _ptr(d_weights),
                                       rows, T, k, H, stream))
    return d_y, d_weights


# ------------------------------------------------- products with fp32 block scales

def fp8_gemm_nt_sf_f32(a, sfa, b, sfb, d, c=None, sfb_gran_n: int = BLOCK):
    """d[M, N] = c + (a . sfa) @ (b . sfb)^T with fp32 scales of any value: sfa [M, K/128];
    sfb [ceil(N/128), K/128] (sfb_gran_n=128) or [N, K/128] (sfb_gran_n=1). d is bf16 or
    fp32; c (optional) has d's dtype and may be d itself (in-place accumulation)."""
    _need(a, "a", _FP8)
    M, K = a.shape
    _need(b, "b", _FP8)
    N = b.shape[0]
    _need(b, "b", _FP8, (N, K))
    if (M | N | K) >> 31:
        _fits("fp8_gemm_nt_sf_f32", M, N, K)
    _need(sfa, "sfa", _F32, (M, K // BLOCK))
    _need(sfb, "sfb", _F32, (_sfb_rows(N, sfb_gran_n), K // BLOCK))
    _need(d, "d", (torch.bfloat16, torch.float32), (M, N))
    if c is not None:
        _need(c, "c", (d.dtype,), (M, N))
    stream = _here(a, sfa, b, sfb, d, c)
    _check("fp8_gemm_nt_sf_f32",
           load().fp8_gemm_nt_sf_f32(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), int(sfb_gran_n), _opt(c), _ptr(d), M, N, K,
                                     int(d.dtype == torch.float32), stream))
    return d


def m_grouped_fp8_gemm_nt_contiguous_sf_f32(a, sfa, b, sfb, d, m_indices):
    """m_grouped_fp8_gemm_nt_contiguous with fp32 scales: sfa [M_total, K/128],
    sfb [G, ceil(N/128), K/128]."""
    _need(a, "a", _FP8)
    M_total, K = a.shape
    _need(b, "b", _FP8)
    G, N = b.shape[0], b.shape[1]
    _need(b, "b", _FP8, (G, N, K))
    if (M_total | N | K | G) >> 31:
        _fits("m_grouped_fp8_gemm_nt_contiguous_sf_f32", M_total, N, K, G)
    _need(sfa, "sfa", _F32, (M_total, K // BLOCK))
    _need(sfb, "sfb", _F32, (G, _sfb_rows(N, BLOCK), K // BLOCK))
    _need(d, "d", _BF16, (M_total, N))
    _need(m_indices, "m_indices", _I32, (M_total,))
    stream = _here(a, sfa, b, sfb, d, m_indices)
    _check("m_grouped_fp8_gemm_nt_contiguous_sf_f32",
           load().m_grouped_fp8_gemm_nt_contiguous_sf_f32(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d),
                                                          _ptr(m_indices), M_total, N, K, G, stream))
    return d


def m_grouped_fp8_gemm_nt_masked_sf_f32(a, sfa, b, sfb, d, masked_m):
    """m_grouped_fp8_gemm_nt_masked with fp32 scales: sfa [G, max_m, K/128],
    sfb [G, ceil(N/128), K/128]."""
    _need(a, "a", _FP8)
    G, max_m, K = a.shape
    _need(b, "b", _FP8)
    N = b.shape[1]
    _need(b, "b", _FP8, (G, N, K))
    if (G | max_m | N | K) >> 31:
        _fits("m_grouped_fp8_gemm_nt_masked_sf_f32", G, max_m, N, K)
    _need(sfa, "sfa", _F32, (G, max_m, K // BLOCK))
    _need(sfb, "sfb", _F32, (G, _sfb_rows(N, BLOCK), K // BLOCK))
    _need(d, "d", _BF16, (G, max_m, N))
    _need(masked_m, "masked_m", _I32, (G,))
    stream = _here(a, sfa, b, sfb, d, masked_m)
    _check("m_grouped_fp8_gemm_nt_masked_sf_f32",
           load().m_grouped_fp8_gemm_nt_masked_sf_f32(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d), _ptr(masked_m),
                                                      G, max_m, N, K, stream))
    return d
