"""Python binding of libhq.so: GPTQ int4 weight quantisation, the Bf16TrilDiagF32 codec, e4m3
layers with block scales and the expert layout of tokens, on NVIDIA B200 (sm_100a).

Argument marshalling only: every function checks tensor dtypes, shapes and devices, turns
them into raw pointers and sizes, and calls the C entry point of the same name (declared in
include/hq.h and include/hq_debug.h).  Every step of the computation runs in the library's
CUDA kernels.  Importing this package fails loudly when libhq.so has not been built
(``python post_weight_quantization_tcgen05_b200/build.py``).
"""

from __future__ import annotations

import ctypes
import os

import torch

# HQ_LIBRARY=libhq_bounds.so selects the bounds-checking build of the same library (hq_debug.h);
# no other name is accepted.
_LIB_NAME = os.environ.get("HQ_LIBRARY", "libhq.so")
if _LIB_NAME not in ("libhq.so", "libhq_bounds.so"):
    raise ImportError(f"HQ_LIBRARY must be libhq.so or libhq_bounds.so, not {_LIB_NAME!r}")
_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), _LIB_NAME)

HQ_OK = 0
HQ_ERR_INVALID = 1
HQ_ERR_UNSUPPORTED = 2
HQ_ERR_NOT_PD = 3
HQ_ERR_TIMEOUT = 4
HQ_ERR_CUDA = 5
HQ_ERR_WORKSPACE = 6
HQ_F32 = 0
HQ_BF16 = 1
# groups N * (K / group) that hq_rtn_quantize_noalloc's fixed scratch holds (hq.h)
HQ_RTN_NOALLOC_MAX_GROUPS = 1048576

# experts that one call handles (hq.h)
HQ_MAX_EXPERTS = 1024

_DTYPE = {torch.float32: HQ_F32, torch.bfloat16: HQ_BF16}


class HQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_NAME} not found at {_LIB_PATH}; build it with "
                      "`python post_weight_quantization_tcgen05_b200/build.py`")

lib = ctypes.CDLL(_LIB_PATH)

_vp, _i64, _int, _f, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_dbl = ctypes.c_double

_SIGS = {
    "hq_status_string": (ctypes.c_char_p, [_int]),
    "hq_abi_version": (_int, []),
    "hq_hessian_accumulate": (_int, [_vp, _vp, _int, _i64, _i64, _vp, _vp]),
    "hq_imatrix": (_int, [_vp, _i64, _i64, _vp, _vp]),
    "hq_gptq_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "hq_gptq_quantize": (_int, [_vp, _int, _i64, _i64, _vp, _i64, _f, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "hq_rtn_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "hq_rtn_quantize": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "hq_rtn_quantize_noalloc": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp]),
    "hq_qerr_terms": (_int, [_vp, _vp, _vp]),
    "hq_qerr_from_terms": (_int, [_vp, _vp, _vp]),
    "hq_gptq_factor_bytes": (_sz, [_i64]),
    "hq_gptq_factor_workspace_bytes": (_sz, [_i64]),
    "hq_gptq_sweep_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "hq_gptq_factorize": (_int, [_vp, _i64, _f, _vp, _sz, _vp, _sz, _vp]),
    "hq_gptq_sweep": (_int, [_vp, _int, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "hq_tril32_count": (_sz, [_i64]),
    "hq_hessian_pack_lower": (_int, [_vp, _i64, _vp, _vp]),
    "hq_hessian_unpack_lower": (_int, [_vp, _i64, _vp, _vp]),
    "hq_hadamard_rotate_weights": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp]),
    "hq_hadamard_rotate_hessian": (_int, [_vp, _i64, _i64, _vp, _vp, _vp]),
    "hq_psd_workspace_bytes": (_sz, [_i64]),
    "hq_hessian_project_psd": (_int, [_vp, _i64, _int, _vp, _sz, _vp]),
    "hq_bf16tril_bytes": (_sz, [_i64]),
    "hq_hessian_pack_bf16tril": (_int, [_vp, _i64, _vp, _vp]),
    "hq_hessian_unpack_bf16tril": (_int, [_vp, _i64, _vp, _vp]),
    "hq_fp8_pitch": (_i64, [_i64]),
    "hq_fp8_quantize_rows": (_int, [_vp, _int, _i64, _i64, _vp, _vp, _vp]),
    "hq_fp8_quantize_blocks": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp]),
    "hq_fp8_gemm": (_int, [_vp, _vp, _i64, _vp, _vp, _i64, _i64, _vp, _int, _vp, _vp]),
    "hq_fp8_linear_workspace_bytes": (_sz, [_i64, _i64]),
    "hq_fp8_linear": (_int, [_vp, _int, _i64, _vp, _vp, _i64, _i64, _vp, _int, _vp, _sz, _vp, _vp]),
    "hq_fp8_expert_gemm": (_int, [_vp, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _int, _vp, _vp]),
    "hq_debug_fp8_gemm_impl": (_int, [_vp, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _int, _vp, _int, _vp]),
    "hq_debug_fp8_gemm_timeout": (_int, [_vp, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _int, _vp, _int, _i64, _int,
                                         _vp]),
    "hq_expert_sort_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "hq_expert_sort": (_int, [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp]),
    "hq_expert_dispatch": (_int, [_vp, _int, _i64, _i64, _vp, _i64, _vp, _vp]),
    "hq_expert_dispatch_fp8": (_int, [_vp, _int, _i64, _i64, _vp, _i64, _vp, _vp, _vp]),
    "hq_expert_combine": (_int, [_vp, _int, _i64, _i64, _vp, _i64, _vp, _vp, _vp]),
    "hq_expert_combine_backward": (_int, [_vp, _vp, _int, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp]),
    "hq_debug_factor": (_int, [_vp, _i64, _f, _vp, _vp, _sz, _vp]),
    "hq_debug_gptq_quantize_impl": (_int, [_vp, _int, _i64, _i64, _vp, _i64, _f, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                           _int, _vp]),
    "hq_debug_hessian_accumulate_impl": (_int, [_vp, _vp, _int, _i64, _i64, _vp, _int, _vp]),
    "hq_debug_hessian_accumulate_timeout": (_int, [_vp, _vp, _i64, _i64, _vp, _i64, _int, _vp]),
    "hq_debug_launch_count": (ctypes.c_uint64, []),
    "hq_debug_bounds_status": (_int, [_vp, _vp]),
    "hq_debug_bounds_selftest": (_int, [_vp]),
    "hq_debug_rcp_f64": (_int, [_vp, _vp, _i64, _vp]),
    "hq_debug_upd_gemm": (_int, [_vp, _i64, _int, _int, _int, _vp, _vp, _i64, _vp, _vp, _i64, _vp]),
    "hq_debug_fp64_mma_rate": (ctypes.c_double, [_vp, _i64, _vp]),
    "hq_debug_timing_start": (_int, [_int]),
    "hq_debug_timing_serialize": (_int, [_int]),
    "hq_debug_timing_stop": (_int, []),
    "hq_debug_timing_read": (_int, [_int, _vp, _vp, _vp]),
    "hq_debug_f64_gemm": (_int, [_vp, _i64, _int, _int, _int, _vp, _i64, _vp, _i64, _dbl, _dbl, _int, _int, _vp,
                                 _i64, _vp]),
    "hq_debug_i8x_scratch_bytes": (_sz, [_int, _int, _int]),
    "hq_debug_i8x_gemm": (_int, [_vp, _i64, _int, _int, _int, _vp, _i64, _vp, _i64, _dbl, _dbl, _int, _int, _vp,
                                 _sz, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def status_string(status: int) -> str:
    return lib.hq_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != HQ_OK:
        raise HQError(status, where)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        # the current stream's handle without building a Stream object (3 us less a call)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dtype(t) -> int:
    if t.dtype not in _DTYPE:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return _DTYPE[t.dtype]


# --------------------------------------------------------------------------- entry points

def hq_abi_version() -> int:
    return lib.hq_abi_version()


def hq_debug_launch_count() -> int:
    return int(lib.hq_debug_launch_count())


def hq_debug_bounds_status():
    """(enabled, violation): whether this is the bounds-checking build, and the first recorded
    failing index check (0 if none; cleared by the call)."""
    en, v = ctypes.c_int(), ctypes.c_int()
    _check(lib.hq_debug_bounds_status(ctypes.byref(en), ctypes.byref(v)), "hq_debug_bounds_status")
    return bool(en.value), int(v.value)


def hq_debug_bounds_selftest(stream=None) -> None:
    """Launch one index check that fails by construction (bounds-checking build only)."""
    _check(lib.hq_debug_bounds_selftest(_stream(stream)), "hq_debug_bounds_selftest")


def bounds_file_tag(name: str) -> int:
    """The tag the bounds-checking build records for source file `name` (bits 16-30)."""
    h = 0
    for c in name.encode():
        h = (h * 31 + c) & 0x7FFF
    return h | 1


def hq_hessian_accumulate(H, X, dev_status=None, stream=None) -> None:
    """H (fp32 [K, K]) += X^T X on the lower triangle; X [T, K] bf16 or fp32."""
    T, K = X.shape
    if H.dtype != torch.float32 or tuple(H.shape) != (K, K):
        raise ValueError("H must be fp32 [K, K]")
    _check(lib.hq_hessian_accumulate(_ptr(H), _ptr(X), _dtype(X), T, K, _ptr(dev_status), _stream(stream)),
           "hq_hessian_accumulate")


def hq_debug_hessian_accumulate_impl(H, X, impl: int, dev_status=None, stream=None) -> None:
    T, K = X.shape
    _check(lib.hq_debug_hessian_accumulate_impl(_ptr(H), _ptr(X), _dtype(X), T, K, _ptr(dev_status), int(impl),
                                                _stream(stream)), "hq_debug_hessian_accumulate_impl")


def hq_debug_hessian_accumulate_timeout(H, X, dev_status, wait_limit_cycles: int, withhold_stage: int = -1,
                                        stream=None) -> None:
    """The tensor-core SYRK with a runtime wait limit and, for the test of its timeout path, one
    operand stage the MMA issuer never releases (hq_debug.h)."""
    if X.dtype != torch.bfloat16:
        raise ValueError("the tensor-core SYRK takes bf16 X")
    T, K = X.shape
    st = lib.hq_debug_hessian_accumulate_timeout(_ptr(H), _ptr(X), T, K, _ptr(dev_status), int(wait_limit_cycles),
                                                 int(withhold_stage), _stream(stream))
    _check(st, "hq_debug_hessian_accumulate_timeout")


def hq_imatrix(H, tokens: int, imp, stream=None) -> None:
    K = H.shape[0]
    _check(lib.hq_imatrix(_ptr(H), K, int(tokens), _ptr(imp), _stream(stream)), "hq_imatrix")


def hq_gptq_workspace_bytes(N: int, K: int, group: int) -> int:
    return int(lib.hq_gptq_workspace_bytes(N, K, group))


def hq_rtn_workspace_bytes(N: int, K: int, group: int) -> int:
    return int(lib.hq_rtn_workspace_bytes(N, K, group))


def hq_gptq_quantize(W, H, group: int, damp: float, codes, scales, workspace, imp=None, want_qerr: bool = True,
                     qerr_dev=None, stream=None):
    """GPTQ int4 of W [N, K] against the undamped fp32 H; returns qerr (host) if requested."""
    N, K = W.shape
    q = ctypes.c_double(float("nan"))
    st = lib.hq_gptq_quantize(_ptr(W), _dtype(W), N, K, _ptr(H), int(group), float(damp), _ptr(imp), _ptr(codes),
                              _ptr(scales), ctypes.byref(q) if want_qerr else None, _ptr(qerr_dev), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "hq_gptq_quantize")
    return q.value if want_qerr else None


def hq_gptq_factor_bytes(K: int) -> int:
    return int(lib.hq_gptq_factor_bytes(K))


def hq_gptq_factor_workspace_bytes(K: int) -> int:
    return int(lib.hq_gptq_factor_workspace_bytes(K))


def hq_gptq_sweep_workspace_bytes(N: int, K: int, group: int) -> int:
    return int(lib.hq_gptq_sweep_workspace_bytes(N, K, group))


def hq_gptq_factorize(H, damp: float, factor, workspace, stream=None) -> None:
    """Damping and factorisation of the undamped fp32 H [K, K] into the factor buffer (uint8)."""
    K = H.shape[0]
    st = lib.hq_gptq_factorize(_ptr(H), K, float(damp), _ptr(factor), factor.numel() * factor.element_size(),
                               _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "hq_gptq_factorize")


def hq_gptq_sweep(W, factor, group: int, codes, scales, workspace, imp=None, want_qerr: bool = True, qerr_dev=None,
                  stream=None):
    """The GPTQ sweep of W [N, K] against a factor buffer; returns qerr (host) if requested."""
    N, K = W.shape
    q = ctypes.c_double(float("nan"))
    st = lib.hq_gptq_sweep(_ptr(W), _dtype(W), N, K, _ptr(factor), int(group), _ptr(imp), _ptr(codes), _ptr(scales),
                           ctypes.byref(q) if want_qerr else None, _ptr(qerr_dev), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "hq_gptq_sweep")
    return q.value if want_qerr else None


def hq_qerr_from_terms(terms_dev, qerr_dev, stream=None) -> None:
    _check(lib.hq_qerr_from_terms(_ptr(terms_dev), _ptr(qerr_dev), _stream(stream)), "hq_qerr_from_terms")


def hq_tril32_count(K: int) -> int:
    return int(lib.hq_tril32_count(K))


def _need_f32(*ts) -> None:
    for t in ts:
        if t.dtype != torch.float32:
            raise ValueError("expected an fp32 tensor")


def hq_hessian_pack_lower(H, packed, stream=None) -> None:
    _need_f32(H, packed)
    K = H.shape[0]
    _check(lib.hq_hessian_pack_lower(_ptr(H), K, _ptr(packed), _stream(stream)), "hq_hessian_pack_lower")


def hq_hessian_unpack_lower(packed, K: int, H, stream=None) -> None:
    _need_f32(H, packed)
    _check(lib.hq_hessian_unpack_lower(_ptr(packed), K, _ptr(H), _stream(stream)), "hq_hessian_unpack_lower")


def hq_debug_gptq_quantize_impl(W, H, group: int, damp: float, codes, scales, workspace, update_impl: int, imp=None,
                                want_qerr: bool = True, qerr_dev=None, stream=None):
    N, K = W.shape
    q = ctypes.c_double(float("nan"))
    st = lib.hq_debug_gptq_quantize_impl(_ptr(W), _dtype(W), N, K, _ptr(H), int(group), float(damp), _ptr(imp),
                                         _ptr(codes), _ptr(scales), ctypes.byref(q) if want_qerr else None,
                                         _ptr(qerr_dev), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                         int(update_impl), _stream(stream))
    _check(st, "hq_debug_gptq_quantize_impl")
    return q.value if want_qerr else None


def hq_rtn_quantize(W, group: int, codes, scales, workspace, imp=None, want_qerr: bool = True, qerr_dev=None,
                    stream=None):
    N, K = W.shape
    q = ctypes.c_double(float("nan"))
    st = lib.hq_rtn_quantize(_ptr(W), _dtype(W), N, K, int(group), _ptr(imp), _ptr(codes), _ptr(scales),
                             ctypes.byref(q) if want_qerr else None, _ptr(qerr_dev), _ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "hq_rtn_quantize")
    return q.value if want_qerr else None


def hq_rtn_quantize_noalloc(W, group: int, codes, scales, imp=None, want_qerr: bool = True, qerr_dev=None,
                            stream=None):
    """hq_rtn_quantize with the library's own fixed scratch instead of a workspace."""
    N, K = W.shape
    q = ctypes.c_double(float("nan"))
    st = lib.hq_rtn_quantize_noalloc(_ptr(W), _dtype(W), N, K, int(group), _ptr(imp), _ptr(codes), _ptr(scales),
                                     ctypes.byref(q) if want_qerr else None, _ptr(qerr_dev), _stream(stream))
    _check(st, "hq_rtn_quantize_noalloc")
    return q.value if want_qerr else None


def hq_psd_workspace_bytes(K: int) -> int:
    return int(lib.hq_psd_workspace_bytes(int(K)))


def hq_hessian_project_psd(H, workspace=None, steps: int = 40, stream=None) -> None:
    """H (fp32 [K, K], symmetric, device) <- its projection onto the PSD cone, in place."""
    K = H.shape[0]
    if workspace is None:
        workspace = alloc_workspace(hq_psd_workspace_bytes(K), H.device)
    _check(lib.hq_hessian_project_psd(_ptr(H), K, int(steps), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _stream(stream)),
           "hq_hessian_project_psd")


def hq_hadamard_rotate_weights(W, signs, block: int, W_out, stream=None) -> None:
    """W_out (fp32 [N, K]) = W R, R = diag(signs) blockdiag(Hadamard_block / sqrt(block))."""
    N, K = W.shape
    _check(lib.hq_hadamard_rotate_weights(_ptr(W), _dtype(W), N, K, int(block), _ptr(signs), _ptr(W_out),
                                          _stream(stream)), "hq_hadamard_rotate_weights")


def hq_hadamard_rotate_hessian(H, signs, block: int, H_out, stream=None) -> None:
    """H_out (fp32 [K, K]) = R^T H R, H read from its lower triangle."""
    K = H.shape[0]
    _check(lib.hq_hadamard_rotate_hessian(_ptr(H), K, int(block), _ptr(signs), _ptr(H_out), _stream(stream)),
           "hq_hadamard_rotate_hessian")


def hq_qerr_terms(workspace, terms_dev, stream=None) -> None:
    """terms_dev (fp64 [2], device) <- the qerr numerator and denominator sums of the last
    quantisation that used `workspace`."""
    _check(lib.hq_qerr_terms(_ptr(workspace), _ptr(terms_dev), _stream(stream)), "hq_qerr_terms")


def hq_debug_factor(H, damp: float, Ut_out, workspace, stream=None) -> None:
    K = H.shape[0]
    _check(lib.hq_debug_factor(_ptr(H), K, float(damp), _ptr(Ut_out), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream)), "hq_debug_factor")


def hq_debug_fp64_mma_rate(stream=None) -> float:
    """Measured fp64 MMA rate (TFLOP/s) of a kernel that does nothing else."""
    scratch = torch.empty(296 * 256, dtype=torch.float64, device="cuda")
    r = lib.hq_debug_fp64_mma_rate(_ptr(scratch), scratch.numel() * 8, _stream(stream))
    if r < 0:
        raise HQError(HQ_ERR_CUDA, "hq_debug_fp64_mma_rate")
    return float(r)


TIMING_CLASSES = {"f64_gemm_128": 0, "f64_gemm_64": 1, "leaf": 2, "sweep": 3, "tf32_gemm": 4, "syrk": 5,
                  "i8x_gemm": 6, "i8x_slice": 7}


def hq_debug_timing_start(classes) -> None:
    """Start event timing of the named kernel classes (see TIMING_CLASSES)."""
    mask = 0
    for c in classes:
        mask |= 1 << TIMING_CLASSES[c]
    _check(lib.hq_debug_timing_start(mask), "hq_debug_timing_start")


def hq_debug_timing_serialize(on: bool) -> None:
    """Run the factorisation's second-stream work on the caller's stream (on) or not (off)."""
    _check(lib.hq_debug_timing_serialize(1 if on else 0), "hq_debug_timing_serialize")


def hq_debug_timing_stop() -> None:
    _check(lib.hq_debug_timing_stop(), "hq_debug_timing_stop")


def hq_debug_timing_read(cls: str):
    """(total ms, total work, launches) recorded for one kernel class."""
    ms, work, n = ctypes.c_double(), ctypes.c_double(), ctypes.c_int64()
    _check(lib.hq_debug_timing_read(TIMING_CLASSES[cls], ctypes.byref(ms), ctypes.byref(work), ctypes.byref(n)),
           "hq_debug_timing_read")
    return ms.value, work.value, n.value


def hq_debug_upd_gemm(C, A_hi, A_lo, B_hi, B_lo, stream=None) -> None:
    """C -= (A_hi + A_lo) (B_hi + B_lo)^T by the lazy-update kernel (3xTF32)."""
    M, Kred = A_hi.shape
    N = B_hi.shape[0]
    _check(lib.hq_debug_upd_gemm(_ptr(C), C.stride(0), M, N, Kred, _ptr(A_hi), _ptr(A_lo), A_hi.stride(0),
                                 _ptr(B_hi), _ptr(B_lo), B_hi.stride(0), _stream(stream)), "hq_debug_upd_gemm")


def hq_debug_rcp_f64(d, out, stream=None) -> None:
    """out = 1 / d (fp64) by the factorisation leaf's pivot reciprocal."""
    _check(lib.hq_debug_rcp_f64(_ptr(d), _ptr(out), d.numel(), _stream(stream)), "hq_debug_rcp_f64")


def hq_debug_f64_gemm(C, A, B, alpha=1.0, beta=0.0, lower=False, tri=0, scratch=None, stream=None) -> None:
    """C = beta C + alpha A B^T (fp64 row-major views, fp64 tensor cores); tri declares a triangular operand."""
    M, Kred = A.shape
    N = B.shape[0]
    _check(lib.hq_debug_f64_gemm(_ptr(C), C.stride(0), M, N, Kred, _ptr(A), A.stride(0), _ptr(B), B.stride(0),
                                 float(alpha), float(beta), int(bool(lower)), int(tri), _ptr(scratch),
                                 0 if scratch is None else scratch.numel(), _stream(stream)), "hq_debug_f64_gemm")


def hq_debug_i8x_gemm(C, A, B, alpha=1.0, beta=0.0, lower=False, tri=0, scratch=None, stream=None) -> None:
    """C = beta C + alpha A B^T (fp64) through the int8-sliced tensor-core GEMM (hq_debug.h)."""
    M, Kred = A.shape
    N = B.shape[0]
    need = lib.hq_debug_i8x_scratch_bytes(M, N, Kred)
    if scratch is None:
        scratch = alloc_workspace(need, C.device)
    st = lib.hq_debug_i8x_gemm(_ptr(C), C.shape[1], M, N, Kred, _ptr(A), A.shape[1], _ptr(B), B.shape[1],
                               float(alpha), float(beta), int(bool(lower)), int(tri), _ptr(scratch),
                               scratch.numel() * scratch.element_size(), _stream(stream))
    _check(st, "hq_debug_i8x_gemm")


def hq_bf16tril_bytes(K: int) -> int:
    return int(lib.hq_bf16tril_bytes(K))


def hq_hessian_pack_bf16tril(H, out, stream=None) -> None:
    K = H.shape[0]
    _check(lib.hq_hessian_pack_bf16tril(_ptr(H), K, _ptr(out), _stream(stream)), "hq_hessian_pack_bf16tril")


def hq_hessian_unpack_bf16tril(inp, K: int, H_full, stream=None) -> None:
    _check(lib.hq_hessian_unpack_bf16tril(_ptr(inp), K, _ptr(H_full), _stream(stream)), "hq_hessian_unpack_bf16tril")


# --------------------------------------------------------------------------- e4m3 layers, experts

_FP8 = (torch.float8_e4m3fn, torch.uint8)


def _ptrs(*tensors):
    """The pointers of contiguous tensors (or None) that all live on the current device."""
    dev = torch._C._cuda_getDevice() if torch.cuda.is_initialized() else -2
    ptrs = []
    for t in tensors:
        if t is None:
            ptrs.append(None)
            continue
        if t.get_device() != dev:
            if not t.is_cuda:
                raise ValueError("expected a CUDA tensor")
            raise ValueError(f"expected tensors on the current device (cuda:{dev}), got {t.device}")
        if not t.is_contiguous():
            raise ValueError("expected a contiguous tensor")
        ptrs.append(t.data_ptr())
    return ptrs


def _want(t, name: str, dtype, shape) -> None:
    if t.dtype != dtype and not (isinstance(dtype, tuple) and t.dtype in dtype):
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, not {tuple(t.shape)}")


def _want_status(dev_status) -> None:
    if dev_status is not None and (dev_status.dtype != torch.int32 or dev_status.numel() < 1):
        raise ValueError("dev_status must be an int32 tensor")


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _pitch(K: int) -> int:
    return (K + 15) // 16 * 16


def hq_fp8_pitch(K: int) -> int:
    """Bytes of a row of codes."""
    return int(lib.hq_fp8_pitch(int(K)))


def hq_fp8_quantize_rows(X, codes, scales, stream=None) -> None:
    """X [M, K] -> e4m3 codes [M, pitch] (float8_e4m3fn or uint8) and scales fp32 [ceil(K/128), M]."""
    M, K = X.shape
    _want(codes, "codes", _FP8, (M, _pitch(K)))
    _want(scales, "scales", torch.float32, (_blocks(K), M))
    x, c, s = _ptrs(X, codes, scales)
    _check(lib.hq_fp8_quantize_rows(x, _dtype(X), M, K, c, s, _stream(stream)), "hq_fp8_quantize_rows")


def hq_fp8_quantize_blocks(W, codes, scales, stream=None) -> None:
    """W [N, K] or [E, N, K] -> codes [.., N, pitch] and scales fp32 [.., ceil(N/128), ceil(K/128)]."""
    *lead, N, K = W.shape
    if len(lead) > 1:
        raise ValueError("W must be [N, K] or [E, N, K]")
    _want(codes, "codes", _FP8, (*lead, N, _pitch(K)))
    _want(scales, "scales", torch.float32, (*lead, _blocks(N), _blocks(K)))
    w, c, s = _ptrs(W, codes, scales)
    _check(lib.hq_fp8_quantize_blocks(w, _dtype(W), lead[0] if lead else 1, N, K, c, s, _stream(stream)),
           "hq_fp8_quantize_blocks")


def hq_fp8_gemm(a_codes, a_scales, w_codes, w_scales, K: int, Y, dev_status=None, stream=None) -> None:
    """Y [M, N] = the product of quantised activations [M, pitch] and a quantised weight [N, pitch]."""
    M, N = Y.shape
    _want(a_codes, "a_codes", _FP8, (M, _pitch(K)))
    _want(a_scales, "a_scales", torch.float32, (_blocks(K), M))
    _want(w_codes, "w_codes", _FP8, (N, _pitch(K)))
    _want(w_scales, "w_scales", torch.float32, (_blocks(N), _blocks(K)))
    _want_status(dev_status)
    a, sa, w, sw, y, st = _ptrs(a_codes, a_scales, w_codes, w_scales, Y, dev_status)
    _check(lib.hq_fp8_gemm(a, sa, M, w, sw, N, K, y, _dtype(Y), st, _stream(stream)), "hq_fp8_gemm")


def hq_fp8_linear_workspace_bytes(M: int, K: int) -> int:
    return int(lib.hq_fp8_linear_workspace_bytes(int(M), int(K)))


def hq_fp8_linear(X, w_codes, w_scales, Y, workspace, dev_status=None, stream=None) -> None:
    """Y [M, N] = X [M, K], quantised on the way, times a quantised weight [N, pitch]."""
    M, K = X.shape
    N = w_codes.shape[0]
    _want(w_codes, "w_codes", _FP8, (N, _pitch(K)))
    _want(w_scales, "w_scales", torch.float32, (_blocks(N), _blocks(K)))
    if tuple(Y.shape) != (M, N):
        raise ValueError(f"Y must have shape {(M, N)}, not {tuple(Y.shape)}")
    _want_status(dev_status)
    x, w, sw, y, ws, st = _ptrs(X, w_codes, w_scales, Y, workspace, dev_status)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.hq_fp8_linear(x, _dtype(X), M, w, sw, N, K, y, _dtype(Y), ws, nbytes, st, _stream(stream)),
           "hq_fp8_linear")


def hq_fp8_expert_gemm(a_codes, a_scales, offsets, w_codes, w_scales, K: int, Y, dev_status=None, stream=None) -> None:
    """Rows offsets[e] .. offsets[e + 1] - 1 of Y [rows, N] = those rows of the quantised activations
    [rows, pitch] times weight e of the quantised [E, N, pitch]; offsets int32 [E + 1], on the device."""
    rows, N = Y.shape
    E = w_codes.shape[0]
    _want(a_codes, "a_codes", _FP8, (rows, _pitch(K)))
    _want(a_scales, "a_scales", torch.float32, (_blocks(K), rows))
    _want(offsets, "offsets", torch.int32, (E + 1,))
    _want(w_codes, "w_codes", _FP8, (E, N, _pitch(K)))
    _want(w_scales, "w_scales", torch.float32, (E, _blocks(N), _blocks(K)))
    _want_status(dev_status)
    a, sa, off, w, sw, y, st = _ptrs(a_codes, a_scales, offsets, w_codes, w_scales, Y, dev_status)
    _check(lib.hq_fp8_expert_gemm(a, sa, rows, off, w, sw, E, N, K, y, _dtype(Y), st, _stream(stream)),
           "hq_fp8_expert_gemm")


def _debug_fp8_gemm(name: str, a_codes, a_scales, offsets, w_codes, w_scales, K: int, Y, dev_status, stream, *last) -> None:
    rows, N = Y.shape
    lead = () if offsets is None else (w_codes.shape[0],)
    _want(a_codes, "a_codes", _FP8, (rows, _pitch(K)))
    _want(a_scales, "a_scales", torch.float32, (_blocks(K), rows))
    if offsets is not None:
        _want(offsets, "offsets", torch.int32, (lead[0] + 1,))
    _want(w_codes, "w_codes", _FP8, (*lead, N, _pitch(K)))
    _want(w_scales, "w_scales", torch.float32, (*lead, _blocks(N), _blocks(K)))
    _want_status(dev_status)
    a, sa, off, w, sw, y, st = _ptrs(a_codes, a_scales, offsets, w_codes, w_scales, Y, dev_status)
    _check(getattr(lib, name)(a, sa, rows, off, w, sw, 1 if offsets is None else w_codes.shape[0], N, K, y, _dtype(Y), st,
                              *last, _stream(stream)), name)


def hq_debug_fp8_gemm_impl(a_codes, a_scales, offsets, w_codes, w_scales, K: int, Y, impl: int, dev_status=None,
                           stream=None) -> None:
    """hq_fp8_gemm (offsets None) or hq_fp8_expert_gemm by a chosen kernel (hq_debug.h)."""
    _debug_fp8_gemm("hq_debug_fp8_gemm_impl", a_codes, a_scales, offsets, w_codes, w_scales, K, Y, dev_status, stream,
                    int(impl))


def hq_debug_fp8_gemm_timeout(a_codes, a_scales, offsets, w_codes, w_scales, K: int, Y, impl: int, dev_status,
                              wait_limit_cycles: int, withhold_stage: int = -1, stream=None) -> None:
    """The same with a runtime wait limit and, for the test of its timeout path, one operand stage that
    the MMA issuer never releases (hq_debug.h)."""
    _debug_fp8_gemm("hq_debug_fp8_gemm_timeout", a_codes, a_scales, offsets, w_codes, w_scales, K, Y, dev_status, stream,
                    int(impl), int(wait_limit_cycles), int(withhold_stage))


def hq_expert_sort_workspace_bytes(T: int, top: int, E: int) -> int:
    return int(lib.hq_expert_sort_workspace_bytes(int(T), int(top), int(E)))


def hq_expert_sort(ids, E: int, offsets, order, position, workspace, stream=None) -> None:
    """Stable sort of the choices ids (int32 [T, top]) by expert: offsets [E + 1], order [T * top]
    and position [T, top], all int32; -1 in position for an id outside [0, E)."""
    T, top = ids.shape
    _want(ids, "ids", torch.int32, (T, top))
    _want(offsets, "offsets", torch.int32, (E + 1,))
    _want(order, "order", torch.int32, (T * top,))
    _want(position, "position", torch.int32, (T, top))
    i, off, o, p, ws = _ptrs(ids, offsets, order, position, workspace)
    _check(lib.hq_expert_sort(i, T, top, E, off, o, p, ws, workspace.numel() * workspace.element_size(),
                              _stream(stream)), "hq_expert_sort")


def hq_expert_dispatch(X, position, rows, stream=None) -> None:
    """rows[position[t, j]] = X[t]; X [T, K], position int32 [T, top], rows [T * top, K]."""
    (T, K), top = X.shape, position.shape[1]
    _want(position, "position", torch.int32, (T, top))
    _want(rows, "rows", X.dtype, (T * top, K))
    x, p, r = _ptrs(X, position, rows)
    _check(lib.hq_expert_dispatch(x, _dtype(X), T, K, p, top, r, _stream(stream)), "hq_expert_dispatch")


def hq_expert_dispatch_fp8(X, position, codes, scales, stream=None) -> None:
    """The same with the rows quantised: codes [T * top, pitch], scales fp32 [ceil(K/128), T * top]."""
    (T, K), top = X.shape, position.shape[1]
    _want(position, "position", torch.int32, (T, top))
    _want(codes, "codes", _FP8, (T * top, _pitch(K)))
    _want(scales, "scales", torch.float32, (_blocks(K), T * top))
    x, p, c, s = _ptrs(X, position, codes, scales)
    _check(lib.hq_expert_dispatch_fp8(x, _dtype(X), T, K, p, top, c, s, _stream(stream)), "hq_expert_dispatch_fp8")


def hq_expert_combine(rows, position, weights, Y, stream=None) -> None:
    """Y[t] = sum_j weights[t, j] rows[position[t, j]]; weights fp32 [T, top] or None (all ones)."""
    (T, K), top = Y.shape, position.shape[1]
    _want(position, "position", torch.int32, (T, top))
    _want(rows, "rows", Y.dtype, (T * top, K))
    if weights is not None:
        _want(weights, "weights", torch.float32, (T, top))
    r, p, w, y = _ptrs(rows, position, weights, Y)
    _check(lib.hq_expert_combine(r, _dtype(Y), T, K, p, top, w, y, _stream(stream)), "hq_expert_combine")


def hq_expert_combine_backward(dY, rows, position, weights, d_rows, d_weights, stream=None) -> None:
    """d_rows[position[t, j]] = weights[t, j] dY[t], d_weights[t, j] = <dY[t], rows[position[t, j]]>."""
    (T, K), top = dY.shape, position.shape[1]
    _want(position, "position", torch.int32, (T, top))
    _want(rows, "rows", dY.dtype, (T * top, K))
    _want(d_rows, "d_rows", dY.dtype, (T * top, K))
    _want(weights, "weights", torch.float32, (T, top))
    _want(d_weights, "d_weights", torch.float32, (T, top))
    g, r, p, w, dr, dw = _ptrs(dY, rows, position, weights, d_rows, d_weights)
    _check(lib.hq_expert_combine_backward(g, r, _dtype(dY), T, K, p, top, w, dr, dw, _stream(stream)),
           "hq_expert_combine_backward")


# --------------------------------------------------------------------------- allocation helpers

def alloc_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A uint8 device buffer of nbytes (torch's caching allocator returns 512-byte aligned blocks)."""
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def gptq_outputs(N: int, K: int, group: int, device="cuda"):
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=device)
    scales = torch.empty((N, K // group), dtype=torch.float32, device=device)
    return codes, scales


def fp8_rows_outputs(M: int, K: int, device="cuda"):
    """Codes [M, pitch] and scales [ceil(K/128), M] of quantised activations."""
    return (torch.empty((M, _pitch(K)), dtype=torch.float8_e4m3fn, device=device),
            torch.empty((_blocks(K), M), dtype=torch.float32, device=device))


def fp8_blocks_outputs(N: int, K: int, E: int | None = None, device="cuda"):
    """Codes [N, pitch] and scales [ceil(N/128), ceil(K/128)] of a quantised weight; [E, ..] with E."""
    lead = () if E is None else (E,)
    return (torch.empty((*lead, N, _pitch(K)), dtype=torch.float8_e4m3fn, device=device),
            torch.empty((*lead, _blocks(N), _blocks(K)), dtype=torch.float32, device=device))


def expert_sort_outputs(T: int, top: int, E: int, device="cuda"):
    """offsets [E + 1], order [T * top] and position [T, top]."""
    return (torch.empty(E + 1, dtype=torch.int32, device=device),
            torch.empty(T * top, dtype=torch.int32, device=device),
            torch.empty((T, top), dtype=torch.int32, device=device))
