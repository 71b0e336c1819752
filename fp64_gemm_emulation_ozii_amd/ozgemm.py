"""ctypes binding of ``libozgemm.so`` (the C-ABI declared in ``include/ozgemm.h``).

Functions carry the C names and only marshal arguments: torch tensors become
device pointers, ``None`` becomes NULL, the stream defaults to torch's
current stream.  Every step of the computation runs in the HIP library; if
the library is missing this module raises instead of computing anything.

A non-zero status raises :class:`OzgemmError` (with ``ozgemm_strerror``'s
text) unless the function is documented to return a value.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libozgemm.so")

OZGEMM_OK = 0
OZGEMM_NOT_CONFIGURED = 1
OZGEMM_RANGE = 2
OZGEMM_WORKSPACE_TOO_SMALL = 3
OZGEMM_HIP_ERROR = 4
OZGEMM_S_MAX = 20
OZGEMM_PANELS_MAX = 16
OZGEMM_Q_LIMIT = 1 << 17
OZGEMM_Q_MAX = 1 << 27
OZGEMM_FAST_Q_LIMIT = 1 << 23  # OS II-fast needs q below this
OZGEMM_NOALLOC_BYTES = 128 << 20  # the fixed device array of ozgemm_dgemm_noalloc
OZGEMM_MAX_ROWS = 2096896  # 2^21 - 256
OZGEMM_ONE_PASS_Q_MIN = 4096  # B read once by ozgemm_dgemm for q in [MIN, MAX] (conservative budget)
OZGEMM_ONE_PASS_Q_MAX = 8192
OZGEMM_EXP_NONFINITE = 0x7FFFFFFF
OZGEMM_BOUND_CONSERVATIVE = 0
OZGEMM_BOUND_FAST = 1
OZGEMM_BOUND_ACCU = 2
OZGEMM_ACCU_Q_MAX = 1 << 16
OZGEMM_S1_RN = 0
OZGEMM_S1_HYBRID = 1
OZGEMM_S1_K_MAX = 16
OZGEMM_S1_MAX_OUT = 136
OZGEMM_F64 = 0
OZGEMM_F32 = 1
OZGEMM_BF16 = 2
OZGEMM_F16 = 3
OZGEMM_E4M3 = 4
OZGEMM_E5M2 = 5
OZGEMM_GROUPS_MAX = 65536
OZGEMM_ORTHO_MAX = 65536
OZGEMM_ORTHO_STEPS_MAX = 64
OZGEMM_ARRAYS_MAX = 65536
OZGEMM_ARRAY_MAX = 1 << 40

#: every symbol the header declares
EXPORTS = (
    "ozgemm_workspace_bytes", "ozgemm_config", "ozgemm_set_stream", "ozgemm_free", "ozgemm_strerror",
    "ozgemm_dgemm", "ozgemm_moduli", "ozgemm_kbits", "ozgemm_plane_dims", "ozgemm_stage_scale",
    "ozgemm_stage_residue", "ozgemm_stage_gemm", "ozgemm_stage_crt", "ozgemm_timing", "ozgemm_phase_ms",
    "ozgemm_scheme1_beta", "ozgemm_scheme1_outputs", "ozgemm_scheme1_workspace_bytes", "ozgemm_scheme1_dgemm",
    "ozgemm_scheme1_stage_split", "ozgemm_scheme1_stage_products", "ozgemm_scheme1_stage_accumulate",
    "ozgemm_set_bound", "ozgemm_bound_budget", "ozgemm_gemm_parts", "ozgemm_phase_calls",
    "ozgemm_dgemm_noalloc", "ozgemm_set_panels", "ozgemm_mfma_ceiling",
    "ozgemm_grouped_gemm", "ozgemm_grouped_gemm_workspace_bytes", "ozgemm_grouped_outer",
    "ozgemm_grouped_outer_workspace_bytes", "ozgemm_orthogonalize", "ozgemm_orthogonalize_workspace_bytes",
    "ozgemm_quantize_blocks", "ozgemm_scaled_gemm", "ozgemm_scaled_gemm_workspace_bytes", "ozgemm_rms_norm",
    "ozgemm_rms_norm_grads", "ozgemm_rms_norm_grads_workspace_bytes", "ozgemm_gradient_norm",
    "ozgemm_gradient_norm_workspace_bytes", "ozgemm_clip_gradients",
)

_lib = None
_workspace = None  # keeps a library-config workspace tensor alive


class OzgemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status}: {ozgemm_strerror(status)}")


def lib():
    """Load the library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m fp64_gemm_emulation_ozii_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    c_int, c_size, vp = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
    ip = ctypes.POINTER(ctypes.c_int)
    sig = {
        "ozgemm_workspace_bytes": (c_size, [c_int, c_int, c_int, c_int]),
        "ozgemm_config": (c_int, [c_int, c_int, c_int, c_int, vp, vp, c_size]),
        "ozgemm_set_stream": (c_int, [vp]),
        "ozgemm_set_panels": (c_int, [c_int]),
        "ozgemm_free": (c_int, []),
        "ozgemm_strerror": (ctypes.c_char_p, [c_int]),
        "ozgemm_dgemm": (c_int, [c_int, c_int, c_int, vp, c_int, vp, c_int, vp, c_int, c_int]),
        "ozgemm_dgemm_noalloc": (c_int, [c_int, c_int, c_int, vp, c_int, vp, c_int, vp, c_int, c_int, vp]),
        "ozgemm_moduli": (c_int, [c_int, ip]),
        "ozgemm_kbits": (c_int, [c_int, c_int]),
        "ozgemm_plane_dims": (c_int, [c_int, c_int, c_int, ip, ip, ip]),
        "ozgemm_stage_scale": (c_int, [c_int, c_int, c_int, c_int, vp, c_int, vp, c_int, vp, vp]),
        "ozgemm_set_bound": (c_int, [c_int]),
        "ozgemm_bound_budget": (c_int, [c_int, c_int, c_int, ip, ip]),
        "ozgemm_stage_residue": (c_int, [c_int, c_int, c_int, c_int, vp, c_int, vp, c_int, vp, vp, vp, vp, vp, vp]),
        "ozgemm_stage_gemm": (c_int, [c_int, c_int, c_int, c_int, vp, vp, vp, vp]),
        "ozgemm_stage_crt": (c_int, [c_int, c_int, c_int, c_int, vp, vp, vp, vp, c_int]),
        "ozgemm_gemm_parts": (c_int, [c_int, c_int, c_int, c_int, ip]),
        "ozgemm_timing": (c_int, [c_int]),
        "ozgemm_phase_ms": (c_int, [ctypes.POINTER(ctypes.c_double), ip]),
        "ozgemm_phase_calls": (c_int, [ctypes.POINTER(ctypes.c_double), c_int, ip]),
        "ozgemm_mfma_ceiling": (c_int, [c_int, c_int, ctypes.c_uint, vp, vp]),
        "ozgemm_scheme1_beta": (c_int, [c_int]),
        "ozgemm_scheme1_outputs": (c_int, [c_int, c_int, c_int]),
        "ozgemm_scheme1_workspace_bytes": (c_size, [c_int, c_int, c_int, c_int, c_int]),
        "ozgemm_scheme1_dgemm": (c_int, [c_int, c_int, c_int, vp, c_int, vp, c_int, vp, c_int, c_int, c_int]),
        "ozgemm_scheme1_stage_split": (c_int, [c_int, c_int, c_int, c_int, c_int, vp, c_int, vp, c_int, vp, vp, vp,
                                               vp]),
        "ozgemm_scheme1_stage_products": (c_int, [c_int, c_int, c_int, c_int, c_int, vp, vp, vp]),
        "ozgemm_scheme1_stage_accumulate": (c_int, [c_int, c_int, c_int, c_int, c_int, vp, vp, vp, vp, c_int]),
    }
    ll = ctypes.c_longlong
    sig.update({
        "ozgemm_grouped_gemm": (c_int, [c_int] * 7 + [vp, c_int, ll, vp, c_int, vp, vp, c_int, vp, c_size, vp]),
        "ozgemm_grouped_gemm_workspace_bytes": (c_size, [c_int] * 6 + [vp, c_int, ll, vp, c_int]),
        "ozgemm_grouped_outer": (c_int, [c_int] * 6 + [vp, c_int, vp, c_int, vp, vp, c_int, ll, vp, c_size, vp]),
        "ozgemm_orthogonalize": (c_int, [c_int] * 4 + [vp, c_int, ll, c_int, ctypes.POINTER(ctypes.c_double),
                                         ctypes.c_double, c_int, vp, c_int, ll, vp, c_size, vp]),
        "ozgemm_orthogonalize_workspace_bytes": (c_size, [c_int] * 5),
        "ozgemm_grouped_outer_workspace_bytes": (c_size, [c_int] * 5 + [vp, c_int, vp, c_int]),
    })
    f64 = ctypes.c_double
    ints, lls, ptrs = ip, ctypes.POINTER(ll), ctypes.POINTER(vp)
    sig.update({
        "ozgemm_quantize_blocks": (c_int, [c_int] * 5 + [vp, c_int] + [vp, c_int, vp, ll, ll] * 2 + [vp]),
        "ozgemm_scaled_gemm": (c_int, [c_int] * 6 + [vp, c_int, vp, c_int, ll, ll, vp, c_int, vp, ll, ll, vp, c_int, vp,
                                       c_size, vp]),
        "ozgemm_scaled_gemm_workspace_bytes": (c_size, [c_int] * 3 + [vp, c_int, c_int, ll, ll, vp, c_int, ll, ll]),
        "ozgemm_rms_norm": (c_int, [c_int] * 5 + [vp, c_int, vp, c_int, vp, f64, vp, c_int, vp, c_int, vp, ll, ll, vp]),
        "ozgemm_rms_norm_grads": (c_int, [c_int] * 4 + [vp, c_int, vp, c_int, vp, vp, c_int, f64, vp, c_int, vp, vp,
                                          c_size, vp]),
        "ozgemm_rms_norm_grads_workspace_bytes": (c_size, [c_int] * 3),
        "ozgemm_gradient_norm": (c_int, [c_int, ints, ptrs, lls, vp, vp, c_size, vp]),
        "ozgemm_gradient_norm_workspace_bytes": (c_size, [c_int, ints, lls]),
        "ozgemm_clip_gradients": (c_int, [c_int, ints, ptrs, lls, ptrs, vp, f64, f64, vp]),
    })
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def _ptr(x):
    """Device pointer of a tensor, an int address, or None (NULL)."""
    if x is None or isinstance(x, int):
        return x
    return x.data_ptr()


def _check(status: int, where: str) -> int:
    if status != OZGEMM_OK:
        raise OzgemmError(status, where)
    return status


def _stream(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _current_stream() -> int:
    """torch's current stream (the first call looks up how to ask for it
    without a Stream object, which takes 5 us less)."""
    global _current_stream
    import torch
    raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    known = torch.cuda.is_initialized

    def ask() -> int:
        if raw is not None and device is not None and known():
            return raw(device())
        return torch.cuda.current_stream().cuda_stream

    _current_stream = ask
    return ask()


# --------------------------------------------------------------------------
# host-only
# --------------------------------------------------------------------------

def ozgemm_strerror(status: int) -> str:
    return lib().ozgemm_strerror(status).decode()


def ozgemm_workspace_bytes(max_m: int, max_n: int, max_q: int, s_max: int) -> int:
    return int(lib().ozgemm_workspace_bytes(max_m, max_n, max_q, s_max))


def ozgemm_moduli(s: int) -> list[int]:
    buf = (ctypes.c_int * max(s, 1))()
    _check(lib().ozgemm_moduli(s, buf), "ozgemm_moduli")
    return list(buf)[:s]


def ozgemm_kbits(s: int, q: int) -> int:
    """Returns k (negative when no bits are left); never raises."""
    return int(lib().ozgemm_kbits(s, q))


def ozgemm_plane_dims(m: int, n: int, q: int):
    a, b, c = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check(lib().ozgemm_plane_dims(m, n, q, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)), "ozgemm_plane_dims")
    return a.value, b.value, c.value


# --------------------------------------------------------------------------
# configuration
# --------------------------------------------------------------------------

def ozgemm_config(s_max: int, max_m: int, max_n: int, max_q: int, stream=None, workspace=None,
                  workspace_bytes: int | None = None, scheme1_k: int = 0, scheme1_variant: int = OZGEMM_S1_RN) -> int:
    """Configure the library.  With ``workspace=None`` a torch uint8 device
    tensor of ``ozgemm_workspace_bytes(...)`` bytes is allocated and kept
    alive here -- or of ``ozgemm_scheme1_workspace_bytes(max_m, max_n, max_q,
    scheme1_k, scheme1_variant)`` bytes when ``scheme1_k`` > 0 and that is
    larger."""
    global _workspace
    need = ozgemm_workspace_bytes(max_m, max_n, max_q, s_max)
    if scheme1_k > 0:
        need = max(need, ozgemm_scheme1_workspace_bytes(max_m, max_n, max_q, scheme1_k, scheme1_variant))
    hs = _stream(stream)
    if workspace is None:
        import torch
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
        workspace_bytes = need
    elif workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    st = lib().ozgemm_config(s_max, max_m, max_n, max_q, hs, _ptr(workspace), workspace_bytes)
    _check(st, "ozgemm_config")  # on failure the previous configuration and its workspace stay
    _release_workspace()
    _workspace = workspace
    return st


def _release_workspace():
    """Drop the workspace reference held here, after every kernel queued on
    the device has finished: the configured stream may differ from the one the
    tensor was allocated on, and the caching allocator would otherwise hand
    the bytes to new work while queued calls still read and write them."""
    global _workspace
    if _workspace is not None:
        import torch
        torch.cuda.synchronize()
    _workspace = None


def ozgemm_set_stream(stream=None) -> int:
    """Later calls go on `stream`.  Work already queued on the previous stream
    is not ordered before them: the caller orders the two streams."""
    return _check(lib().ozgemm_set_stream(_stream(stream)), "ozgemm_set_stream")


def ozgemm_set_panels(panels: int) -> int:
    """Column panels of the ozgemm_dgemm pipeline: 0 or 1 no pipeline (the
    default), 2..OZGEMM_PANELS_MAX that many panels where the shape allows."""
    return _check(lib().ozgemm_set_panels(panels), "ozgemm_set_panels")


def ozgemm_free() -> int:
    st = lib().ozgemm_free()
    _release_workspace()
    return st


# --------------------------------------------------------------------------
# compute (raw C-ABI signatures; matrices are column-major device buffers)
# --------------------------------------------------------------------------

def ozgemm_dgemm(m, n, q, A, lda, B, ldb, C, ldc, s, check: bool = True) -> int:
    st = lib().ozgemm_dgemm(m, n, q, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, s)
    return _check(st, "ozgemm_dgemm") if check else st


def ozgemm_dgemm_noalloc(m, n, q, A, lda, B, ldb, C, ldc, s, stream=None, check: bool = True) -> int:
    st = lib().ozgemm_dgemm_noalloc(m, n, q, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, s, _stream(stream))
    return _check(st, "ozgemm_dgemm_noalloc") if check else st


def ozgemm_stage_scale(m, n, q, s, A, lda, B, ldb, e, f, check: bool = True) -> int:
    st = lib().ozgemm_stage_scale(m, n, q, s, _ptr(A), lda, _ptr(B), ldb, _ptr(e), _ptr(f))
    return _check(st, "ozgemm_stage_scale") if check else st


def ozgemm_stage_residue(m, n, q, s, A, lda, B, ldb, e, f, Ares, Bres, Aprime=None, Bprime=None,
                         check: bool = True) -> int:
    st = lib().ozgemm_stage_residue(m, n, q, s, _ptr(A), lda, _ptr(B), ldb, _ptr(e), _ptr(f), _ptr(Ares),
                                    _ptr(Bres), _ptr(Aprime), _ptr(Bprime))
    return _check(st, "ozgemm_stage_residue") if check else st


def ozgemm_stage_gemm(m, n, q, s, Ares, Bres, Ct=None, rt=None, check: bool = True) -> int:
    st = lib().ozgemm_stage_gemm(m, n, q, s, _ptr(Ares), _ptr(Bres), _ptr(Ct), _ptr(rt))
    return _check(st, "ozgemm_stage_gemm") if check else st


def ozgemm_stage_crt(m, n, q, s, rt, e, f, C, ldc, check: bool = True) -> int:
    st = lib().ozgemm_stage_crt(m, n, q, s, _ptr(rt), _ptr(e), _ptr(f), _ptr(C), ldc)
    return _check(st, "ozgemm_stage_crt") if check else st


def ozgemm_gemm_parts(m: int, n: int, q: int, s: int) -> int:
    """K parts of the residue-only product of an m x n x q call (needs a device)."""
    p = ctypes.c_int()
    _check(lib().ozgemm_gemm_parts(m, n, q, s, ctypes.byref(p)), "ozgemm_gemm_parts")
    return p.value


def ozgemm_set_bound(mode: int) -> int:
    return _check(lib().ozgemm_set_bound(mode), "ozgemm_set_bound")


def ozgemm_bound_budget(s: int, q: int, mode: int):
    """(kappa_A, kappa_B) of the bit budget, or raises."""
    a, b = ctypes.c_int(), ctypes.c_int()
    _check(lib().ozgemm_bound_budget(s, q, mode, ctypes.byref(a), ctypes.byref(b)), "ozgemm_bound_budget")
    return a.value, b.value


def ozgemm_scheme1_beta(q: int) -> int:
    return lib().ozgemm_scheme1_beta(q)


def ozgemm_scheme1_outputs(k: int, variant: int, q: int) -> int:
    return lib().ozgemm_scheme1_outputs(k, variant, q)


def ozgemm_scheme1_workspace_bytes(m: int, n: int, q: int, k: int, variant: int) -> int:
    return lib().ozgemm_scheme1_workspace_bytes(m, n, q, k, variant)


def ozgemm_scheme1_dgemm(m, n, q, A, lda, B, ldb, C, ldc, k, variant=OZGEMM_S1_RN, check: bool = True) -> int:
    st = lib().ozgemm_scheme1_dgemm(m, n, q, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, k, variant)
    return _check(st, "ozgemm_scheme1_dgemm") if check else st


def ozgemm_scheme1_stage_split(m, n, q, k, variant, A, lda, B, ldb, Aslices, Bslices, gA, gB,
                               check: bool = True) -> int:
    st = lib().ozgemm_scheme1_stage_split(m, n, q, k, variant, _ptr(A), lda, _ptr(B), ldb, _ptr(Aslices),
                                          _ptr(Bslices), _ptr(gA), _ptr(gB))
    return _check(st, "ozgemm_scheme1_stage_split") if check else st


def ozgemm_scheme1_stage_products(m, n, q, k, variant, Aslices, Bslices, P, check: bool = True) -> int:
    st = lib().ozgemm_scheme1_stage_products(m, n, q, k, variant, _ptr(Aslices), _ptr(Bslices), _ptr(P))
    return _check(st, "ozgemm_scheme1_stage_products") if check else st


def ozgemm_scheme1_stage_accumulate(m, n, q, k, variant, P, gA, gB, C, ldc, check: bool = True) -> int:
    st = lib().ozgemm_scheme1_stage_accumulate(m, n, q, k, variant, _ptr(P), _ptr(gA), _ptr(gB), _ptr(C), ldc)
    return _check(st, "ozgemm_scheme1_stage_accumulate") if check else st


def ozgemm_timing(enable: bool) -> int:
    return _check(lib().ozgemm_timing(1 if enable else 0), "ozgemm_timing")


def ozgemm_phase_ms():
    """Returns ([scale, residue, gemm, crt] total milliseconds, calls)."""
    buf = (ctypes.c_double * 4)()
    calls = ctypes.c_int()
    _check(lib().ozgemm_phase_ms(buf, ctypes.byref(calls)), "ozgemm_phase_ms")
    return list(buf), calls.value


def ozgemm_mfma_ceiling(blocks: int, steps: int, seed: int, sink, stream=None, check: bool = True) -> int:
    """Launch the int8 matrix-core rate probe (asynchronous on `stream`, a
    torch stream or None for the current one); sink: int32 device tensor of
    at least 4 * blocks elements."""
    import torch
    if sink.numel() < 4 * blocks or sink.element_size() != 4 or not sink.is_contiguous():
        raise ValueError("sink must be a contiguous 4-byte tensor of at least 4 * blocks elements")
    s = stream if stream is not None else torch.cuda.current_stream()
    st = lib().ozgemm_mfma_ceiling(blocks, steps, seed & 0xFFFFFFFF, _ptr(sink), s.cuda_stream)
    return _check(st, "ozgemm_mfma_ceiling") if check else st


def ozgemm_phase_calls():
    """Per-call phase times: a list of [scale, residue, gemm, crt] ms, one per
    timed call."""
    calls = ctypes.c_int()
    _check(lib().ozgemm_phase_calls(None, 0, ctypes.byref(calls)), "ozgemm_phase_calls")
    n = calls.value
    buf = (ctypes.c_double * max(4 * n, 1))()
    _check(lib().ozgemm_phase_calls(buf, n, ctypes.byref(calls)), "ozgemm_phase_calls")
    return [list(buf[4 * c:4 * c + 4]) for c in range(n)]


# --------------------------------------------------------------------------
# products over ragged groups (raw C-ABI signatures; column-major)
# --------------------------------------------------------------------------

# the workspace's argument number: what a call returns that needs one and has none
_GEMM_NO_WORKSPACE = -16
_OUTER_NO_WORKSPACE = -15


def _room(workspace, nbytes: int, device, stream: int):
    """(tensor kept alive, pointer, bytes) of a call's workspace: the given
    one, or one from torch's allocator.

    The allocator hands a freed block out again to work of the stream that was
    current when it was allocated, and only after what that stream has queued
    by then.  So the block is taken while the stream that the call runs on is the
    current one."""
    if workspace is not None:
        return workspace, _ptr(workspace), workspace.numel() * workspace.element_size()
    if nbytes == 0:
        return None, None, 0
    import torch
    if stream == _current_stream():
        t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif 0 < stream < 4096 or stream & 1:  # HIP's names for the legacy stream and a thread's own: no stream object's address
        raise ValueError(f"a call on the stream {stream:#x} needs its workspace given")
    else:
        with torch.cuda.stream(torch.cuda.ExternalStream(stream, device) if stream else
                               torch.cuda.default_stream(device)):
            t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return t, t.data_ptr(), nbytes


def ozgemm_grouped_gemm_workspace_bytes(type, groups, m, n, q, transa, A, lda, stridea, B, ldb) -> int:
    return int(lib().ozgemm_grouped_gemm_workspace_bytes(type, groups, m, n, q, transa, _ptr(A), lda, stridea,
                                                         _ptr(B), ldb))


def ozgemm_grouped_gemm(type, ctype, groups, m, n, q, transa, A, lda, stridea, B, ldb, offsets, C, ldc,
                        workspace=None, stream=None, check: bool = True) -> int:
    """With ``workspace=None`` the bytes the call needs, if any, come from
    torch's allocator, on the stream that the call runs on (``stream``: a torch
    stream or a handle; the current one by default); a given workspace (a device
    tensor) stays the caller's."""
    L, hs = lib(), _stream(stream)
    ops = (type, ctype, groups, m, n, q, transa, _ptr(A), lda, stridea, _ptr(B), ldb, _ptr(offsets), _ptr(C), ldc)
    st = None
    if workspace is None:  # operands are usually read in place
        st = L.ozgemm_grouped_gemm(*ops, None, 0, hs)
        if st == OZGEMM_OK:
            return st
    if st is None or st == _GEMM_NO_WORKSPACE:
        need = 0 if workspace is not None else ozgemm_grouped_gemm_workspace_bytes(type, groups, m, n, q, transa, A,
                                                                                  lda, stridea, B, ldb)
        keep, ws, nbytes = _room(workspace, need, getattr(B, "device", "cuda"), hs)
        st = L.ozgemm_grouped_gemm(*ops, ws, nbytes, hs)
    return _check(st, "ozgemm_grouped_gemm") if check else st


def ozgemm_grouped_outer_workspace_bytes(type, groups, m, q, n, A, lda, B, ldb) -> int:
    return int(lib().ozgemm_grouped_outer_workspace_bytes(type, groups, m, q, n, _ptr(A), lda, _ptr(B), ldb))


def ozgemm_grouped_outer(type, ctype, groups, m, q, n, A, lda, B, ldb, offsets, C, ldc, stridec, workspace=None,
                         stream=None, check: bool = True) -> int:
    """Workspace as for :func:`ozgemm_grouped_gemm`."""
    L, hs = lib(), _stream(stream)
    ops = (type, ctype, groups, m, q, n, _ptr(A), lda, _ptr(B), ldb, _ptr(offsets), _ptr(C), ldc, stridec)
    st = _OUTER_NO_WORKSPACE if workspace is None else None
    if workspace is None and type != OZGEMM_F32:
        st = L.ozgemm_grouped_outer(*ops, None, 0, hs)
    if st is None or st == _OUTER_NO_WORKSPACE:
        need = 0 if workspace is not None else ozgemm_grouped_outer_workspace_bytes(type, groups, m, q, n, A, lda, B,
                                                                                   ldb)
        keep, ws, nbytes = _room(workspace, need, getattr(B, "device", "cuda"), hs)
        st = L.ozgemm_grouped_outer(*ops, ws, nbytes, hs)
    return _check(st, "ozgemm_grouped_outer") if check else st


def ozgemm_orthogonalize_workspace_bytes(type, batch, m, n, s) -> int:
    return int(lib().ozgemm_orthogonalize_workspace_bytes(type, batch, m, n, s))


def ozgemm_orthogonalize(type, batch, m, n, G, ldg, strideg, steps, coeffs, eps, s, O, ldo, strideo, workspace=None,
                         stream=None, check: bool = True) -> int:
    """``coeffs``: 3 * steps host numbers.  Workspace as for
    :func:`ozgemm_grouped_gemm`."""
    hs = _stream(stream)
    co = (ctypes.c_double * max(3 * steps, 1))(*coeffs) if coeffs is not None else None
    need = ozgemm_orthogonalize_workspace_bytes(type, batch, m, n, s)
    keep, ws, nbytes = _room(workspace, need, getattr(G, "device", "cuda"), hs)
    st = lib().ozgemm_orthogonalize(type, batch, m, n, _ptr(G), ldg, strideg, steps, co, eps, s, _ptr(O), ldo,
                                    strideo, ws, nbytes, hs)
    return _check(st, "ozgemm_orthogonalize") if check else st


# --------------------------------------------------------------------------
# a layer in 8 bits, and the clipping of gradients (raw C-ABI signatures)
# --------------------------------------------------------------------------

def ozgemm_quantize_blocks(type, qtype, rows, n, q, X, ldx, V, ldv, S, srow, sblock, Vt=None, ldvt=0, St=None, strow=0,
                           stblock=0, stream=None, check: bool = True) -> int:
    st = lib().ozgemm_quantize_blocks(type, qtype, rows, n, q, _ptr(X), ldx, _ptr(V), ldv, _ptr(S), srow, sblock,
                                      _ptr(Vt), ldvt, _ptr(St), strow, stblock, _stream(stream))
    return _check(st, "ozgemm_quantize_blocks") if check else st


_SCALED_NO_WORKSPACE = -20


def ozgemm_scaled_gemm_workspace_bytes(m, n, q, A, lda, rows_a, sarow, sablock, B, ldb, sbrow, sbblock) -> int:
    return int(lib().ozgemm_scaled_gemm_workspace_bytes(m, n, q, _ptr(A), lda, rows_a, sarow, sablock, _ptr(B),
                                                        ldb, sbrow, sbblock))


def ozgemm_scaled_gemm(atype, btype, ctype, m, n, q, A, lda, SA, rows_a, sarow, sablock, B, ldb, SB, sbrow, sbblock, C,
                       ldc, workspace=None, stream=None, check: bool = True) -> int:
    """Workspace as for :func:`ozgemm_grouped_gemm`."""
    L, hs = lib(), _stream(stream)
    ops = (atype, btype, ctype, m, n, q, _ptr(A), lda, _ptr(SA), rows_a, sarow, sablock, _ptr(B), ldb, _ptr(SB), sbrow,
           sbblock, _ptr(C), ldc)
    st = _SCALED_NO_WORKSPACE
    if workspace is None:  # operands are usually read in place
        st = L.ozgemm_scaled_gemm(*ops, None, 0, hs)
    if st == _SCALED_NO_WORKSPACE:
        need = 0 if workspace is not None else ozgemm_scaled_gemm_workspace_bytes(
            m, n, q, A, lda, rows_a, sarow, sablock, B, ldb, sbrow, sbblock)
        keep, ws, nbytes = _room(workspace, need, getattr(B, "device", "cuda"), hs)
        st = L.ozgemm_scaled_gemm(*ops, ws, nbytes, hs)
    return _check(st, "ozgemm_scaled_gemm") if check else st


def ozgemm_rms_norm(type, ytype, wtype, n, q, X, ldx, R, ldr, w, eps, H, ldh, Y, ldy, S=None, srow=0, sblock=0,
                    stream=None, check: bool = True) -> int:
    st = lib().ozgemm_rms_norm(type, ytype, wtype, n, q, _ptr(X), ldx, _ptr(R), ldr, _ptr(w), eps, _ptr(H), ldh,
                               _ptr(Y), ldy, _ptr(S), srow, sblock, _stream(stream))
    return _check(st, "ozgemm_rms_norm") if check else st


def ozgemm_rms_norm_grads_workspace_bytes(n, q, dw) -> int:
    return int(lib().ozgemm_rms_norm_grads_workspace_bytes(n, q, dw))


def ozgemm_rms_norm_grads(type, wtype, n, q, dY, lddy, H, ldh, w, dH, lddh, eps, dX, lddx, dw, workspace=None,
                          stream=None, check: bool = True) -> int:
    """Workspace as for :func:`ozgemm_grouped_gemm`."""
    hs = _stream(stream)
    need = 0 if workspace is not None else ozgemm_rms_norm_grads_workspace_bytes(n, q, 1 if dw is not None else 0)
    keep, ws, nbytes = _room(workspace, need, getattr(H, "device", "cuda"), hs)
    st = lib().ozgemm_rms_norm_grads(type, wtype, n, q, _ptr(dY), lddy, _ptr(H), ldh, _ptr(w), _ptr(dH), lddh, eps,
                                     _ptr(dX), lddx, _ptr(dw), ws, nbytes, hs)
    return _check(st, "ozgemm_rms_norm_grads") if check else st


def _arrays(types, tensors, sizes):
    """C arrays of the types, addresses and sizes."""
    n = max(1, len(types))
    return ((ctypes.c_int * n)(*types), (ctypes.c_void_p * n)(*[t if isinstance(t, int) else t.data_ptr() for t in tensors]),
            (ctypes.c_longlong * n)(*sizes))


def ozgemm_gradient_norm_workspace_bytes(types, sizes) -> int:
    t, _, s = _arrays(types, [], sizes)
    return int(lib().ozgemm_gradient_norm_workspace_bytes(len(types), t, s))


def _gradient_norm(count, t, p, s, norm, workspace, hs) -> int:
    need = 0 if workspace is not None else int(lib().ozgemm_gradient_norm_workspace_bytes(count, t, s))
    keep, ws, nbytes = _room(workspace, need, getattr(norm, "device", "cuda"), hs)
    return lib().ozgemm_gradient_norm(count, t, p, s, _ptr(norm), ws, nbytes, hs)


def ozgemm_gradient_norm(types, arrays, sizes, norm, workspace=None, stream=None, check: bool = True) -> int:
    """``types``, ``arrays`` (tensors or addresses) and ``sizes``: lists of one
    length.  Workspace as for :func:`ozgemm_grouped_gemm`."""
    st = _gradient_norm(len(types), *_arrays(types, arrays, sizes), norm, workspace, _stream(stream))
    return _check(st, "ozgemm_gradient_norm") if check else st


def ozgemm_clip_gradients(types, arrays, sizes, out, norm, most, eps, measured: bool = True, workspace=None,
                          stream=None, check: bool = True) -> int:
    """With ``measured=False`` the norm is worked out first (:func:`ozgemm_gradient_norm`, with that workspace)."""
    hs = _stream(stream)
    t, p, s = _arrays(types, arrays, sizes)
    o = p if out is arrays else (ctypes.c_void_p * max(1, len(types)))(*[
        x if isinstance(x, int) else x.data_ptr() for x in out])
    st = OZGEMM_OK if measured else _gradient_norm(len(types), t, p, s, norm, workspace, hs)
    if st == OZGEMM_OK:
        st = lib().ozgemm_clip_gradients(len(types), t, p, s, o, _ptr(norm), most, eps, hs)
    return _check(st, "ozgemm_clip_gradients") if check else st
