"""Python binding of the GB300 Muon update library (``include/muon.h``).

Argument marshalling only: every step of the update runs in the library's CUDA
kernels.  The functions keep the C names; tensors are PyTorch CUDA tensors
(PyTorch supplies device memory and streams).  Loading fails loudly when the
shared library has not been built: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libmuon_gb300.so")

MUON_OK = 0
MUON_EINVAL = -1
MUON_EDTYPE = -2
MUON_ENOMEM = -3
MUON_ECUDA = -4
MUON_ENONFINITE = -5
MUON_ETIMEOUT = -6
MUON_ENOTSUP = -7

MUON_F32 = 0
MUON_BF16 = 1
MUON_F16 = 2

MUON_I32 = 32
MUON_I64 = 64

MUON_PATH_AUTO = 0
MUON_PATH_PLAIN = 1
MUON_PATH_GRAM = 2

QUINTIC = (3.4445, -4.7750, 2.0315)

#: every entry point include/muon.h declares
EXPORTS = (
    "muon_ns_orthogonalize", "muon_ns_orthogonalize_noalloc", "muon_noalloc_sync_status", "muon_step",
    "muon_set_ns_config",
    "muon_set_ns_precision", "muon_autotune",
    "muon_tune_save", "muon_tune_load", "muon_last_path", "muon_sync_status",
    "muon_status_str", "muon_last_error_message", "muon_ns_flops", "muon_launch_count",
    "muon_set_kernel_timing", "muon_kernel_timing_read", "muon_debug_gemm", "muon_debug_arm_stall",
    "muon_group_create", "muon_group_step", "muon_group_destroy", "muon_group_set_host_io",
    "muon_owner_plan", "muon_adamw_step",
    "muon_pack_plan", "muon_pack",
    "muon_distill_loss", "muon_policy_loss", "muon_preference_loss",
    "muon_glu_forward", "muon_glu_backward",
)

_lib = None


class MuonError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_str(status)} ({last_error_message()})")


def lib() -> ctypes.CDLL:
    """The loaded shared library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                          "(nvcc, sm_103a); there is no CPU fallback")
    L = ctypes.CDLL(LIB_PATH)
    i64, i32, f32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_void_p
    f3 = ctypes.POINTER(ctypes.c_float)
    ip = ctypes.POINTER(ctypes.c_int)
    i64p = ctypes.POINTER(ctypes.c_int64)
    dp = ctypes.POINTER(ctypes.c_double)
    sig = {
        "muon_ns_orthogonalize": (i32, [vp, i64, i64, i64, i32, f3, i32, ip, i32, vp]),
        "muon_ns_orthogonalize_noalloc": (i32, [vp, i64, i64, i64, i32, f3, i32, ip, i32, vp]),
        "muon_noalloc_sync_status": (i32, [vp]),
        "muon_step": (i32, [ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp), i64p, i64p, i64,
                            i32, i32, f32, f32, f32, i32, vp]),
        "muon_set_ns_config": (i32, [f3, i32, ip, i32, i32]),
        "muon_autotune": (i32, [i64p, i64p, i64, i32, vp]),
        "muon_tune_save": (i32, [ctypes.c_char_p]),
        "muon_tune_load": (i32, [ctypes.c_char_p]),
        "muon_last_path": (i32, [i64, i64, i32, ip]),
        "muon_sync_status": (i32, [vp]),
        "muon_status_str": (ctypes.c_char_p, [i32]),
        "muon_last_error_message": (ctypes.c_char_p, []),
        "muon_ns_flops": (i32, [i64, i64, i32, ip, i32, dp, dp]),
        "muon_launch_count": (i64, []),
        "muon_debug_arm_stall": (i32, [i32, i32]),
        "muon_set_kernel_timing": (i32, [i32]),
        "muon_kernel_timing_read": (i32, [ctypes.c_char_p, i64p, dp, dp, i32]),
        "muon_debug_gemm": (i32, [vp, vp, vp, i64, i64, i64, i64, i32, i32, i32, i32,
                                  f32, f32, f32, f32, i32, vp]),
        "muon_group_create": (i32, [ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp), i64p, i64p, i64,
                                    i32, i32, ctypes.POINTER(vp)]),
        "muon_group_step": (i32, [vp, f32, f32, f32, i32, vp]),
        "muon_group_destroy": (i32, [vp]),
        "muon_group_set_host_io": (i32, [vp, ctypes.POINTER(vp), ctypes.POINTER(vp)]),
        "muon_owner_plan": (i32, [i64p, i64p, i64, i32, i32, ip, dp, dp, ip]),
        "muon_adamw_step": (i32, [ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp),
                                  i64p, i64, i32, i32, f32, f32, f32, f32, f32, i64, vp]),
        "muon_pack_plan": (i32, [i64p, i64p, ip, i64, i32, i64, i64p, i64p]),
        "muon_pack": (i32, [ctypes.POINTER(vp), i64p, i64p, i64p, i64, i32, vp, i32, vp]),
        "muon_distill_loss": (i32, [vp, i64, i64, i64, i32, vp, i32, vp, i32, i64, vp, vp, f32, vp, vp, i64, vp]),
        "muon_policy_loss": (i32, [vp, i64, i64, i64, i32, vp, i32, vp, vp, vp, vp, f32, f32, f32, f32, vp, vp,
                                   vp, i64, vp]),
        "muon_preference_loss": (i32, [vp, i64, i64, i64, i32, vp, i32, vp, i32, i64, vp, vp, f32, f32, f32, i32,
                                       vp, vp, vp, i64, vp]),
        "muon_glu_forward": (i32, [vp] * 6 + [i64, i64, i64, i32, i32, vp]),
        "muon_glu_backward": (i32, [vp] * 9 + [i64, i64, i64, i32, i32, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


# ---------------------------------------------------------------------------
# helpers
# ---------------------------------------------------------------------------

def status_str(status: int) -> str:
    return lib().muon_status_str(int(status)).decode()


def last_error_message() -> str:
    return lib().muon_last_error_message().decode()


def _check(status: int, what: str) -> None:
    if status != MUON_OK:
        raise MuonError(status, what)


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return MUON_F32
    if t.dtype == torch.bfloat16:
        return MUON_BF16
    if t.dtype == torch.float16:
        return MUON_F16
    raise TypeError(f"unsupported dtype {t.dtype}: float32, bfloat16 or float16")


_raw_stream = None      # (handle of a device's current stream, current device), once torch has CUDA up


def _stream_ptr(stream) -> int:
    global _raw_stream
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream[0](_raw_stream[1]())     # the handle without a Stream object around it
        import torch
        raw, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
        if raw is not None and dev is not None and torch.cuda.is_initialized():
            _raw_stream = (raw, dev)
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ints(vals):
    vals = list(vals or [])
    return (ctypes.c_int * max(1, len(vals)))(*vals), len(vals)


def _cuda_contig(t, name):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


# ---------------------------------------------------------------------------
# the entry points
# ---------------------------------------------------------------------------

def muon_ns_orthogonalize(x, coeffs=QUINTIC, steps: int = 5, segments=(2, 2, 1), stream=None):
    """In place: x (m x n or batch x m x n) <- NS(x / ||x||_F).  segments=None: plain NS."""
    _cuda_contig(x, "x")
    if x.dim() == 2:
        batch, m, n = 1, x.shape[0], x.shape[1]
    elif x.dim() == 3:
        batch, m, n = x.shape
    else:
        raise ValueError("x must be 2-D or 3-D")
    c = (ctypes.c_float * 3)(*coeffs)
    segs, nseg = _ints(segments)
    _check(lib().muon_ns_orthogonalize(x.data_ptr(), m, n, batch, _dtype_code(x), c, steps, segs, nseg,
                                       _stream_ptr(stream)), "muon_ns_orthogonalize")
    return x


def muon_ns_orthogonalize_noalloc(x, coeffs=QUINTIC, steps: int = 5, segments=(2, 2, 1), stream=None):
    """Same as muon_ns_orthogonalize, inside the library's fixed 64 MiB scratch
    array: no device memory is allocated (for callers that may not allocate)."""
    _cuda_contig(x, "x")
    if x.dim() == 2:
        batch, m, n = 1, x.shape[0], x.shape[1]
    elif x.dim() == 3:
        batch, m, n = x.shape
    else:
        raise ValueError("x must be 2-D or 3-D")
    c = (ctypes.c_float * 3)(*coeffs)
    segs, nseg = _ints(segments)
    _check(lib().muon_ns_orthogonalize_noalloc(x.data_ptr(), m, n, batch, _dtype_code(x), c, steps, segs, nseg,
                                               _stream_ptr(stream)), "muon_ns_orthogonalize_noalloc")
    return x


def muon_step(params, grads, moms, lr: float, beta: float, wd: float, nesterov: bool, stream=None):
    """One Muon step over lists of matrices (updated in place: params, moms)."""
    arr = _step_arrays(params, grads, moms)
    if arr is None:
        return
    _check(lib().muon_step(*arr, float(lr), float(beta), float(wd), 1 if nesterov else 0, _stream_ptr(stream)),
           "muon_step")


def _step_arrays(params, grads, moms):
    k = len(params)
    if not (len(grads) == k and len(moms) == k):
        raise ValueError("params, grads and moms must have the same length")
    if k == 0:
        return None
    pd = _dtype_code(params[0])
    md = _dtype_code(moms[0])
    for i in range(k):
        p, g, mo = params[i], grads[i], moms[i]
        for t, nm in ((p, "param"), (g, "grad"), (mo, "mom")):
            _cuda_contig(t, nm)
            if t.dim() != 2:
                raise ValueError(f"{nm} {i} must be 2-D")
        if p.shape != g.shape or p.shape != mo.shape:
            raise ValueError(f"shape mismatch at {i}")
        if _dtype_code(p) != pd or _dtype_code(g) != pd or _dtype_code(mo) != md:
            raise TypeError(f"dtype mismatch at {i}")
    VP = ctypes.c_void_p * k
    I64 = ctypes.c_int64 * k
    return (VP(*[p.data_ptr() for p in params]), VP(*[g.data_ptr() for g in grads]),
            VP(*[m.data_ptr() for m in moms]), I64(*[p.shape[0] for p in params]),
            I64(*[p.shape[1] for p in params]), k, pd, md)


def muon_group_create(params, grads, moms):
    """Registers a fixed set of matrices; returns an opaque group handle."""
    arr = _step_arrays(params, grads, moms)
    if arr is None:
        raise ValueError("a group needs at least one matrix")
    out = ctypes.c_void_p()
    _check(lib().muon_group_create(*arr, ctypes.byref(out)), "muon_group_create")
    return out.value


def muon_group_step(handle, lr: float, beta: float, wd: float, nesterov: bool, stream=None):
    _check(lib().muon_group_step(handle, float(lr), float(beta), float(wd), 1 if nesterov else 0,
                                 _stream_ptr(stream)), "muon_group_step")


def muon_group_destroy(handle):
    if handle:
        lib().muon_group_destroy(handle)


class MuonGroup:
    """The optimizer object of a training loop: a fixed set of (param, grad,
    momentum) CUDA tensors stepped many times.  The tensors must stay alive and
    at the same addresses for the group's lifetime (update them in place)."""

    def __init__(self, params, grads, moms):
        self._refs = (list(params), list(grads), list(moms))
        self.handle = muon_group_create(*self._refs)

    def step(self, lr: float, beta: float = 0.95, wd: float = 0.0, nesterov: bool = True, stream=None):
        muon_group_step(self.handle, lr, beta, wd, nesterov, stream)

    def set_host_io(self, host_grads=None, host_params=None):
        """Pinned CPU tensors (same shapes and dtypes as the group's gradients
        and parameters) that every step copies the gradients from and the
        updated parameters to, overlapped with the update; None turns a
        direction off."""
        k = len(self._refs[0])
        arrs = []
        for lst, nm in ((host_grads, "host_grads"), (host_params, "host_params")):
            if lst is None:
                arrs.append(None)
                continue
            lst = list(lst)
            if len(lst) != k:
                raise ValueError(f"{nm} must hold {k} tensors")
            for t, ref in zip(lst, self._refs[1] if nm == "host_grads" else self._refs[0]):
                if t.device.type != "cpu" or not t.is_contiguous() or t.shape != ref.shape or t.dtype != ref.dtype:
                    raise ValueError(f"{nm}: contiguous CPU tensors of the group's shapes and dtypes required")
            arrs.append((ctypes.c_void_p * k)(*[t.data_ptr() for t in lst]))
        self._host_refs = (host_grads, host_params)     # kept alive while the group uses them
        _check(lib().muon_group_set_host_io(self.handle, arrs[0], arrs[1]), "muon_group_set_host_io")

    def close(self):
        if self.handle:
            muon_group_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def muon_set_ns_precision(dtype: int = -1):
    """NS working precision for 16-bit parameters: -1 follows them, MUON_BF16
    or MUON_F16 forces that type."""
    _check(lib().muon_set_ns_precision(int(dtype)), "muon_set_ns_precision")


def muon_set_ns_config(coeffs=QUINTIC, steps: int = 5, segments=(2, 2, 1), path: int = MUON_PATH_AUTO):
    c = (ctypes.c_float * 3)(*coeffs) if coeffs is not None else None
    segs, nseg = _ints(segments)
    _check(lib().muon_set_ns_config(c, steps, segs, nseg, path), "muon_set_ns_config")


def muon_autotune(shapes, dtype: int = MUON_BF16, stream=None):
    shapes = list(shapes)
    k = len(shapes)
    I64 = ctypes.c_int64 * max(1, k)
    _check(lib().muon_autotune(I64(*[s[0] for s in shapes]), I64(*[s[1] for s in shapes]), k, dtype,
                               _stream_ptr(stream)), "muon_autotune")


def muon_tune_save(path: str):
    _check(lib().muon_tune_save(path.encode()), "muon_tune_save")


def muon_tune_load(path: str) -> int:
    r = lib().muon_tune_load(path.encode())
    if r < 0:
        raise MuonError(r, "muon_tune_load")
    return r


def muon_last_path(m: int, n: int, dtype: int):
    out = ctypes.c_int(-1)
    r = lib().muon_last_path(m, n, dtype, ctypes.byref(out))
    return out.value if r == MUON_OK else None


def muon_sync_status(stream=None) -> int:
    return lib().muon_sync_status(_stream_ptr(stream))


def muon_noalloc_sync_status(stream=None) -> int:
    """Status word of the allocation-free calls (read and cleared; allocates nothing)."""
    return lib().muon_noalloc_sync_status(_stream_ptr(stream))


def muon_ns_flops(m: int, n: int, path: int, segments=(2, 2, 1)):
    segs, nseg = _ints(segments)
    nom, alg = ctypes.c_double(), ctypes.c_double()
    _check(lib().muon_ns_flops(m, n, path, segs, nseg, ctypes.byref(nom), ctypes.byref(alg)), "muon_ns_flops")
    return nom.value, alg.value


def muon_launch_count() -> int:
    return lib().muon_launch_count()


#: kernels the bounded-wait test hook can stall
STALL_PRODUCT = 1
STALL_SMALL = 2


def muon_debug_arm_stall(kernel: int, stage: int = 0) -> None:
    """Test hook: the next launch of `kernel` leaves one stage unfilled, so its
    bounded wait runs out and muon_sync_status reports MUON_ETIMEOUT."""
    _check(lib().muon_debug_arm_stall(int(kernel), int(stage)), "muon_debug_arm_stall")


def muon_set_kernel_timing(enable: bool):
    lib().muon_set_kernel_timing(1 if enable else 0)


def muon_kernel_timing_read():
    """{class name: (launches, total_ms, algorithmic work)}; resets the record."""
    n = 16
    names = ctypes.create_string_buffer(32 * n)
    launches = (ctypes.c_int64 * n)()
    ms = (ctypes.c_double * n)()
    work = (ctypes.c_double * n)()
    k = lib().muon_kernel_timing_read(names, launches, ms, work, n)
    out = {}
    for i in range(k):
        nm = names.raw[32 * i:32 * i + 32].split(b"\0", 1)[0].decode()
        if launches[i]:
            out[nm] = (int(launches[i]), float(ms[i]), float(work[i]))
    return out


MUON_DEBUG_TF32 = 3
MUON_DEBUG_TF32_CHUNKED = 4


def muon_debug_gemm(A, B, C, b_kmajor=True, symmetric=False, poly=None, alpha=1.0, tile_n=0, stream=None,
                    tf32=False, tf32_chunked=False):
    """C[b] = alpha * A[b] op(B[b]) (or the fused polynomial when poly=(a, b, c)).
    tf32=True multiplies fp32 tensors on the TF32 tensor-core path;
    tf32_chunked=True does too, accumulating K in chunks summed in
    round-to-nearest fp32."""
    for t, nm in ((A, "A"), (B, "B"), (C, "C")):
        _cuda_contig(t, nm)
    batch = A.shape[0] if A.dim() == 3 else 1
    M, K = A.shape[-2], A.shape[-1]
    N = B.shape[-2] if b_kmajor else B.shape[-1]
    pa, pb, pc = poly if poly is not None else (0.0, 0.0, 0.0)
    code = MUON_DEBUG_TF32_CHUNKED if tf32_chunked else (MUON_DEBUG_TF32 if tf32 else _dtype_code(A))
    _check(lib().muon_debug_gemm(A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K, batch, code,
                                 1 if b_kmajor else 0, 1 if symmetric else 0, 1 if poly is not None else 0,
                                 float(alpha), float(pa), float(pb), float(pc), tile_n, _stream_ptr(stream)),
           "muon_debug_gemm")
    return C


def muon_owner_plan(shapes, ranks: int, dtype: int = MUON_BF16):
    """Owner rank per matrix for a multi-rank step (greedy longest-processing-
    time first on measured or modelled per-matrix costs).
    Returns (owners, per-rank loads, makespan, measured)."""
    shapes = list(shapes)
    k = len(shapes)
    I64 = ctypes.c_int64 * max(1, k)
    owners = (ctypes.c_int * max(1, k))()
    loads = (ctypes.c_double * max(1, ranks))()
    mk = ctypes.c_double()
    meas = ctypes.c_int()
    _check(lib().muon_owner_plan(I64(*[s[0] for s in shapes]), I64(*[s[1] for s in shapes]), k, dtype, ranks,
                                 owners, loads, ctypes.byref(mk), ctypes.byref(meas)), "muon_owner_plan")
    return list(owners)[:k], list(loads)[:ranks], mk.value, bool(meas.value)


def muon_pack_plan(shapes, owners, ranks: int, align_elems: int = 8):
    """Packed exchange layout: (element offset per matrix, segment length);
    rank r's owned matrices fill segment [r seg, (r+1) seg)."""
    shapes, owners = list(shapes), list(owners)
    k = len(shapes)
    if len(owners) != k:
        raise ValueError("one owner per matrix")
    I64 = ctypes.c_int64 * max(1, k)
    off = I64()
    seg = ctypes.c_int64()
    _check(lib().muon_pack_plan(I64(*[s[0] for s in shapes]), I64(*[s[1] for s in shapes]),
                                (ctypes.c_int * max(1, k))(*owners), k, int(ranks), int(align_elems), off,
                                ctypes.byref(seg)), "muon_pack_plan")
    return list(off)[:k], seg.value


def muon_pack(mats, offsets, packed, to_packed: bool = True, stream=None):
    """Copies CUDA matrices into (to_packed) or out of a packed CUDA buffer of
    the same dtype, matrix i at element offset offsets[i]."""
    k = len(mats)
    if len(offsets) != k:
        raise ValueError("one offset per matrix")
    if k == 0:
        return
    dt = _dtype_code(packed)
    _cuda_contig(packed, "packed")
    for i, t in enumerate(mats):
        _cuda_contig(t, f"matrix {i}")
        if _dtype_code(t) != dt:
            raise TypeError(f"matrix {i}: dtype differs from the packed buffer")
        if offsets[i] < 0 or offsets[i] + t.numel() > packed.numel():
            raise ValueError(f"matrix {i} does not fit the packed buffer at offset {offsets[i]}")
    shp = [(t.shape[0], t.numel() // t.shape[0]) if t.dim() >= 1 and t.shape[0] > 0 else (1, t.numel())
           for t in mats]
    VP = ctypes.c_void_p * k
    I64 = ctypes.c_int64 * k
    _check(lib().muon_pack(VP(*[t.data_ptr() for t in mats]), I64(*[s[0] for s in shp]), I64(*[s[1] for s in shp]),
                           I64(*offsets), k, dt, packed.data_ptr(), 1 if to_packed else 0, _stream_ptr(stream)),
           "muon_pack")


def muon_adamw_step(params, grads, exp_avgs, exp_avg_sqs, lr: float, beta1: float = 0.9, beta2: float = 0.999,
                    eps: float = 1e-8, wd: float = 0.0, step: int = 1, stream=None):
    """AdamW over lists of CUDA tensors of any shape (params, moments in place)."""
    k = len(params)
    if not (len(grads) == k and len(exp_avgs) == k and len(exp_avg_sqs) == k):
        raise ValueError("tensor lists must have the same length")
    if k == 0:
        return
    pd, sd = _dtype_code(params[0]), _dtype_code(exp_avgs[0])
    for i in range(k):
        for t, nm, dt in ((params[i], "param", pd), (grads[i], "grad", pd), (exp_avgs[i], "exp_avg", sd),
                          (exp_avg_sqs[i], "exp_avg_sq", sd)):
            _cuda_contig(t, nm)
            if _dtype_code(t) != dt or t.numel() != params[i].numel():
                raise TypeError(f"{nm} {i}: dtype or size mismatch")
    VP = ctypes.c_void_p * k
    _check(lib().muon_adamw_step(VP(*[t.data_ptr() for t in params]), VP(*[t.data_ptr() for t in grads]),
                                 VP(*[t.data_ptr() for t in exp_avgs]), VP(*[t.data_ptr() for t in exp_avg_sqs]),
                                 (ctypes.c_int64 * k)(*[t.numel() for t in params]), k, pd, sd, float(lr),
                                 float(beta1), float(beta2), float(eps), float(wd), int(step),
                                 _stream_ptr(stream)), "muon_adamw_step")


# ---------------------------------------------------------------------------
# losses over the vocabulary, with their gradients
# ---------------------------------------------------------------------------
#
# These calls and the feed-forward block's stand outside autograd: their results
# carry no graph, whatever their inputs require, and the caller passes the
# gradients on (logits.backward(grad)).  A tensor that the caller gives to be
# written counts as changed in place.


def _written(t) -> None:
    """Moves the version of a tensor that a call has written, so that a backward pass that saved its old values says so."""
    import torch
    if not t.is_inference():
        torch.autograd.graph.increment_version(t)


def _on_stream(stream):
    """Context in which new tensors belong to `stream` (None: the current one)."""
    import contextlib

    import torch
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def _index_code(t, name) -> int:
    import torch
    d = t.dtype
    if d is torch.int64:
        return MUON_I64
    if d is torch.int32:
        return MUON_I32
    raise TypeError(f"{name}: int32 or int64 required, got {d}")


def _rows_of(t, name):
    """(pointer, row pitch) of a rows x cols CUDA tensor whose rows are contiguous."""
    if not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA tensor with contiguous rows")
    rows, cols = t.shape
    if t.is_contiguous():
        return t.data_ptr(), cols or 1
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D CUDA tensor with contiguous rows")
    pitch = t.stride(0) if rows > 1 else max(1, cols)
    if pitch < cols:
        raise ValueError(f"{name}: rows overlap")
    return t.data_ptr(), max(pitch, 1)


def _vector(t, n, name, dtype=None):
    """Pointer of a contiguous CUDA tensor of n elements; None stays NULL."""
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if t.numel() != n:
        raise ValueError(f"{name}: {n} elements required, got {t.numel()}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name}: {dtype} required, got {t.dtype}")
    return t.data_ptr()


def _loss_outputs(logits, grad, stream, *sizes):
    """The gradient (a new tensor unless one was given), its pointer and pitch, and fp32 vectors of the given sizes."""
    import torch
    if stream is not None:
        with _on_stream(stream):
            return _loss_outputs(logits, grad, None, *sizes)
    dev, f32, empty = logits.device, torch.float32, torch.empty
    if grad is None:
        shape = logits.shape
        grad = empty(shape, dtype=logits.dtype, device=dev)
        gp, ldg = grad.data_ptr(), shape[1] or 1
    elif grad.shape != logits.shape or grad.dtype is not logits.dtype:
        raise ValueError("grad must have the logits' shape and dtype")
    else:
        gp, ldg = _rows_of(grad, "grad")
        _written(grad)
    return (grad, gp, ldg, *[empty(n, dtype=f32, device=dev) for n in sizes])


def muon_distill_loss(logits, teacher_idx, teacher_logits, teacher_lse=None, weights=None, temperature: float = 1.0,
                      grad=None, stream=None):
    """Distillation from a teacher's top logits: teacher_idx (int32 or int64)
    and teacher_logits, both rows x k; teacher_lse (rows, fp32) keeps the
    teacher's remaining mass as one more class, None renormalises over the k.
    Returns (loss per row, gradient of the loss' sum); grad may be a tensor to
    write into, the logits themselves included."""
    import torch
    f32 = torch.float32
    lp, ld = _rows_of(logits, "logits")
    rows, vocab = logits.shape
    if teacher_idx.dim() != 2 or teacher_idx.shape != teacher_logits.shape or teacher_idx.shape[0] != rows:
        raise ValueError("teacher_idx and teacher_logits must be rows x k")
    k = teacher_idx.shape[1]
    args = (lp, ld, rows, vocab, _dtype_code(logits), _vector(teacher_idx, rows * k, "teacher_idx"),
            _index_code(teacher_idx, "teacher_idx"), _vector(teacher_logits, rows * k, "teacher_logits"),
            _dtype_code(teacher_logits), k, _vector(teacher_lse, rows, "teacher_lse", f32),
            _vector(weights, rows, "weights", f32), temperature)
    grad, gp, ldg, loss = _loss_outputs(logits, grad, stream, rows)
    st = lib().muon_distill_loss(*args, loss.data_ptr(), gp, ldg, _stream_ptr(stream))
    if st:
        _check(st, "muon_distill_loss")
    return loss, grad


def muon_policy_loss(logits, tokens, advantages, old_logp=None, ref_logp=None, weights=None,
                     temperature: float = 1.0, clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0,
                     grad=None, stream=None):
    """Clipped policy loss with a KL term towards ref_logp, one sampled token
    per row.  Returns (loss per row, log-probability per row, gradient of the
    loss' sum)."""
    import torch
    f32 = torch.float32
    lp, ld = _rows_of(logits, "logits")
    rows, vocab = logits.shape
    args = (lp, ld, rows, vocab, _dtype_code(logits), _vector(tokens, rows, "tokens"), _index_code(tokens, "tokens"),
            _vector(advantages, rows, "advantages", f32), _vector(old_logp, rows, "old_logp", f32),
            _vector(ref_logp, rows, "ref_logp", f32), _vector(weights, rows, "weights", f32), temperature, clip_low,
            clip_high, kl_coef)
    grad, gp, ldg, loss, logp = _loss_outputs(logits, grad, stream, rows, rows)
    st = lib().muon_policy_loss(*args, loss.data_ptr(), logp.data_ptr(), gp, ldg, _stream_ptr(stream))
    if st:
        _check(st, "muon_policy_loss")
    return loss, logp, grad


def muon_preference_loss(logits, tokens, seq_bounds, ref_logp=None, weights=None, beta: float = 0.1,
                         margin: float = 0.0, label_smoothing: float = 0.0, average: bool = False, grad=None,
                         stream=None):
    """Preference loss of paired sequences packed along the rows: seq_bounds
    (2 pairs + 1 offsets, int32 or int64, on the device) alternates chosen and
    rejected; tokens are labels, negative ones left out.  Returns (loss per
    pair, sequence log-probabilities, gradient of the loss' sum)."""
    import torch
    f32 = torch.float32
    lp, ld = _rows_of(logits, "logits")
    rows, vocab = logits.shape
    nb = seq_bounds.numel()
    if nb % 2 != 1:
        raise ValueError("seq_bounds needs 2 pairs + 1 offsets")
    pairs = nb // 2
    args = (lp, ld, rows, vocab, _dtype_code(logits), _vector(tokens, rows, "tokens"), _index_code(tokens, "tokens"),
            _vector(seq_bounds, nb, "seq_bounds"), _index_code(seq_bounds, "seq_bounds"), pairs,
            _vector(ref_logp, 2 * pairs, "ref_logp", f32), _vector(weights, pairs, "weights", f32), beta, margin,
            label_smoothing, 1 if average else 0)
    grad, gp, ldg, loss, seq = _loss_outputs(logits, grad, stream, pairs, 2 * pairs)
    st = lib().muon_preference_loss(*args, loss.data_ptr(), seq.data_ptr(), gp, ldg, _stream_ptr(stream))
    if st:
        _check(st, "muon_preference_loss")
    return loss, seq, grad


# ---------------------------------------------------------------------------
# gated feed-forward block
# ---------------------------------------------------------------------------

#: activations of the gated feed-forward block
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}


def _glu_args(x, w_gate, w_up, act):
    dt = x.dtype
    if not (x.is_cuda and w_gate.is_cuda and w_up.is_cuda and x.is_contiguous() and w_gate.is_contiguous()
            and w_up.is_contiguous() and x.dim() == 2 and w_gate.dim() == 2 and w_up.dim() == 2
            and w_gate.dtype is dt and w_up.dtype is dt):
        for t, nm in ((x, "x"), (w_gate, "w_gate"), (w_up, "w_up")):
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{nm} must be a contiguous CUDA tensor")
            if t.dim() != 2:
                raise ValueError(f"{nm} must be 2-D")
            if t.dtype is not dt:
                raise TypeError(f"{nm}: dtype differs from x")
    tokens, hidden = x.shape
    shape = w_gate.shape
    if shape[1] != hidden or w_up.shape != shape:
        raise ValueError("x is tokens x hidden, w_gate and w_up ffn x hidden")
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"act {act!r}: one of {sorted(ACTIVATIONS)}")
    return tokens, hidden, shape[0], _dtype_code(x), code


def _new(stream, *like):
    """New contiguous tensors of the (shape, tensor to take dtype and device from) pairs given."""
    import torch
    if stream is not None:
        with _on_stream(stream):
            return _new(None, *like)
    return [torch.empty(shape, dtype=t.dtype, device=t.device) for shape, t in like]


def muon_glu_forward(x, w_gate, w_up, act: str = "silu", save: bool = True, stream=None):
    """act(x w_gate^T) * (x w_up^T) in one kernel (bf16 or fp16; x tokens x
    hidden, weights ffn x hidden).  Returns (h, gate, up) for the backward
    pass, or h alone with save=False."""
    tokens, hidden, ffn, dt, code = _glu_args(x, w_gate, w_up, act)
    out = _new(stream, *[((tokens, ffn), x)] * (3 if save else 1))
    ptrs = [t.data_ptr() for t in out] if save else (out[0].data_ptr(), None, None)
    st = lib().muon_glu_forward(x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), *ptrs, tokens, hidden, ffn, dt, code,
                                _stream_ptr(stream))
    if st:
        _check(st, "muon_glu_forward")
    return tuple(out) if save else out[0]


def muon_glu_backward(x, w_gate, w_up, gate, up, dh, act: str = "silu", need_dx: bool = True, dw_gate=None, dw_up=None,
                      stream=None):
    """Gradients (dx, dw_gate, dw_up) of muon_glu_forward from dh and the gate
    and up it returned.  dw_gate and dw_up may be tensors to write into (the
    gradients a MuonGroup reads); need_dx=False leaves dx out (None)."""
    tokens, hidden, ffn, dt, code = _glu_args(x, w_gate, w_up, act)
    for t, nm in ((gate, "gate"), (up, "up"), (dh, "dh")):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{nm} must be a contiguous CUDA tensor")
        if t.shape != (tokens, ffn) or t.dtype is not x.dtype:
            raise ValueError(f"{nm} must be tokens x ffn of x's dtype")
    for t, nm in ((dw_gate, "dw_gate"), (dw_up, "dw_up")):
        if t is not None:
            _cuda_contig(t, nm)
            if t.shape != w_gate.shape or t.dtype is not x.dtype:
                raise ValueError(f"{nm} must be ffn x hidden of x's dtype")
    want = ([((tokens, hidden), x)] if need_dx else []) + [((ffn, hidden), x)] * ((dw_gate is None) + (dw_up is None))
    new = _new(stream, *want)
    for t in (dw_gate, dw_up):
        if t is not None:
            _written(t)
    dx = new.pop(0) if need_dx else None
    dw_gate = new.pop(0) if dw_gate is None else dw_gate
    dw_up = new.pop(0) if dw_up is None else dw_up
    st = lib().muon_glu_backward(x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), gate.data_ptr(), up.data_ptr(),
                                 dh.data_ptr(), dx.data_ptr() if need_dx else None, dw_gate.data_ptr(),
                                 dw_up.data_ptr(), tokens, hidden, ffn, dt, code, _stream_ptr(stream))
    if st:
        _check(st, "muon_glu_backward")
    return dx, dw_gate, dw_up
