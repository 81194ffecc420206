"""Thin Python binding of liblaplex.so (argument marshalling only).

Every function here checks tensor dtypes/devices/shapes, allocates outputs and
workspace with torch (device memory is the only thing torch provides), and calls
the C ABI of include/laplex.h with raw pointers and the current CUDA stream.
All arithmetic runs in the library's CUDA kernels; there is no CPU path and no
fallback: a missing or unloadable library raises ``LaplexError``.

Host (CPU) tensors are accepted by the ``*_host`` helpers, which copy inputs to
the device, call the same entry point and copy the result back (the end-to-end
path a user without device buffers takes).

Calls may come from several host threads, on one stream or on several: each
enqueues its kernels as a whole.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblaplex.so")

OK, EINVAL, ENONFINITE, EWORKSPACE, ECUDA, ETIMEOUT = range(6)
BUILD_ACCURATE_EXP = 1  # laplex_build_flags() bit
F32, F64, F16, BF16 = range(4)
(OP_SORT, OP_SYM, OP_GENERAL, OP_PHASED, OP_GRAM, OP_BACKWARD, OP_BACKWARD_GENERAL, OP_GRAM_MATRIX,
 OP_BACKWARD_PHASED, OP_PERMUTE, OP_SYM_PLANNED, OP_SORT_CARRY, OP_SYM_UNSORTED) = range(13)

LINATTN_FORWARD, LINATTN_BACKWARD, LINATTN_BACKWARD_DECAY = range(3)

_lib = None
_lock = threading.Lock()
_P = ctypes.c_void_p
_I64 = ctypes.c_int64


class LaplexError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


_STATUS_NAMES = {OK: "LAPLEX_OK", EINVAL: "LAPLEX_EINVAL", ENONFINITE: "LAPLEX_ENONFINITE",
                 EWORKSPACE: "LAPLEX_EWORKSPACE", ECUDA: "LAPLEX_ECUDA",
                 ETIMEOUT: "LAPLEX_ETIMEOUT"}


class _Rows(ctypes.Structure):
    """laplex_rows"""
    _fields_ = [("ptr", _P), ("token_stride", _I64), ("head_stride", _I64)]


class _LinattnShape(ctypes.Structure):
    """laplex_linattn_shape"""
    _fields_ = [("tokens", _I64), ("seqs", _I64), ("cu_seqlens", _P), ("hq", ctypes.c_int32), ("hkv", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("log_decay", _P), ("scale", ctypes.c_double),
                ("dtype", ctypes.c_int)]


_R = ctypes.POINTER(_Rows)
_S = ctypes.POINTER(_LinattnShape)

#: every symbol include/laplex.h declares, with its ctypes signature
SIGNATURES = {
    "laplex_version": ([], ctypes.c_int),
    "laplex_build_flags": ([], ctypes.c_int),
    "laplex_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "laplex_last_error": ([], ctypes.c_char_p),
    "laplex_workspace_size": ([ctypes.c_int, _I64, _I64, _I64, ctypes.c_int,
                               ctypes.POINTER(ctypes.c_size_t)], ctypes.c_int),
    "laplex_workspace_init": ([_P, ctypes.c_size_t, _P], ctypes.c_int),
    "laplex_get_device_status": ([_P, _P], ctypes.c_int),
    "laplex_sort_anchors": ([_P, _I64, ctypes.c_int, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "laplex_matvec_sym": ([_P, _P, _I64, _P, _P, _I64, ctypes.c_int, _P, ctypes.c_size_t, _P],
                          ctypes.c_int),
    "laplex_matvec_general": ([_P, _P, _I64, _P, _P, _I64, _P, _P, _I64, ctypes.c_int,
                               ctypes.c_int, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "laplex_matvec_phased": ([_P, _P, _P, _I64, _P, _P, _P, _I64, _P, _P, _I64, ctypes.c_int,
                              ctypes.c_int, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "laplex_gram": ([_P, _P, _P, _I64, _P, _P, _P, _I64, _P, _P, _P, _I64, ctypes.c_int, _P,
                     ctypes.c_size_t, _P], ctypes.c_int),
    "laplex_backward": ([_P, _P, _I64, _P, _P, _P, _P, ctypes.c_int, _P, ctypes.c_size_t, _P],
                        ctypes.c_int),
    "laplex_backward_general": ([_P, _P, _I64, _P, _P, _I64, _P, _P, _P, _P, _P, ctypes.c_int, _P,
                                 ctypes.c_size_t, _P], ctypes.c_int),
    "laplex_backward_phased": ([_P, _P, _P, _I64, _P, _P, _P, _I64, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int,
                                _P, ctypes.c_size_t, _P], ctypes.c_int),
    "laplex_gram_matrix": ([_P, _P, _I64, _P, _P, _I64, _P, _P, _I64, ctypes.c_int, _P, ctypes.c_size_t, _P],
                           ctypes.c_int),
    "laplex_matvec_sym_noalloc": ([_P, _P, _I64, _P, _P, _P], ctypes.c_int),
    "laplex_set_profile_events": ([_P, _P], ctypes.c_int),
    "laplex_set_status_word": ([_P], ctypes.c_int),
    "laplex_test_set_sort_wait": ([ctypes.c_uint32, ctypes.c_int], ctypes.c_int),
    "laplex_permute": ([_P, _P, _I64, ctypes.c_int, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "laplex_invert_perm": ([_P, _I64, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "laplex_matvec_sym_planned": ([_P, _P, _P, _I64, _P, _P, ctypes.c_int, _P, ctypes.c_size_t, _P],
                                  ctypes.c_int),
    "laplex_sort_anchors_carry": ([_P, _P, _I64, ctypes.c_int, _P, _P, _P, _P, ctypes.c_size_t, _P],
                                  ctypes.c_int),
    "laplex_matvec_sym_unsorted": ([_P, _P, _I64, ctypes.c_int, _P, _P, _P, _P, ctypes.c_size_t, _P],
                                   ctypes.c_int),
    "laplex_linattn_workspace_size": ([_S, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)], ctypes.c_int),
    "laplex_linattn": ([_S, _R, _R, _R, _P, _R, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "laplex_linattn_backward": ([_S, _R, _R, _R, _R, _P, _P, _R, _R, _R, _P, _P, _P, ctypes.c_size_t, _P],
                                ctypes.c_int),
    "laplex_test_set_linattn_wait": ([ctypes.c_uint32, ctypes.c_int], ctypes.c_int),
    "laplex_linattn_step": ([_S, _R, _R, _R, _P, _I64, _P, _R, _P], ctypes.c_int),
    "laplex_embed": ([_P, _I64, _I64, _I64, _P, ctypes.c_int, _I64, ctypes.c_double, _P, _I64, ctypes.c_int, _P],
                     ctypes.c_int),
    "laplex_embed_backward_workspace_size": ([_I64, _I64, _I64, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)],
                                             ctypes.c_int),
    "laplex_embed_backward": ([_P, ctypes.c_int, _I64, _P, _I64, _I64, _I64, ctypes.c_double, ctypes.c_int, _P, _I64,
                               ctypes.c_int, ctypes.c_int, _P, ctypes.c_size_t, _P], ctypes.c_int),
}


def lib():
    """The loaded library (raises LaplexError if it cannot be loaded)."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise LaplexError(ECUDA, f"{LIB_PATH} is missing: build it with "
                                             "`python -m exact_laplace_b200.build` (nvcc, sm_100a)")
                try:
                    L = ctypes.CDLL(LIB_PATH)
                except OSError as e:
                    raise LaplexError(ECUDA, f"cannot load {LIB_PATH}: {e}") from e
                for name, (args, res) in SIGNATURES.items():
                    f = getattr(L, name)
                    f.argtypes = args
                    f.restype = res
                _lib = L
    return _lib


def _check(status: int):
    if status != OK:
        raise LaplexError(status, lib().laplex_last_error().decode())


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.float64:
        return F64
    raise LaplexError(EINVAL, f"dtype {t.dtype} is not float32/float64")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dev(*ts):
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise LaplexError(EINVAL, "tensors must be on a CUDA device (use the *_host helpers "
                                      "for host buffers)")
        if not t.is_contiguous():
            raise LaplexError(EINVAL, "tensors must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise LaplexError(EINVAL, "tensors are on different devices")
    return dev


def _perm(p):
    if p is not None and p.dtype != torch.int32:
        raise LaplexError(EINVAL, "perm must be int32")
    return p


#: held from the workspace's lookup until the call has enqueued its last kernel.  Host threads that share a
#: stream share its workspace, and the library gives up the interpreter's lock: without this one a call's
#: kernels could land between the passes of another's.  (One lock for all streams: what it holds up is the
#: launches alone, some 10 us, while the rest of a call is under the interpreter's lock anyway.)
class _Enqueue:
    def __init__(self):
        self._lock = threading.RLock()
        self._elsewhere = False  # this call reports to a word of its own

    def __enter__(self):
        self._lock.acquire()

    def report_to(self, word):
        _check(lib().laplex_set_status_word(word.data_ptr()))
        self._elsewhere = True

    def __exit__(self, *exc):
        if self._elsewhere:
            self._elsewhere = False
            lib().laplex_set_status_word(None)
        self._lock.release()


_enqueue = _Enqueue()


def _serial(call):
    @functools.wraps(call)
    def locked(*args, **kwargs):
        with _enqueue:
            return call(*args, **kwargs)
    return locked


class Workspace:
    """Device workspace cache (one growing buffer per device and stream).

    The header is zeroed when a stream's first buffer is allocated, and goes along
    into a larger one; the library keeps its sticky status word there.  Calls
    captured into a graph in memory of the graph's own share one word per device.
    ``status()`` synchronises and reports both."""

    _cache: dict = {}
    _words: dict = {}

    @classmethod
    def get(cls, device, nbytes: int) -> "torch.Tensor":
        key = (device, torch.cuda.current_stream(device).cuda_stream)
        old = cls._cache.get(key)
        if old is not None and old.numel() >= nbytes:
            return old
        buf = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
        if old is not None and not torch.cuda.is_current_stream_capturing():
            buf[:256].copy_(old[:256])  # the status of the calls before, in the stream's order
        cls._cache[key] = buf
        return buf

    @classmethod
    def captured_word(cls, device) -> "torch.Tensor":
        """The status word of captured calls, while one is captured."""
        word = cls._words.get(device)
        if word is None:
            word = torch.empty(64, dtype=torch.int32, device=device)
            side = torch.cuda.Stream(device)  # (a memset inside the graph would run at every replay)
            while _capturing(side):
                side = torch.cuda.Stream(device)
            _check(lib().laplex_workspace_init(word.data_ptr(), 256, side.cuda_stream))
            cls._words[device] = word
        return word

    @classmethod
    def status(cls, device=None) -> None:
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        key = (device, torch.cuda.current_stream(device).cuda_stream)
        buf = cls._cache.get(key)
        if buf is not None:
            _check(lib().laplex_get_device_status(_ptr(buf), _stream(device)))
        word = cls._words.get(device)
        if word is not None:
            torch.cuda.synchronize(device)  # (replays may be on any stream)
            _check(lib().laplex_get_device_status(_ptr(word), _stream(device)))


def _capturing(stream) -> bool:
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def workspace_size(op: int, n: int, k: int = 0, B: int = 1, dtype=torch.float32) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().laplex_workspace_size(op, n, k, B, F64 if dtype == torch.float64 else F32,
                                       ctypes.byref(out)))
    return out.value


def _ws(op, n, k, B, dtype, device):
    nb = workspace_size(op, n, k, B, dtype)
    buf = Workspace.get(device, nb)
    return buf, buf.numel()


def set_profile_events(before=None, after=None) -> None:
    """Record two torch.cuda.Event objects around the dominant kernel of the
    following calls on this thread (both recorded once first, so that their CUDA
    events exist); None, None switches it off."""
    h = [None if e is None else ctypes.c_void_p(e.cuda_event) for e in (before, after)]
    _check(lib().laplex_set_profile_events(h[0], h[1]))


def test_set_sort_wait(polls: int = 0, force_expiry: bool = False) -> None:
    """Test hook: bound of the sort's look-back waits on this thread (0: the
    default) and whether every wait is made to run to that bound."""
    _check(lib().laplex_test_set_sort_wait(polls, 1 if force_expiry else 0))


def test_set_linattn_wait(polls: int = 0, force_expiry: bool = False) -> None:
    """Test hook: bound of the waits in linattn's and linattn_backward's kernels of
    16-bit rows on this thread (0: the default) and whether they are made to run out."""
    _check(lib().laplex_test_set_linattn_wait(polls, 1 if force_expiry else 0))


def device_status(device=None) -> None:
    """Synchronise and raise if a kernel recorded a device-side error: in a call on
    the current stream, or in a captured call of a sequence operator on any stream."""
    Workspace.status(device)


# ----------------------------------------------------------------------------- calls

@_serial
def sort_anchors(a: torch.Tensor, sorted_out=None, perm_out=None):
    """(sorted, perm): the anchors ascending and the int32 permutation, ties by index."""
    dev = _dev(a, sorted_out, perm_out)
    n = a.numel()
    s = torch.empty_like(a) if sorted_out is None else sorted_out
    p = torch.empty(n, dtype=torch.int32, device=dev) if perm_out is None else perm_out
    ws, nb = _ws(OP_SORT, n, 0, 1, a.dtype, dev)
    _check(lib().laplex_sort_anchors(_ptr(a), n, _dt(a), _ptr(s), _ptr(p), _ptr(ws), nb,
                                     _stream(dev)))
    return s, p


@_serial
def sort_anchors_carry(a: torch.Tensor, x: torch.Tensor, sorted_out=None, perm_out=None, xs_out=None):
    """(sorted, perm, xs): the sort of laplex_sort_anchors with x carried along,
    xs[r] = x[perm[r]]."""
    dev = _dev(a, x, sorted_out, perm_out, xs_out)
    n = a.numel()
    if x.numel() != n or x.dtype != a.dtype:
        raise LaplexError(EINVAL, "x must have n elements and the anchors' dtype")
    s = torch.empty_like(a) if sorted_out is None else sorted_out
    p = torch.empty(n, dtype=torch.int32, device=dev) if perm_out is None else perm_out
    xs = torch.empty_like(x) if xs_out is None else xs_out
    ws, nb = _ws(OP_SORT_CARRY, n, 0, 1, a.dtype, dev)
    _check(lib().laplex_sort_anchors_carry(_ptr(a), _ptr(x), n, _dt(a), _ptr(s), _ptr(p), _ptr(xs), _ptr(ws), nb,
                                           _stream(dev)))
    return s, p, xs


@_serial
def matvec_sym_unsorted(a: torch.Tensor, x: torch.Tensor, out=None, sorted_out=None, perm_out=None):
    """(y, sorted, perm): y = K x on anchors and x in the caller's order (one
    column), in one call: the sort carrying x, the product, y back to caller order."""
    dev = _dev(a, x, out, sorted_out, perm_out)
    n = a.numel()
    if x.numel() != n or x.dtype != a.dtype:
        raise LaplexError(EINVAL, "x must have n elements and the anchors' dtype")
    y = torch.empty_like(x) if out is None else out
    s = torch.empty_like(a) if sorted_out is None else sorted_out
    p = torch.empty(n, dtype=torch.int32, device=dev) if perm_out is None else perm_out
    ws, nb = _ws(OP_SYM_UNSORTED, n, 0, 1, a.dtype, dev)
    _check(lib().laplex_matvec_sym_unsorted(_ptr(a), _ptr(x), n, _dt(a), _ptr(y), _ptr(s), _ptr(p), _ptr(ws), nb,
                                            _stream(dev)))
    return y, s, p


@_serial
def matvec_sym(sorted_anchors: torch.Tensor, x: torch.Tensor, perm=None, out=None):
    """y = K x for K_ij = exp(-|a_i - a_j|) given the sorted anchors (and perm, if x is
    in the caller's order).  x: [n] or [n, B]."""
    dev = _dev(sorted_anchors, x, _perm(perm), out)
    n = sorted_anchors.numel()
    B = 1 if x.dim() == 1 else x.shape[1]
    if x.shape[0] != n or x.dtype != sorted_anchors.dtype:
        raise LaplexError(EINVAL, "x must have n rows and the anchors' dtype")
    y = torch.empty_like(x) if out is None else out
    ws, nb = _ws(OP_SYM, n, 0, B, x.dtype, dev)
    _check(lib().laplex_matvec_sym(_ptr(sorted_anchors), _ptr(perm), n, _ptr(x), _ptr(y), B,
                                   _dt(x), _ptr(ws), nb, _stream(dev)))
    return y


@_serial
def permute(src: torch.Tensor, idx: torch.Tensor, out=None):
    """dst[idx[i]] = src[i] (4- or 8-byte elements, moved as bits); idx int32."""
    dev = _dev(src, _perm(idx), out)
    n = src.numel()
    if idx.numel() != n or src.element_size() not in (4, 8):
        raise LaplexError(EINVAL, "src and idx must have n elements; src of 4 or 8 bytes")
    dst = torch.empty_like(src) if out is None else out
    dt = F64 if src.element_size() == 8 else F32
    ws, nb = _ws(OP_PERMUTE, n, 0, 1, torch.float64 if dt == F64 else torch.float32, dev)
    _check(lib().laplex_permute(_ptr(src), _ptr(idx), n, dt, _ptr(dst), _ptr(ws), nb, _stream(dev)))
    return dst


@_serial
def invert_perm(perm: torch.Tensor, out=None):
    """inv with inv[perm[r]] = r (int32)."""
    dev = _dev(_perm(perm), out)
    n = perm.numel()
    inv = torch.empty_like(perm) if out is None else out
    ws, nb = _ws(OP_PERMUTE, n, 0, 1, torch.float32, dev)
    _check(lib().laplex_invert_perm(_ptr(perm), n, _ptr(inv), _ptr(ws), nb, _stream(dev)))
    return inv


def matvec_sym_noalloc(sorted_anchors: torch.Tensor, x: torch.Tensor, perm=None, out=None):
    """laplex_matvec_sym_noalloc: y = K x (fp32, one column) with the library's
    fixed device scratch instead of a workspace (n <= 2^30)."""
    dev = _dev(sorted_anchors, x, _perm(perm), out)
    n = sorted_anchors.numel()
    if x.numel() != n or x.dtype != torch.float32 or sorted_anchors.dtype != torch.float32:
        raise LaplexError(EINVAL, "fp32 anchors and x with n elements")
    y = torch.empty_like(x) if out is None else out
    _check(lib().laplex_matvec_sym_noalloc(_ptr(sorted_anchors), _ptr(perm), n, _ptr(x), _ptr(y), _stream(dev)))
    return y


@_serial
def matvec_sym_planned(sorted_anchors: torch.Tensor, perm: torch.Tensor, inv: torch.Tensor, x: torch.Tensor,
                       out=None):
    """y = K x for x, y in the caller's order (one column), through the plan
    (sorted, perm, inv): bucketed moves into and out of sorted order."""
    dev = _dev(sorted_anchors, _perm(perm), _perm(inv), x, out)
    n = sorted_anchors.numel()
    if x.numel() != n or x.dtype != sorted_anchors.dtype:
        raise LaplexError(EINVAL, "x must have n elements and the anchors' dtype")
    y = torch.empty_like(x) if out is None else out
    ws, nb = _ws(OP_SYM_PLANNED, n, 0, 1, x.dtype, dev)
    _check(lib().laplex_matvec_sym_planned(_ptr(sorted_anchors), _ptr(perm), _ptr(inv), n, _ptr(x), _ptr(y),
                                           _dt(x), _ptr(ws), nb, _stream(dev)))
    return y


@_serial
def matvec_general(sa, sb, x, pa=None, pb=None, transpose=False, out=None):
    """y = K x (x on the b side) or, with transpose, y = K^T x (x on the a side)."""
    dev = _dev(sa, sb, x, _perm(pa), _perm(pb), out)
    n, k = sa.numel(), sb.numel()
    B = 1 if x.dim() == 1 else x.shape[1]
    nin, nout = (n, k) if transpose else (k, n)
    if x.shape[0] != nin:
        raise LaplexError(EINVAL, f"x must have {nin} rows")
    y = torch.empty((nout,) + tuple(x.shape[1:]), dtype=x.dtype, device=dev) if out is None else out
    ws, nb = _ws(OP_GENERAL, n, k, B, x.dtype, dev)
    _check(lib().laplex_matvec_general(_ptr(sa), _ptr(pa), n, _ptr(sb), _ptr(pb), k, _ptr(x),
                                       _ptr(y), B, int(bool(transpose)), _dt(x), _ptr(ws), nb,
                                       _stream(dev)))
    return y


@_serial
def matvec_phased(sa, phi, x, pa=None, sb=None, psi=None, pb=None, transpose=False, out=None):
    """Phased product, K_ij = exp(-|a_i - b_j|) cos(phi_i - psi_j); sb=None: b = a."""
    dev = _dev(sa, phi, x, _perm(pa), sb, psi, _perm(pb), out)
    n = sa.numel()
    k = 0 if sb is None else sb.numel()
    B = 1 if x.dim() == 1 else x.shape[1]
    nout = n if sb is None else (k if transpose else n)
    y = torch.empty((nout,) + tuple(x.shape[1:]), dtype=x.dtype, device=dev) if out is None else out
    ws, nb = _ws(OP_PHASED, n, k, B, x.dtype, dev)
    _check(lib().laplex_matvec_phased(_ptr(sa), _ptr(pa), _ptr(phi), n, _ptr(sb), _ptr(pb),
                                      _ptr(psi), k, _ptr(x), _ptr(y), B, int(bool(transpose)),
                                      _dt(x), _ptr(ws), nb, _stream(dev)))
    return y


@_serial
def gram(sa, v, pa=None, phi=None, D=None, sb=None, pb=None, psi=None, out=None):
    """z = K^T diag(D) K v (D = 1 when None); sb=None: symmetric K."""
    dev = _dev(sa, v, _perm(pa), phi, D, sb, _perm(pb), psi, out)
    n = sa.numel()
    k = 0 if sb is None else sb.numel()
    B = 1 if v.dim() == 1 else v.shape[1]
    z = torch.empty_like(v) if out is None else out
    ws, nb = _ws(OP_GRAM, n, k, B, v.dtype, dev)
    _check(lib().laplex_gram(_ptr(sa), _ptr(pa), _ptr(phi), n, _ptr(sb), _ptr(pb), _ptr(psi), k,
                             _ptr(D), _ptr(v), _ptr(z), B, _dt(v), _ptr(ws), nb, _stream(dev)))
    return z


@_serial
def backward(sorted_anchors, x, g, perm=None, dx_out=None, da_out=None):
    """(dx, da) of L = <g, K x>: dx = K g, da = dL/da (sign(0) = 0 at ties)."""
    dev = _dev(sorted_anchors, x, g, _perm(perm), dx_out, da_out)
    n = sorted_anchors.numel()
    dx = torch.empty_like(x) if dx_out is None else dx_out
    da = torch.empty_like(x) if da_out is None else da_out
    ws, nb = _ws(OP_BACKWARD, n, 0, 1, x.dtype, dev)
    _check(lib().laplex_backward(_ptr(sorted_anchors), _ptr(perm), n, _ptr(x), _ptr(g), _ptr(dx),
                                 _ptr(da), _dt(x), _ptr(ws), nb, _stream(dev)))
    return dx, da


@_serial
def backward_general(sa, sb, x, g, pa=None, pb=None):
    """(dx, da, db) of L = <g, K x>, K_ij = exp(-|a_i - b_j|): dx = K^T g and the
    anchor gradients (sign(0) = 0 at ties).  g, da follow pa; x, dx, db follow pb."""
    dev = _dev(sa, sb, x, g, _perm(pa), _perm(pb))
    n, k = sa.numel(), sb.numel()
    dx = torch.empty_like(x)
    da = torch.empty_like(g)
    db = torch.empty_like(x)
    ws, nb = _ws(OP_BACKWARD_GENERAL, n, k, 1, x.dtype, dev)
    _check(lib().laplex_backward_general(_ptr(sa), _ptr(pa), n, _ptr(sb), _ptr(pb), k, _ptr(x), _ptr(g),
                                         _ptr(dx), _ptr(da), _ptr(db), _dt(x), _ptr(ws), nb,
                                         _stream(dev)))
    return dx, da, db


@_serial
def backward_phased(sa, phi, x, g, pa=None, sb=None, psi=None, pb=None):
    """Gradients of L = <g, K x>, K_ij = exp(-|a_i - b_j|) cos(phi_i - psi_j).

    sb given: (dx, dphi, dpsi, da, db); phi, g, dphi, da follow pa, and psi, x,
    dx, dpsi, db follow pb.  sb None (b = a, psi = phi): (dx, dphi, da) with the
    shared anchors' and phases' total gradients."""
    dev = _dev(sa, phi, x, g, _perm(pa), sb, psi, _perm(pb))
    n = sa.numel()
    sym = sb is None
    k = n if sym else sb.numel()
    dx, dphi, da = torch.empty_like(x), torch.empty_like(g), torch.empty_like(g)
    dpsi = None if sym else torch.empty_like(x)
    db = None if sym else torch.empty_like(x)
    ws, nb = _ws(OP_BACKWARD_PHASED, n, k, 1, x.dtype, dev)
    # a NULL sb selects the symmetric case: an empty b side gets a non-NULL
    # pointer (the workspace's; nothing is read from it when k = 0)
    sbp = _ptr(sb) if sym or k > 0 else _ptr(ws)
    _check(lib().laplex_backward_phased(_ptr(sa), _ptr(pa), _ptr(phi), n, sbp, _ptr(pb), _ptr(psi), k,
                                        _ptr(x), _ptr(g), _ptr(dx), _ptr(dphi), _ptr(dpsi), _ptr(da), _ptr(db),
                                        _dt(x), _ptr(ws), nb, _stream(dev)))
    return (dx, dphi, da) if sym else (dx, dphi, dpsi, da, db)


@_serial
def gram_matrix(sa, sb, D=None, pa=None, pb=None, out=None):
    """M = A diag(D) A^T, A_ij = exp(-|a_i - b_j|), as an [n, n] tensor (rows and
    columns follow pa; sorted order without it).  D follows pb; None means 1."""
    dev = _dev(sa, sb, D, _perm(pa), _perm(pb), out)
    n, k = sa.numel(), sb.numel()
    M = torch.empty((n, n), dtype=sa.dtype, device=dev) if out is None else out
    ws, nb = _ws(OP_GRAM_MATRIX, n, k, 1, sa.dtype, dev)
    _check(lib().laplex_gram_matrix(_ptr(sa), _ptr(pa), n, _ptr(sb), _ptr(pb), k, _ptr(D), _ptr(M),
                                    M.stride(0) if n else max(n, 1), _dt(sa), _ptr(ws), nb, _stream(dev)))
    return M


@_serial
def matvec_sym_noalloc(sorted_anchors: torch.Tensor, x: torch.Tensor, perm=None, out=None):
    """y = K x through laplex_matvec_sym_noalloc: fp32, x of shape [n], n <= 2^30.

    For callers that cannot give the library a workspace: the scratch is a fixed
    array inside the library (shared by all calls on a device, so calls that may
    overlap on the GPU must be serialised by the caller)."""
    dev = _dev(sorted_anchors, x, _perm(perm), out)
    if x.dtype != torch.float32 or x.dim() != 1:
        raise LaplexError(EINVAL, "matvec_sym_noalloc takes fp32 x of shape [n]")
    n = sorted_anchors.numel()
    y = torch.empty_like(x) if out is None else out
    _check(lib().laplex_matvec_sym_noalloc(_ptr(sorted_anchors), _ptr(perm), n, _ptr(x), _ptr(y),
                                           _stream(dev)))
    return y


# ----------------------------------------------------------------------------- sequence operators

_SEQ_DTYPES = {torch.float32: F32, torch.float64: F64, torch.float16: F16, torch.bfloat16: BF16}


class LinattnGrads(NamedTuple):
    """Gradients of linattn; dstate and dlog_decay are None where not asked for."""
    dq: torch.Tensor
    dk: torch.Tensor
    dv: torch.Tensor
    dstate: Optional[torch.Tensor]
    dlog_decay: Optional[torch.Tensor]


_HERE_CTX = contextlib.nullcontext()


def _on(dev):
    """The device of the tensors made current: the library works on the current one."""
    return _HERE_CTX if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def _raw_stream(dev) -> int:
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _seq_dt(*ts) -> int:
    first = ts[0].dtype
    for t in ts:
        if t is not None and t.dtype != first:
            raise LaplexError(EINVAL, f"rows of {first} and of {t.dtype}")
    dt = _SEQ_DTYPES.get(first)
    if dt is None:
        raise LaplexError(EINVAL, f"dtype {first} is not float16, bfloat16, float32 or float64")
    return dt


def _seq_dev(*ts):
    """The tensors' common CUDA device."""
    at = None
    for t in ts:
        if t is None:
            continue
        d = t.get_device()  # -1: not CUDA
        if d < 0:
            raise LaplexError(EINVAL, "tensors must be on a CUDA device")
        if at is None:
            at = d
        elif d != at:
            raise LaplexError(EINVAL, "tensors are on different devices")
    return ts[0].device


def _packed(name, x):
    """[tokens, heads, dim] of x, which may also be [seqs, length, heads, dim]."""
    if x.dim() == 3 and x.stride(2) == 1:
        return x
    if x.dim() == 4:
        n, m = x.shape[:2]
        if n > 1 and m > 1 and x.stride(0) != m * x.stride(1):
            raise LaplexError(EINVAL, f"{name}: the sequences of a 4-d tensor must follow one another")
        step = x.stride(1) if m > 1 else x.stride(0)
        x = x.as_strided((n * m,) + tuple(x.shape[2:]), (step,) + x.stride()[2:])
    if x.dim() != 3:
        raise LaplexError(EINVAL, f"{name} must be [tokens, heads, dim] or [seqs, length, heads, dim]")
    if x.numel() and x.stride(2) != 1 and x.shape[2] > 1:
        raise LaplexError(EINVAL, f"{name}: the last dimension must be contiguous")
    return x


def _rows(x):
    if x is None:
        return None
    st = x.stride()
    return ctypes.byref(_Rows(x.data_ptr(), st[0], st[1]))


def _addr(x):
    return None if x is None else x.data_ptr()


def _new(shape, dtype, dev):
    return torch.empty(*shape, dtype=dtype, device=dev)  # (sizes one by one: 0.8 us less than as a tuple)


def _state(name, x, shape, dtype):
    if x is not None:
        if x.shape != shape or x.dtype != dtype or not x.is_contiguous():
            raise LaplexError(EINVAL, f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    return x


def _shape(q3, k3, v3, seqs, cu, log_decay, scale, dt):
    """The checked laplex_linattn_shape of packed q, k, v."""
    t, hq, dk = q3.shape
    hkv, dv = k3.shape[1], v3.shape[2]
    if k3.shape != (t, hkv, dk) or v3.shape != (t, hkv, dv):
        raise LaplexError(EINVAL, f"shapes of q {tuple(q3.shape)}, k {tuple(k3.shape)} and v {tuple(v3.shape)}")
    acc = torch.float64 if dt == F64 else torch.float32
    if log_decay.shape != (hkv,) or log_decay.dtype != acc or not log_decay.is_contiguous():
        raise LaplexError(EINVAL, f"log_decay must be a contiguous {acc} tensor of {hkv} heads")
    s = _LinattnShape(t, seqs, None if cu is None else cu.data_ptr(), hq, hkv, dk, dv, log_decay.data_ptr(),
                      float(dk ** -0.5 if scale is None else scale), dt)
    return s, acc


def _seqs(q, cu):
    if cu is None:
        return q.shape[0] if q.dim() == 4 else 1
    if cu.dtype != torch.int32 or cu.dim() != 1 or cu.numel() < 1 or not cu.is_contiguous():
        raise LaplexError(EINVAL, "cu_seqlens must be a contiguous int32 tensor [seqs + 1]")
    return cu.numel() - 1


def _seq_ws(dev, raw, nbytes):
    """Workspace of a sequence operator on stream `raw`: the stream's, or while a
    graph is captured one of the graph's own memory (the stream's may be replaced
    by a larger one while the graph lives, and two graphs may run at the same time).
    The graph may hand that memory to its later calls, so the call's status goes
    to a word outside it."""
    if not torch.cuda.is_current_stream_capturing():
        buf = Workspace._cache.get((dev, raw))
        if buf is None or buf.numel() < nbytes:
            buf = Workspace.get(dev, nbytes)
    else:
        buf = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        _enqueue.report_to(Workspace.captured_word(dev))
    return buf


_ws_sizes: dict = {}  # workspace bytes by shape; at most 4096 of them


def _keep_size(key, nbytes):
    if len(_ws_sizes) >= 4096:
        _ws_sizes.clear()
    _ws_sizes[key] = nbytes


def _linattn_ws(s, call, dev, raw):
    key = (s.tokens, s.seqs, s.cu_seqlens is None, s.hq, s.hkv, s.dk, s.dv, s.dtype, call)
    nbytes = _ws_sizes.get(key)
    if nbytes is None:
        out = ctypes.c_size_t(0)
        _check(lib().laplex_linattn_workspace_size(ctypes.byref(s), call, ctypes.byref(out)))
        nbytes = out.value
        _keep_size(key, nbytes)
    return _seq_ws(dev, raw, nbytes)


def linattn(q, k, v, log_decay, scale=None, cu_seqlens=None, state=None, return_state=False, out=None,
            state_out=None):
    """Decayed linear attention: S_t = e^lam S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.

    q [tokens, hq, dk], k [tokens, hkv, dk], v [tokens, hkv, dv] (float16,
    bfloat16, float32 or float64; slices with a contiguous last dimension are
    taken as they are), or 4-d [seqs, length, heads, dim].  log_decay [hkv]:
    lam, float32 (float64 for float64 rows).  cu_seqlens: int32 [seqs + 1], the
    bounds of packed sequences; rows behind the last bound are left as they are
    (unset where this call made the output).  state [seqs, hkv, dk, dv]: the
    states before the first tokens.  scale: dk ** -0.5 by default.

    Expanded tensors (a stride of 0) are refused: pass a copy.  16-bit rows take
    one rounding more than the output's own inside the products; the same rows
    in float32 take none.  No autograd graph is recorded, whatever the inputs
    require: the gradients are linattn_backward's.

    Returns o, or (o, states behind the last tokens) with return_state or
    state_out (which may be `state` itself)."""
    dev = _seq_dev(q, k, v, log_decay, cu_seqlens, state, out, state_out)
    seqs = _seqs(q, cu_seqlens)
    q3, k3, v3 = _packed("q", q), _packed("k", k), _packed("v", v)
    s, acc = _shape(q3, k3, v3, seqs, cu_seqlens, log_decay, scale, _seq_dt(q, k, v, out))
    shape = (seqs, s.hkv, s.dk, s.dv)
    _state("state", state, shape, acc)
    _state("state_out", state_out, shape, acc)
    with _on(dev), _enqueue:
        if out is None:
            out = _new(q.shape[:-1] + (s.dv,), q.dtype, dev)
        elif out.shape != q.shape[:-1] + (s.dv,):
            raise LaplexError(EINVAL, f"out must have the shape {tuple(q.shape[:-1]) + (s.dv,)}")
        if return_state and state_out is None:
            state_out = _new(shape, acc, dev)
        raw = _raw_stream(dev)
        ws = _linattn_ws(s, LINATTN_FORWARD, dev, raw)
        _check(lib().laplex_linattn(ctypes.byref(s), _rows(q3), _rows(k3), _rows(v3), _addr(state),
                                    _rows(_packed("out", out)), _addr(state_out), ws.data_ptr(), ws.numel(), raw))
    return out if state_out is None else (out, state_out)


def linattn_backward(q, k, v, log_decay, dout, scale=None, cu_seqlens=None, state=None, dstate=None,
                     return_dstate=None, return_dlog_decay=False, out=None):
    """Gradients of <dout, o> + <dstate, states behind the last tokens> of linattn.

    Arguments as in linattn; dout [tokens, hq, dv] (the expanded gradient of a sum
    as a copy), dstate [seqs, hkv, dk, dv] or None (zero).  Returns LinattnGrads(dq, dk, dv, dstate, dlog_decay): dstate,
    the gradient of `state`, where return_dstate is set (by default where `state`
    is given), dlog_decay [hkv] where return_dlog_decay is set.  out: (dq, dk,
    dv) to write into."""
    dev = _seq_dev(q, k, v, log_decay, dout, cu_seqlens, state, dstate, *(out or ()))
    seqs = _seqs(q, cu_seqlens)
    q3, k3, v3, do3 = _packed("q", q), _packed("k", k), _packed("v", v), _packed("dout", dout)
    s, acc = _shape(q3, k3, v3, seqs, cu_seqlens, log_decay, scale, _seq_dt(q, k, v, dout, *(out or ())))
    if do3.shape != (s.tokens, s.hq, s.dv):
        raise LaplexError(EINVAL, f"dout must have the shape {(s.tokens, s.hq, s.dv)}")
    shape = (seqs, s.hkv, s.dk, s.dv)
    _state("state", state, shape, acc)
    _state("dstate", dstate, shape, acc)
    with _on(dev), _enqueue:
        if out is None:
            out = tuple(_new(x.shape, x.dtype, dev) for x in (q, k, v))
        elif any(a.shape != b.shape for a, b in zip(out, (q, k, v))):
            raise LaplexError(EINVAL, "out must have the shapes of q, k and v")
        dq, dk, dv = out
        ds = None
        if return_dstate or (return_dstate is None and state is not None):
            ds = _new(shape, acc, dev)
        dl = torch.empty(s.hkv, dtype=acc, device=dev) if return_dlog_decay else None
        raw = _raw_stream(dev)
        ws = _linattn_ws(s, LINATTN_BACKWARD_DECAY if return_dlog_decay else LINATTN_BACKWARD, dev, raw)
        _check(lib().laplex_linattn_backward(
            ctypes.byref(s), _rows(q3), _rows(k3), _rows(v3), _rows(do3), _addr(state), _addr(dstate),
            _rows(_packed("dq", dq)), _rows(_packed("dk", dk)), _rows(_packed("dv", dv)), _addr(ds), _addr(dl),
            ws.data_ptr(), ws.numel(), raw))
    return LinattnGrads(dq, dk, dv, ds, dl)


def linattn_step(q, k, v, log_decay, states, slots=None, scale=None, out=None):
    """One token per row of linattn against a cache of states, updated in place.

    q [rows, hq, dk], k [rows, hkv, dk], v [rows, hkv, dv]; states [num_slots,
    hkv, dk, dv] (float32; float64 for float64 rows).  slots: int32 [rows], the
    state of each row (None: row n uses state n); a row whose slot is outside
    the cache gets zeros, rows that name one slot are applied in row order.
    Returns o [rows, hq, dv].  No autograd graph is recorded."""
    dev = _seq_dev(q, k, v, log_decay, states, slots, out)
    if q.dim() != 3:
        raise LaplexError(EINVAL, "q must be [rows, heads, dim]")
    q3, k3, v3 = _packed("q", q), _packed("k", k), _packed("v", v)
    s, acc = _shape(q3, k3, v3, 1, None, log_decay, scale, _seq_dt(q, k, v, out))
    if states.dim() != 4:
        raise LaplexError(EINVAL, "states must be [num_slots, hkv, dk, dv]")
    _state("states", states, (states.shape[0], s.hkv, s.dk, s.dv), acc)
    if slots is not None and (slots.dtype != torch.int32 or slots.shape != (s.tokens,) or not slots.is_contiguous()):
        raise LaplexError(EINVAL, "slots must be a contiguous int32 tensor [rows]")
    with _on(dev):
        if out is None:
            out = _new((s.tokens, s.hq, s.dv), q.dtype, dev)
        elif out.shape != (s.tokens, s.hq, s.dv):
            raise LaplexError(EINVAL, f"out must have the shape {(s.tokens, s.hq, s.dv)}")
        _check(lib().laplex_linattn_step(ctypes.byref(s), _rows(q3), _rows(k3), _rows(v3), states.data_ptr(),
                                         states.shape[0], _addr(slots), _rows(_packed("out", out)), _raw_stream(dev)))
    return out


def _tokens(tokens):
    if tokens.dtype not in (torch.int32, torch.int64) or not tokens.is_contiguous():
        raise LaplexError(EINVAL, "tokens must be a contiguous int32 or int64 tensor")
    return tokens.element_size()


def _table(name, x, dim=None):
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1) or (dim is not None and x.shape[1] != dim):
        raise LaplexError(EINVAL, f"{name} must be 2-d with contiguous rows" + ("" if dim is None else f" of {dim}"))
    return x.stride(0)


def embed(table, tokens, scale=1.0, out=None):
    """scale * table[tokens]: [*tokens.shape, dim]; a row of zeros for a token
    outside the table (padding).  table [rows, dim] of float16, bfloat16,
    float32 or float64; tokens int32 or int64.  No autograd graph is recorded:
    the table's gradient is embed_backward's."""
    dev = _seq_dev(table, tokens, out)
    dt, tb, ld = _seq_dt(table, out), _tokens(tokens), _table("table", table)
    shape = tokens.shape + (table.shape[1],)
    with _on(dev):
        if out is None:
            out = _new(shape, table.dtype, dev)
        elif out.shape != shape or (out.dim() != 2 and not out.is_contiguous()):
            raise LaplexError(EINVAL, f"out must have the shape {shape}")
        o2 = out if out.dim() == 2 else out.view(-1, table.shape[1])
        _check(lib().laplex_embed(table.data_ptr(), ld, table.shape[0], table.shape[1], tokens.data_ptr(), tb,
                                  tokens.numel(), float(scale), o2.data_ptr(), _table("out", o2), dt, _raw_stream(dev)))
    return out


def embed_backward(tokens, g, rows, scale=1.0, out=None, accumulate=False, dtype=None):
    """Gradient of embed in the table: [rows, dim] with scale times the sum of the
    rows of g (summed in fp32, in order of their positions) that name each row.

    g [*tokens.shape, dim].  out: a [rows, dim] tensor of g's type or float32 to
    write, or with accumulate to add into (rows that no token names are then
    left as they are); dtype: the type of a fresh one (g's by default)."""
    dev = _seq_dev(tokens, g, out)
    dt, tb = _seq_dt(g), _tokens(tokens)
    if g.shape[:-1] != tokens.shape:
        raise LaplexError(EINVAL, f"g must have the shape {tuple(tokens.shape)} + (dim,)")
    if g.dim() != 2:
        if not g.is_contiguous():
            raise LaplexError(EINVAL, "g of other than two dimensions must be contiguous")
        g = g.view(-1, g.shape[-1])
    dim, ld = g.shape[1], _table("g", g)
    if accumulate and out is None:
        raise LaplexError(EINVAL, "accumulate needs out")
    with _on(dev), _enqueue:
        if out is None:
            out = _new((rows, dim), dtype or g.dtype, dev)
        if out.shape[0] != rows or out.dtype not in (g.dtype, torch.float32):
            raise LaplexError(EINVAL, f"out must have {rows} rows of {g.dtype} or float32")
        key = (tokens.numel(), rows, dim, dt)
        nbytes = _ws_sizes.get(key)
        if nbytes is None:
            size = ctypes.c_size_t(0)
            _check(lib().laplex_embed_backward_workspace_size(*key, ctypes.byref(size)))
            nbytes = size.value
            _keep_size(key, nbytes)
        raw = _raw_stream(dev)
        ws = _seq_ws(dev, raw, nbytes)
        _check(lib().laplex_embed_backward(tokens.data_ptr(), tb, tokens.numel(), g.data_ptr(), ld, rows, dim,
                                           float(scale), int(bool(accumulate)), out.data_ptr(), _table("out", out, dim),
                                           dt, _SEQ_DTYPES[out.dtype], ws.data_ptr(), ws.numel(), raw))
    return out


# ----------------------------------------------------------------------------- host buffers

def matvec_sym_host(sorted_anchors: torch.Tensor, x: torch.Tensor, perm=None, device="cuda",
                    out=None):
    """End-to-end symmetric product from HOST tensors: copies the inputs to the device
    (non-blocking from pinned memory), runs laplex_matvec_sym, copies y back."""
    s_d = sorted_anchors.to(device, non_blocking=True)
    x_d = x.to(device, non_blocking=True)
    p_d = None if perm is None else perm.to(device, non_blocking=True)
    y_d = matvec_sym(s_d, x_d, p_d)
    if out is None:
        return y_d.cpu()
    out.copy_(y_d, non_blocking=True)
    return out


class HostStreamer:
    """Symmetric products of a stream of host batches (pinned tensors), with the
    copies overlapped: batch k's host-to-device copy runs on one CUDA stream
    while batch k-1 is computed on a second and batch k-2's result returns on a
    third.  Device buffers are double-buffered; events order each buffer's
    reuse.  Only copies and laplex_matvec_sym calls are enqueued (no host-side
    arithmetic).

    submit(sorted_h, x_h, y_h, perm_h=None) enqueues one batch and returns at
    once; y_h is complete after synchronize()."""

    def __init__(self, n: int, B: int = 1, dtype=torch.float32, device="cuda", with_perm=False):
        self.dev = torch.device(device)
        self.n, self.B = n, B
        shape = (n,) if B == 1 else (n, B)
        self.h2d = torch.cuda.Stream(self.dev)
        self.comp = torch.cuda.Stream(self.dev)
        self.d2h = torch.cuda.Stream(self.dev)
        self.bufs = []
        for _ in range(2):
            self.bufs.append({
                "s": torch.empty(n, dtype=dtype, device=self.dev),
                "x": torch.empty(shape, dtype=dtype, device=self.dev),
                "y": torch.empty(shape, dtype=dtype, device=self.dev),
                "p": torch.empty(n, dtype=torch.int32, device=self.dev) if with_perm else None,
                "loaded": torch.cuda.Event(), "computed": torch.cuda.Event(),
                "drained": torch.cuda.Event()})
        self.k = 0

    def submit(self, sorted_h, x_h, y_h, perm_h=None):
        b = self.bufs[self.k % 2]
        with torch.cuda.stream(self.h2d):
            self.h2d.wait_event(b["computed"])  # s, x, p free once the product that read them is done
            b["s"].copy_(sorted_h, non_blocking=True)
            b["x"].copy_(x_h, non_blocking=True)
            if perm_h is not None:
                b["p"].copy_(perm_h, non_blocking=True)
            b["loaded"].record(self.h2d)
        with torch.cuda.stream(self.comp):
            self.comp.wait_event(b["loaded"])
            self.comp.wait_event(b["drained"])  # y free once its last copy back is done
            matvec_sym(b["s"], b["x"], b["p"] if perm_h is not None else None, out=b["y"])
            b["computed"].record(self.comp)
        with torch.cuda.stream(self.d2h):
            self.d2h.wait_event(b["computed"])
            y_h.copy_(b["y"], non_blocking=True)
            b["drained"].record(self.d2h)
        self.k += 1

    def synchronize(self):
        """Wait for every submitted batch; raise if a product recorded a device error."""
        torch.cuda.synchronize(self.dev)
        with torch.cuda.stream(self.comp):
            Workspace.status(self.dev)
