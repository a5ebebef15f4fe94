"""Python binding of libqgemv.so, the MI355X (gfx950) quantized GEMV library.

Argument marshalling only: every step of the computation runs in the library's
HIP kernels. torch supplies device memory and the current stream. The binding
raises if the compiled library is missing: there is no fallback path.
"""
from __future__ import annotations

import array
import ctypes
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqgemv.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "qgemv.h")

MAX_BATCH = 8
SMALLN_MAX = 32
I8_MAX_K = 131071
BEAM_MAX = 32
BEAM_MAX_SELECT = 64
BEAM_MAX_STATES = 56
F8_BLOCK = 128
F8_MAX_K = 131072
EXPERTS_MAX = 1024
EXPERTS_MAX_K = 32

_lib = None


class QGError(RuntimeError):
    def __init__(self, func: str, status: int, detail: str):
        super().__init__(f"{func}: status {status}: {detail}")
        self.status = status


class _Problem(ctypes.Structure):
    _fields_ = [("w_packed", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("M", ctypes.c_int64), ("K", ctypes.c_int64)]


class _GemmProblem(ctypes.Structure):
    _fields_ = [("w_packed", ctypes.c_void_p), ("X", ctypes.c_void_p), ("ldx", ctypes.c_int64),
                ("Y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("M", ctypes.c_int64), ("K", ctypes.c_int64),
                ("N", ctypes.c_int64)]


class _GemmQ81Problem(ctypes.Structure):
    _fields_ = [("w_packed", ctypes.c_void_p), ("xq", ctypes.c_void_p), ("Y", ctypes.c_void_p),
                ("ldy", ctypes.c_int64), ("M", ctypes.c_int64), ("K", ctypes.c_int64), ("N", ctypes.c_int64)]


class _LaunchOverride(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("gemv_waves", "smalln_form", "smalln_waves", "smalln_tiles",
                                            "smalln_depth", "verify_form", "verify_waves", "verify_tiles")]


# kernel forms a launch override can force (include/qgemv.h)
FORM_AUTO = 0
FORM_SMALLN_REGS, FORM_SMALLN_LDS, FORM_SMALLN_LDS1, FORM_SMALLN_DOT, FORM_SMALLN_STREAM, FORM_SMALLN_WALK, \
    FORM_SMALLN_SPLIT, FORM_SMALLN_SLICE = 1, 2, 3, 4, 5, 6, 7, 8
FORM_VERIFY_MFMA, FORM_VERIFY_DOT, FORM_VERIFY_STREAM = 1, 2, 3


class _TopkOut(ctypes.Structure):
    _fields_ = [("index", ctypes.c_void_p), ("logit", ctypes.c_void_p), ("logprob", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("token", ctypes.c_void_p)]


class _Sampler(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("top_p", ctypes.c_float), ("min_p", ctypes.c_float),
                ("u", ctypes.c_void_p)]


class _BeamIn(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("logits_type", ctypes.c_int), ("ld", ctypes.c_int64),
                ("batch", ctypes.c_int64), ("beams", ctypes.c_int), ("vocab", ctypes.c_int64),
                ("score", ctypes.c_void_p), ("finished", ctypes.c_void_p), ("length", ctypes.c_void_p),
                ("length_penalty", ctypes.c_double), ("eos", ctypes.c_int32)]


class _BeamOut(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("token", "parent", "score", "finished", "length")]


class _BeamState(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("src_row", ctypes.c_int64),
                ("dst_row", ctypes.c_int64), ("src_outer", ctypes.c_int64), ("dst_outer", ctypes.c_int64),
                ("outer", ctypes.c_int64), ("span", ctypes.c_int64)]


class _F8Grouped(ctypes.Structure):
    _fields_ = [("w_packed", ctypes.c_void_p), ("w_scale", ctypes.c_void_p), ("xq", ctypes.c_void_p), ("ldx", ctypes.c_int64),
                ("x_scale", ctypes.c_void_p), ("ldxs", ctypes.c_int64), ("x_rows", ctypes.c_int64), ("row", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("Y", ctypes.c_void_p), ("y_type", ctypes.c_int),
                ("ldy", ctypes.c_int64), ("M", ctypes.c_int64), ("K", ctypes.c_int64), ("experts", ctypes.c_int64),
                ("rows", ctypes.c_int64)]


class _ExpertsOut(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("expert", "weight", "position", "row", "offsets")]


_P, _I64, _SZ, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int

_SIGS = {
    "qg_abi_version": (_I, []),
    "qg_status_string": (ctypes.c_char_p, [_I]),
    "qg_last_error": (ctypes.c_char_p, []),
    "qg_q4k_bytes": (_SZ, [_I64, _I64]),
    "qg_q8_0_bytes": (_SZ, [_I64, _I64]),
    "qg_q6k_bytes": (_SZ, [_I64, _I64]),
    "qg_pack_q4k": (_I, [_P, _P, _I64, _I64, _P]),
    "qg_pack_q8_0": (_I, [_P, _P, _I64, _I64, _P]),
    "qg_pack_q6k": (_I, [_P, _P, _I64, _I64, _P]),
    "qg_workspace_clear": (_I, [_P, _SZ, _P]),
    "qgemv_q4k": (_I, [_P, _P, _P, _I64, _I64, _P]),
    "qgemv_q4k_batch": (_I, [ctypes.POINTER(_Problem), _I, _P]),
    "qgemv_q8_0": (_I, [_P, _P, _P, _I64, _I64, _P]),
    "qg_q8_1_bytes": (_SZ, [_I64]),
    "qg_quantize_q8_1": (_I, [_P, _I64, _P, _P]),
    "qg_quantize_q8_1_columns": (_I, [_P, _I64, _I64, _I64, _P, _P]),
    "qgemv_q4k_q8_1": (_I, [_P, _P, _P, _I64, _I64, _P]),
    "qgemv_q4k_q8_1_batch": (_I, [ctypes.POINTER(_Problem), _I, _P]),
    "qgemm_q4k_q8_1_smalln": (_I, [_P, _P, _P, _I64, _I64, _I64, _I64, _P]),
    "qgemm_q4k_q8_1_smalln_batch": (_I, [ctypes.POINTER(_GemmQ81Problem), _I, _P]),
    "qgemv_q6k": (_I, [_P, _P, _P, _I64, _I64, _P]),
    "qgemm_q4k_smalln": (_I, [_P, _P, _I64, _P, _I64, _I64, _I64, _I64, _P]),
    "qgemm_q4k_smalln_batch": (_I, [ctypes.POINTER(_GemmProblem), _I, _P]),
    "qgemm_q4k_smalln_batch_workspace_bytes": (_SZ, [ctypes.POINTER(_GemmProblem), _I]),
    "qgemm_q4k_smalln_batch_ws": (_I, [ctypes.POINTER(_GemmProblem), _I, _P, _SZ, _P]),
    "qg_set_launch_override": (_I, [ctypes.c_void_p]),
    "qg_get_launch_override": (_I, [ctypes.c_void_p]),
    "lmhead_argmax_verify_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "lmhead_argmax_verify": (_I, [_P, _P, _I64, _I64, _I64, _I64, _P, _SZ, _P, _P, _P]),
    "lmhead_argmax_verify_q8_1_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "lmhead_argmax_verify_q8_1": (_I, [_P, _P, _I64, _I64, _I64, _P, _SZ, _P, _P, _P]),
    "lmhead_argmax_workspace_bytes": (_SZ, [_I64, _I64]),
    "logits_topk_workspace_bytes": (_SZ, [_I64]),
    "logits_topk": (_I, [_P, _I64, _I, ctypes.POINTER(_Sampler), _P, _SZ, ctypes.POINTER(_TopkOut), _P]),
    "lmhead_topk_workspace_bytes": (_SZ, [_I64, _I64]),
    "lmhead_topk": (_I, [_P, _P, _I64, _I64, _I, _P, ctypes.POINTER(_Sampler), _P, _SZ, ctypes.POINTER(_TopkOut),
                         _P]),
    "lmhead_argmax": (_I, [_P, _P, _I64, _I64, _P, _SZ, _P, _P, _P]),
    "lmhead_argmax_noalloc": (_I, [_P, _P, _I64, _I64, _P, _P, _P]),
    "qg_i8_bytes": (_SZ, [_I64, _I64]),
    "qg_pack_i8": (_I, [_P, _I64, _P, _I64, _I64, _P]),
    "qg_quantize_i8_rows": (_I, [_P, _I, _I64, _I64, _I64, _P, _I64, _P, _P]),
    "qgemm_i8_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "qgemm_i8": (_I, [_P, _P, _P, _I64, _P, _P, _P, _I, _I64, _I64, _I64, _I64, _P, _SZ, _P]),
    "logits_beam_select_workspace_bytes": (_SZ, [_I, _I64, _I, _I64, _I]),
    "logits_beam_select": (_I, [ctypes.POINTER(_BeamIn), _I, _P, _SZ, ctypes.POINTER(_BeamOut), _P]),
    "qg_beam_reorder": (_I, [_P, _I, _P, _I64, _I, _I, _P]),
    "qg_beam_reorder_check": (_I, [_P, _I, _P, _I64, _I, _I]),
    "qg_f8_bytes": (_SZ, [_I64, _I64, _I64]),
    "qg_pack_f8": (_I, [_P, _I64, _I64, _P, _I64, _I64, _I64, _P]),
    "qg_quantize_f8_rows": (_I, [_P, _I, _I64, _I, _P, _I64, _I64, _P, _I64, _P, _I64, _P]),
    "qgemm_f8_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I]),
    "qgemm_f8": (_I, [_P, _P, _P, _I64, _P, _I64, _P, _P, _I, _I64, _I64, _I64, _I64, _P, _SZ, _P]),
    "qgemm_f8_grouped": (_I, [ctypes.POINTER(_F8Grouped), _P]),
    "logits_expert_select_workspace_bytes": (_SZ, [_I64, _I, _I]),
    "logits_expert_select": (_I, [_P, _I, _I64, _I64, _I, _I, _I, ctypes.c_float, _P, _SZ, ctypes.POINTER(_ExpertsOut), _P]),
    "qg_expert_combine": (_I, [_P, _I, _I64, _I64, _P, _P, _I, _P, _I64, _P, _I, _I64, _I64, _I64, _P]),
}


def lib() -> ctypes.CDLL:
    """Load libqgemv.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with quantized_gemv_argmax_amd.build.build() "
                               "(hipcc, gfx950); there is no fallback implementation")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions include/qgemv.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^\s*(?:const\s+)?[a-z_0-9]+\s*\*?\s*([a-z_][a-z_0-9]*)\s*\(", text, flags=re.M)
    return sorted(set(names))


def status_string(s: int) -> str:
    return lib().qg_status_string(int(s)).decode()


def last_error() -> str:
    return lib().qg_last_error().decode()


def _check(func: str, status: int):
    if status != 0:
        raise QGError(func, status, f"{status_string(status)}: {last_error()}")


def _stream(device=None) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors must live on the GPU")


# ------------------------------------------------------------------ workspace
class Workspace:
    """A device scratch buffer reused across calls on one stream (grown on demand).
    It starts all-zero. Three kinds of calls use one: "zeros" (the LM-head and top-k
    calls) needs it so and leaves it so; "counters" (qgemm_q4k_smalln_batch_ws) needs its
    counters zero and leaves the rest undefined; "scratch" (qgemm_i8, qgemm_f8,
    logits_beam_select, logits_expert_select) needs nothing and leaves all of it undefined. One workspace may serve the first two
    in turn, cleared between them by the calls themselves, but not those and the third,
    whichever came first. Outgrown buffers are kept, as a captured graph may still hold
    them; a buffer is at least twice the one before it, so that together they are smaller
    than the current one. release_outgrown() frees them."""

    def __init__(self, device=None, nbytes: int = 0):
        self.device = torch.device(device if device is not None else "cuda")
        self.buf = None
        self.outgrown = []
        self.kinds = set()  # of the calls it has served
        if nbytes:
            self.ensure(nbytes)

    def ensure(self, nbytes: int):
        if nbytes and (self.buf is None or self.buf.numel() < nbytes):
            if self.buf is not None:
                self.outgrown.append(self.buf)
            with torch.inference_mode(False):  # (an inference tensor could not be cleared outside that mode)
                self.buf = torch.zeros(max(nbytes, 1 << 20, 2 * self.nbytes()), dtype=torch.uint8, device=self.device)
        return self

    def release_outgrown(self):
        """Frees the buffers that growing has replaced: once no captured graph that used
        this workspace will be replayed, and its calls on other streams have ended."""
        self.outgrown.clear()
        return self

    def serve(self, nbytes: int, kind: str):
        """ensure(nbytes) for a call of `kind`, zeros where it needs them."""
        if kind not in self.kinds:
            if self.kinds and "scratch" in (kind, *self.kinds):
                raise ValueError("a workspace of qgemm_i8, qgemm_f8, logits_beam_select or logits_expert_select, which leave it "
                                 "undefined, cannot serve a call that needs zeros, nor the other way round: give each kind its own")
            self.kinds.add(kind)
        self.ensure(nbytes)
        # A captured "counters" call may have run since, so this is not done once. (A
        # captured "zeros" call does not come here again: served() sees to that one.)
        if kind == "zeros" and "counters" in self.kinds:
            self.clear()
        return self

    def served(self, kind: str):
        """After a call of `kind`: clears what it left, where other calls need zeros."""
        if kind == "counters" and "zeros" in self.kinds:
            self.clear()

    def clear(self):
        """Zeros on the current stream (a call that failed may have left something else)."""
        if self.buf is not None:
            self.buf.zero_()
        return self

    def ptr(self) -> int | None:
        return None if self.buf is None else self.buf.data_ptr()

    def nbytes(self) -> int:
        return 0 if self.buf is None else self.buf.numel()


_default_ws: dict = {}


def default_workspace(device=None) -> Workspace:
    dev = torch.device(device if device is not None else "cuda")
    key = (dev.type, dev.index if dev.index is not None else torch.cuda.current_device())
    if key not in _default_ws:
        _default_ws[key] = Workspace(dev)
        _default_ws[key].kinds.add("zeros")  # handed to a "scratch" call first, it would refuse its own
    return _default_ws[key]


def _ws(ws: Workspace | None, need: int, device) -> Workspace:
    ws = ws if ws is not None else default_workspace(device)
    return ws.serve(need, "zeros")


# ------------------------------------------------------------------ sizes / packing
def q4k_bytes(M: int, K: int) -> int:
    return int(lib().qg_q4k_bytes(M, K))


def q8_0_bytes(M: int, K: int) -> int:
    return int(lib().qg_q8_0_bytes(M, K))


def q6k_bytes(M: int, K: int) -> int:
    return int(lib().qg_q6k_bytes(M, K))


def pack_q4k(canonical: torch.Tensor, M: int, K: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """Repack canonical Q4_K bytes (uint8 device tensor) into the library's layout."""
    _need_cuda(canonical)
    n = q4k_bytes(M, K)
    if canonical.numel() != n or canonical.dtype != torch.uint8:
        raise ValueError(f"expected {n} uint8 bytes of Q4_K blocks")
    out = out if out is not None else torch.empty(n, dtype=torch.uint8, device=canonical.device)
    _check("qg_pack_q4k", lib().qg_pack_q4k(_ptr(canonical), _ptr(out), M, K, _stream(canonical.device)))
    return out


def pack_q8_0(canonical: torch.Tensor, M: int, K: int, out: torch.Tensor | None = None) -> torch.Tensor:
    _need_cuda(canonical)
    n = q8_0_bytes(M, K)
    if canonical.numel() != n or canonical.dtype != torch.uint8:
        raise ValueError(f"expected {n} uint8 bytes of Q8_0 blocks")
    out = out if out is not None else torch.empty(n, dtype=torch.uint8, device=canonical.device)
    _check("qg_pack_q8_0", lib().qg_pack_q8_0(_ptr(canonical), _ptr(out), M, K, _stream(canonical.device)))
    return out


def pack_q6k(canonical: torch.Tensor, M: int, K: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """Repack canonical Q6_K bytes (uint8 device tensor) into the library's layout."""
    _need_cuda(canonical)
    n = q6k_bytes(M, K)
    if canonical.numel() != n or canonical.dtype != torch.uint8:
        raise ValueError(f"expected {n} uint8 bytes of Q6_K blocks")
    out = out if out is not None else torch.empty(n, dtype=torch.uint8, device=canonical.device)
    _check("qg_pack_q6k", lib().qg_pack_q6k(_ptr(canonical), _ptr(out), M, K, _stream(canonical.device)))
    return out


# ------------------------------------------------------------------ launch override
class launch_override:
    """Context manager (or plain call through .set()) that forces kernel forms or
    launch shapes on this host thread for tests and measurements, through
    qg_set_launch_override; fields not given keep the automatic choice. Example:
    `with qg.launch_override(smalln_form=qg.FORM_SMALLN_LDS, smalln_tiles=2): ...`"""

    def __init__(self, **fields):
        self.o = _LaunchOverride()
        for k, v in fields.items():
            if k not in dict(_LaunchOverride._fields_):
                raise TypeError(f"unknown launch override field {k!r}")
            setattr(self.o, k, int(v))
        self._prev = None

    def set(self):
        _check("qg_set_launch_override", lib().qg_set_launch_override(ctypes.byref(self.o)))

    def __enter__(self):
        self._prev = _LaunchOverride()
        _check("qg_get_launch_override", lib().qg_get_launch_override(ctypes.byref(self._prev)))
        self.set()
        return self

    def __exit__(self, *exc):
        _check("qg_set_launch_override", lib().qg_set_launch_override(ctypes.byref(self._prev)))
        return False


def get_launch_override() -> dict:
    o = _LaunchOverride()
    _check("qg_get_launch_override", lib().qg_get_launch_override(ctypes.byref(o)))
    return {n: getattr(o, n) for n, _ in _LaunchOverride._fields_}


# ------------------------------------------------------------------ products
def qgemv_q4k(w: torch.Tensor, x: torch.Tensor, M: int, K: int, y: torch.Tensor | None = None) -> torch.Tensor:
    """y[M] = W x for a packed Q4_K matrix (fp32 x, y)."""
    _need_cuda(w, x, y)
    y = y if y is not None else torch.empty(M, dtype=torch.float32, device=x.device)
    _check("qgemv_q4k", lib().qgemv_q4k(_ptr(w), _ptr(x), _ptr(y), M, K, _stream(x.device)))
    return y


def qgemv_q4k_batch(problems):
    """problems: list of (w_packed, x, y, M, K); one launch for all of them."""
    arr = (_Problem * len(problems))()
    dev = None
    for i, (w, x, y, M, K) in enumerate(problems):
        _need_cuda(w, x, y)
        dev = x.device
        arr[i] = _Problem(_ptr(w), _ptr(x), _ptr(y), M, K)
    _check("qgemv_q4k_batch", lib().qgemv_q4k_batch(arr, len(problems), _stream(dev)))
    return [p[2] for p in problems]


def qgemv_q8_0(w: torch.Tensor, x: torch.Tensor, M: int, K: int, y: torch.Tensor | None = None) -> torch.Tensor:
    _need_cuda(w, x, y)
    y = y if y is not None else torch.empty(M, dtype=torch.float32, device=x.device)
    _check("qgemv_q8_0", lib().qgemv_q8_0(_ptr(w), _ptr(x), _ptr(y), M, K, _stream(x.device)))
    return y


def q8_1_bytes(K: int) -> int:
    return int(lib().qg_q8_1_bytes(K))


def q8_1_views(xq: torch.Tensor, K: int):
    """(d float32[K/32], q int8[K], s int16[K/32]) views of a quantized-activation buffer."""
    nc = K // 32
    q_off = -(-4 * nc // 16) * 16
    s_off = -(-(q_off + K) // 16) * 16
    return (xq[:4 * nc].view(torch.float32), xq[q_off:q_off + K].view(torch.int8),
            xq[s_off:s_off + 2 * nc].view(torch.int16))


def quantize_q8_1(x: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Int8 activations with a float32 scale and a block sum per 32 (uint8 buffer)."""
    _need_cuda(x, out)
    K = x.numel()
    n = q8_1_bytes(K)
    out = out if out is not None else torch.empty(n, dtype=torch.uint8, device=x.device)
    _check("qg_quantize_q8_1", lib().qg_quantize_q8_1(_ptr(x), K, _ptr(out), _stream(x.device)))
    return out


def qgemv_q4k_q8_1(w: torch.Tensor, xq: torch.Tensor, M: int, K: int, y: torch.Tensor | None = None) -> torch.Tensor:
    """y[M] = W xq for a packed Q4_K matrix and quantized activations."""
    _need_cuda(w, xq, y)
    y = y if y is not None else torch.empty(M, dtype=torch.float32, device=xq.device)
    _check("qgemv_q4k_q8_1", lib().qgemv_q4k_q8_1(_ptr(w), _ptr(xq), _ptr(y), M, K, _stream(xq.device)))
    return y


def qgemv_q4k_q8_1_batch(problems):
    """problems: list of (w_packed, xq, y, M, K); one launch for all of them."""
    arr = (_Problem * len(problems))()  # same field layout as qg_gemv_q8_1_problem
    dev = None
    for i, (w, xq, y, M, K) in enumerate(problems):
        _need_cuda(w, xq, y)
        dev = xq.device
        arr[i] = _Problem(_ptr(w), _ptr(xq), _ptr(y), M, K)
    _check("qgemv_q4k_q8_1_batch", lib().qgemv_q4k_q8_1_batch(arr, len(problems), _stream(dev)))
    return [p[2] for p in problems]


def quantize_q8_1_columns(X: torch.Tensor, out: torch.Tensor | None = None, K: int | None = None) -> torch.Tensor:
    """X (N, ldx) fp32, row n = column n (its first K = ldx entries unless K is
    given) -> N consecutive Q8_1 buffers of q8_1_bytes(K) bytes, in one launch."""
    _need_cuda(X, out)
    N, ldx = X.shape
    if X.stride(1) != 1 or X.stride(0) != ldx:
        raise ValueError("X must be a contiguous (N, ldx) tensor")
    K = ldx if K is None else K
    nb = q8_1_bytes(K)
    out = out if out is not None else torch.empty(N * nb, dtype=torch.uint8, device=X.device)
    _check("qg_quantize_q8_1_columns",
           lib().qg_quantize_q8_1_columns(_ptr(X), ldx, K, N, _ptr(out), _stream(X.device)))
    return out


def qgemm_q4k_q8_1_smalln(w: torch.Tensor, xq: torch.Tensor, M: int, K: int, N: int,
                          Y: torch.Tensor | None = None) -> torch.Tensor:
    """Y (N, ldy) = W Xq for N <= 8 quantized columns (quantize_q8_1_columns)."""
    _need_cuda(w, xq, Y)
    Y = Y if Y is not None else torch.empty((N, (M + 3) // 4 * 4), dtype=torch.float32, device=xq.device)
    if Y.shape[0] != N or Y.stride(1) != 1:
        raise ValueError("Y must be a contiguous (N, ldy) tensor")
    _check("qgemm_q4k_q8_1_smalln", lib().qgemm_q4k_q8_1_smalln(_ptr(w), _ptr(xq), _ptr(Y), Y.stride(0), M, K, N,
                                                                _stream(xq.device)))
    return Y


def qgemm_q4k_q8_1_smalln_batch(problems):
    """problems: list of (w_packed, xq, Y, M, K) with Y (N, ldy) and xq holding N
    quantized columns; one launch for all of them."""
    arr = (_GemmQ81Problem * len(problems))()
    dev = None
    for i, (w, xq, Y, M, K) in enumerate(problems):
        _need_cuda(w, xq, Y)
        dev = xq.device
        if Y.stride(1) != 1:
            raise ValueError("Y must be a contiguous (N, ldy) tensor")
        arr[i] = _GemmQ81Problem(_ptr(w), _ptr(xq), _ptr(Y), Y.stride(0), M, K, Y.shape[0])
    _check("qgemm_q4k_q8_1_smalln_batch", lib().qgemm_q4k_q8_1_smalln_batch(arr, len(problems), _stream(dev)))
    return [p[2] for p in problems]


def qgemv_q6k(w: torch.Tensor, x: torch.Tensor, M: int, K: int, y: torch.Tensor | None = None) -> torch.Tensor:
    """y[M] = W x for a packed Q6_K matrix (fp32 x, y)."""
    _need_cuda(w, x, y)
    y = y if y is not None else torch.empty(M, dtype=torch.float32, device=x.device)
    _check("qgemv_q6k", lib().qgemv_q6k(_ptr(w), _ptr(x), _ptr(y), M, K, _stream(x.device)))
    return y


def qgemm_q4k_smalln(w: torch.Tensor, X: torch.Tensor, M: int, K: int, Y: torch.Tensor | None = None) -> torch.Tensor:
    """X: (N, ldx) fp32, row n = column n of the K x N operand (ldx >= K, ldx % 4 == 0).
    Returns Y as (N, ldy) with Y[n, :M] = W X[n, :K]."""
    _need_cuda(w, X, Y)
    N, ldx = X.shape
    if X.stride(1) != 1 or X.stride(0) != ldx:
        raise ValueError("X must be a contiguous (N, ldx) tensor")
    if Y is None:
        ldy = (M + 3) // 4 * 4
        Y = torch.empty((N, ldy), dtype=torch.float32, device=X.device)
    ldy = Y.shape[1]
    _check("qgemm_q4k_smalln", lib().qgemm_q4k_smalln(_ptr(w), _ptr(X), ldx, _ptr(Y), ldy, M, K, N,
                                                        _stream(X.device)))
    return Y


def _gemm_problems(problems):
    arr = (_GemmProblem * len(problems))()
    dev = None
    for i, (w, X, Y, M, K) in enumerate(problems):
        _need_cuda(w, X, Y)
        dev = X.device
        N, ldx = X.shape
        if X.stride(1) != 1 or X.stride(0) != ldx or Y.stride(1) != 1 or Y.shape[0] != N:
            raise ValueError("X and Y must be contiguous (N, ld) tensors with the same N")
        arr[i] = _GemmProblem(_ptr(w), _ptr(X), ldx, _ptr(Y), Y.stride(0), M, K, N)
    return arr, dev


def qgemm_q4k_smalln_batch(problems):
    """problems: list of (w_packed, X, Y, M, K) with X (N, ldx) and Y (N, ldy) as in
    qgemm_q4k_smalln; one launch for all of them. Returns the Y tensors."""
    arr, dev = _gemm_problems(problems)
    _check("qgemm_q4k_smalln_batch", lib().qgemm_q4k_smalln_batch(arr, len(problems), _stream(dev)))
    return [p[2] for p in problems]


def qgemm_q4k_smalln_batch_workspace_bytes(problems) -> int:
    arr, _ = _gemm_problems(problems)
    return lib().qgemm_q4k_smalln_batch_workspace_bytes(arr, len(problems))


def qgemm_q4k_smalln_batch_ws(problems, ws: Workspace | None = None):
    """qgemm_q4k_smalln_batch with a workspace (sized by
    qgemm_q4k_smalln_batch_workspace_bytes; a per-device scratch buffer if None),
    which lets the library split few-tile, many-column products over K slices. One
    workspace serves batches of any shapes; its counters come back zero and the rest
    of it undefined (all of it zero if it also serves the LM-head or top-k calls). Calls
    sharing a workspace (the scratch one included) must not overlap: calls on concurrent
    streams pass workspaces of their own."""
    arr, dev = _gemm_problems(problems)
    need = lib().qgemm_q4k_smalln_batch_workspace_bytes(arr, len(problems))
    if ws is None:  # scratch contents: never the zero-kept workspace of the LM-head calls
        key = ("scratch", str(dev))
        ws = _default_ws.setdefault(key, Workspace(dev))
    if need:
        ws.serve(need, "counters")
    _check("qgemm_q4k_smalln_batch_ws",
           lib().qgemm_q4k_smalln_batch_ws(arr, len(problems), ws.ptr(), ws.nbytes(), _stream(dev)))
    if need:
        ws.served("counters")
    return [p[2] for p in problems]


def lmhead_argmax(w: torch.Tensor, x: torch.Tensor, M: int, K: int, out_index: torch.Tensor | None = None,
                  out_value: torch.Tensor | None = None, ws: Workspace | None = None):
    """Fused Q8_0 LM head + argmax. Returns (index int32[1], value float32[1]) device tensors."""
    _need_cuda(w, x, out_index, out_value)
    out_index = out_index if out_index is not None else torch.empty(1, dtype=torch.int32, device=x.device)
    out_value = out_value if out_value is not None else torch.empty(1, dtype=torch.float32, device=x.device)
    need = int(lib().lmhead_argmax_workspace_bytes(M, K))
    ws = _ws(ws, need, x.device)
    _check("lmhead_argmax", lib().lmhead_argmax(_ptr(w), _ptr(x), M, K, ws.ptr(), ws.nbytes(), _ptr(out_index),
                                                  _ptr(out_value), _stream(x.device)))
    return out_index, out_value


def lmhead_argmax_noalloc(w: torch.Tensor, x: torch.Tensor, M: int, K: int, out_index: torch.Tensor | None = None,
                          out_value: torch.Tensor | None = None):
    """lmhead_argmax with the partials in the library's own per-GPU array (no
    workspace; calls on one GPU must not overlap). Returns (index, value) tensors."""
    _need_cuda(w, x, out_index, out_value)
    out_index = out_index if out_index is not None else torch.empty(1, dtype=torch.int32, device=x.device)
    out_value = out_value if out_value is not None else torch.empty(1, dtype=torch.float32, device=x.device)
    _check("lmhead_argmax_noalloc", lib().lmhead_argmax_noalloc(_ptr(w), _ptr(x), M, K, _ptr(out_index),
                                                                _ptr(out_value), _stream(x.device)))
    return out_index, out_value


def lmhead_argmax_verify(w: torch.Tensor, X: torch.Tensor, M: int, K: int, out_index: torch.Tensor | None = None,
                         out_value: torch.Tensor | None = None, ws: Workspace | None = None):
    """Batched greedy verification on a Q8_0 LM head. X: fp32 (N, ldx), row n = column n.
    Returns (index int32[N], value float32[N]) device tensors."""
    _need_cuda(w, X, out_index, out_value)
    N, ldx = X.shape
    if X.stride(1) != 1 or X.stride(0) != ldx:
        raise ValueError("X must be a contiguous (N, ldx) tensor")
    oi = out_index if out_index is not None else torch.empty(N, dtype=torch.int32, device=X.device)
    ov = out_value if out_value is not None else torch.empty(N, dtype=torch.float32, device=X.device)
    need = int(lib().lmhead_argmax_verify_workspace_bytes(M, K, N))
    ws = _ws(ws, need, X.device)
    _check("lmhead_argmax_verify", lib().lmhead_argmax_verify(_ptr(w), _ptr(X), ldx, M, K, N, ws.ptr(), ws.nbytes(),
                                                              _ptr(oi), _ptr(ov), _stream(X.device)))
    return oi, ov


def lmhead_argmax_verify_q8_1(w: torch.Tensor, xq: torch.Tensor, M: int, K: int, N: int,
                              out_index: torch.Tensor | None = None, out_value: torch.Tensor | None = None,
                              ws: Workspace | None = None):
    """Batched greedy verification on a Q8_0 LM head against N <= 8 quantized columns
    (quantize_q8_1_columns). Returns (index int32[N], value float32[N]) device tensors."""
    _need_cuda(w, xq, out_index, out_value)
    oi = out_index if out_index is not None else torch.empty(N, dtype=torch.int32, device=xq.device)
    ov = out_value if out_value is not None else torch.empty(N, dtype=torch.float32, device=xq.device)
    need = int(lib().lmhead_argmax_verify_q8_1_workspace_bytes(M, K, N))
    ws = _ws(ws, need, xq.device)
    _check("lmhead_argmax_verify_q8_1",
           lib().lmhead_argmax_verify_q8_1(_ptr(w), _ptr(xq), M, K, N, ws.ptr(), ws.nbytes(), _ptr(oi), _ptr(ov),
                                           _stream(xq.device)))
    return oi, ov


# ------------------------------------------------------------------ top-k / log-softmax / sampling
class TopK:
    """Device outputs of a top-k call: index[k] (int32), logit[k], logprob[k], lse[1]
    and, when a sampler was given, token[1] (int32)."""

    def __init__(self, k: int, device, sample: bool):
        self.index = torch.empty(k, dtype=torch.int32, device=device)
        self.logit = torch.empty(k, dtype=torch.float32, device=device)
        self.logprob = torch.empty(k, dtype=torch.float32, device=device)
        self.lse = torch.empty(1, dtype=torch.float32, device=device)
        self.token = torch.empty(1, dtype=torch.int32, device=device) if sample else None

    def _c(self) -> _TopkOut:
        return _TopkOut(_ptr(self.index), _ptr(self.logit), _ptr(self.logprob), _ptr(self.lse), _ptr(self.token))


def _sampler(sampler):
    """sampler: None or (temperature, top_p, min_p, u) with u a 1-element fp32 device tensor."""
    if sampler is None:
        return None
    T, top_p, min_p, u = sampler
    _need_cuda(u)
    if u.dtype != torch.float32 or u.numel() < 1:
        raise ValueError("u must be a float32 device tensor holding one uniform number")
    return ctypes.pointer(_Sampler(T, top_p, min_p, _ptr(u)))


def logits_topk(logits: torch.Tensor, k: int, sampler=None, ws: Workspace | None = None,
                out: TopK | None = None) -> TopK:
    """Top-k rows, log-softmax and (optionally) one sampled token of an fp32 logit
    vector on the device."""
    _need_cuda(logits)
    M = logits.numel()
    out = out if out is not None else TopK(k, logits.device, sampler is not None)
    need = int(lib().logits_topk_workspace_bytes(M))
    ws = _ws(ws, need, logits.device)
    oc = out._c()
    _check("logits_topk", lib().logits_topk(_ptr(logits), M, k, _sampler(sampler), ws.ptr(), ws.nbytes(),
                                            ctypes.byref(oc), _stream(logits.device)))
    return out


def lmhead_topk(w: torch.Tensor, x: torch.Tensor, M: int, K: int, k: int, logits: torch.Tensor | None = None,
                sampler=None, ws: Workspace | None = None, out: TopK | None = None):
    """Q8_0 LM head fused with top-k, log-softmax and sampling. Returns (TopK, logits);
    the logits stay in device memory."""
    _need_cuda(w, x, logits)
    logits = logits if logits is not None else torch.empty(M, dtype=torch.float32, device=x.device)
    out = out if out is not None else TopK(k, x.device, sampler is not None)
    need = int(lib().lmhead_topk_workspace_bytes(M, K))
    ws = _ws(ws, need, x.device)
    oc = out._c()
    _check("lmhead_topk", lib().lmhead_topk(_ptr(w), _ptr(x), M, K, k, _ptr(logits), _sampler(sampler), ws.ptr(),
                                            ws.nbytes(), ctypes.byref(oc), _stream(x.device)))
    return out, logits


# ------------------------------------------------------------------ int8 rows and products
_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


def _launch(name, gpu, *args):
    """Calls the library's `name` on GPU `gpu`'s current stream with that GPU the current
    one (kernels launch there); raises on an error status."""
    f = getattr(lib(), name)
    if torch._C._cuda_getDevice() == gpu:
        status = f(*args, torch._C._cuda_getCurrentRawStream(gpu))
    else:
        with torch.cuda.device(gpu):
            status = f(*args, torch._C._cuda_getCurrentRawStream(gpu))
    if status:
        _check(name, status)


def _int32(**values):
    """The library's 32-bit arguments would take a larger number's low 32 bits."""
    for name, v in values.items():
        if not -(1 << 31) <= v < 1 << 31:
            raise ValueError(f"{name}={v} does not fit 32 bits")


def _gpu(name, t, dtypes):
    """Index of the GPU that holds t, a tensor of one of `dtypes`."""
    if not isinstance(t, torch.Tensor) or t.get_device() < 0:
        raise ValueError(f"{name} must be a tensor on the GPU")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    return t.get_device()


def _same(name, t, dtypes, index, shape):
    """t: contiguous, of one of `dtypes` and of `shape`, on GPU `index`."""
    if isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype in dtypes and t.shape == shape and \
            t.is_contiguous():
        return
    if _gpu(name, t, dtypes) != index:
        raise ValueError(f"{name} is on GPU {t.get_device()}, the other operands on GPU {index}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _rows_of(name, t, dtypes, index, rows, width):
    """(rows, width, row stride in elements) of t, 2-D with contiguous rows of at least
    `width` on GPU `index`; rows None: any number."""
    if isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype in dtypes and t.dim() == 2:
        n, m = t.shape
        ld, one = t.stride()
        if (rows is None or n == rows) and m >= width and (one == 1 or m <= 1):
            return n, m, ld if n > 1 or ld > m else m
    if _gpu(name, t, dtypes) != index:
        raise ValueError(f"{name} is on GPU {t.get_device()}, the other operands on GPU {index}")
    if t.dim() == 2 and not ((rows is None or t.shape[0] == rows) and t.shape[1] >= width):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {'any' if rows is None else rows} rows of at least {width}")
    raise ValueError(f"{name} must be 2-D with contiguous rows")


def _scratch(ws, need, device):
    """(address, bytes, owner) of a call's workspace: the caller's, grown if need be, or one
    of the call's own, so that calls on several streams and captured graphs never share."""
    if ws is not None:
        ws.serve(need, "scratch")
        if ws.buf is not None and ws.buf.device != device:
            raise ValueError(f"the workspace is on {ws.buf.device}, the operands on {device}")
        return ws.ptr(), ws.nbytes(), ws.buf
    buf = torch.empty_strided((need,), (1,), dtype=torch.uint8, device=device)
    return buf.data_ptr(), need, buf


_F32, _I8, _U8, _I32 = (torch.float32,), (torch.int8,), (torch.uint8,), (torch.int32,)
_FLAGS = (torch.bool, torch.uint8)


def i8_bytes(M: int, K: int) -> int:
    return int(lib().qg_i8_bytes(M, K))


def pack_i8(w: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Lay out row-major int8 weights (M, K), rows at any stride, for qgemm_i8
    (uint8 buffer of i8_bytes(M, K) bytes)."""
    gpu = _gpu("w", w, _I8)
    M, K, ldw = _rows_of("w", w, _I8, gpu, None, 0)
    n = i8_bytes(M, K)
    if n == 0:
        raise ValueError(f"no int8 layout for a {M} x {K} matrix")
    if out is None:
        out = torch.empty(n, dtype=torch.uint8, device=w.device)
    _same("out", out, _U8, gpu, (n,))
    _launch("qg_pack_i8", gpu, w.data_ptr(), ldw, out.data_ptr(), M, K)
    return out


def quantize_i8_rows(x: torch.Tensor, out: torch.Tensor | None = None, scale: torch.Tensor | None = None):
    """Int8 rows of x (N, K) in fp32, fp16 or bf16, a scale each (max|x| / 127):
    tokens for qgemm_i8, or the rows of a weight matrix before pack_i8. Returns
    (q int8 (N, ldq), scale float32 (N)), ldq = K rounded up to 64, zeros beyond K."""
    gpu = _gpu("x", x, _TYPES)
    N, K, ldx = _rows_of("x", x, _TYPES, gpu, None, 0)
    kp = (K + 63) // 64 * 64
    if out is None:
        out, ldq = torch.empty_strided((N, kp), (kp, 1), dtype=torch.int8, device=x.device), kp
    else:
        ldq = _rows_of("out", out, _I8, gpu, N, kp)[2]
    if scale is None:
        scale = torch.empty_strided((N,), (1,), dtype=torch.float32, device=x.device)
    else:
        _same("scale", scale, _F32, gpu, (N,))
    _launch("qg_quantize_i8_rows", gpu, x.data_ptr(), _TYPES[x.dtype], ldx, N, K, out.data_ptr(), ldq, scale.data_ptr())
    return out, scale


def qgemm_i8_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib().qgemm_i8_workspace_bytes(M, K, N))


def qgemm_i8(w: torch.Tensor, w_scale: torch.Tensor, xq: torch.Tensor, x_scale: torch.Tensor, M: int, K: int,
             bias: torch.Tensor | None = None, Y: torch.Tensor | None = None, dtype: torch.dtype = torch.float32,
             ws: Workspace | None = None) -> torch.Tensor:
    """Y[n, m] = x_scale[n] w_scale[m] sum_k xq[n, k] wq[m, k] (+ bias[m]) for weights
    packed by pack_i8 and rows quantized by quantize_i8_rows. Returns Y (N, ldy) of
    `dtype` (fp32, fp16 or bf16) with Y[:, :M] written. Without ws, a call that needs
    a workspace (products split along K) allocates its own."""
    L = lib()
    gpu = _gpu("w", w, _U8)
    if w.numel() != L.qg_i8_bytes(M, K) or not w.is_contiguous():
        raise ValueError(f"w is not a packed {M} x {K} matrix")
    N, _, ldx = _rows_of("xq", xq, _I8, gpu, None, (K + 63) // 64 * 64)
    _same("w_scale", w_scale, _F32, gpu, (M,))
    _same("x_scale", x_scale, _F32, gpu, (N,))
    if bias is not None:
        _same("bias", bias, _F32, gpu, (M,))
    if Y is None:
        if dtype not in _TYPES:
            raise ValueError(f"no output of type {dtype}")
        ldy = (M + 3) // 4 * 4
        Y = torch.empty_strided((N, ldy), (ldy, 1), dtype=dtype, device=w.device)
    else:
        ldy = _rows_of("Y", Y, _TYPES, gpu, N, M)[2]
        dtype = Y.dtype
    need = L.qgemm_i8_workspace_bytes(M, K, N)
    wp, wb, keep = _scratch(ws, need, w.device) if need else (None, 0, None)
    _launch("qgemm_i8", gpu, w.data_ptr(), w_scale.data_ptr(), xq.data_ptr(), ldx, x_scale.data_ptr(),
            None if bias is None else bias.data_ptr(), Y.data_ptr(), _TYPES[dtype], ldy, M, K, N, wp, wb)
    return Y


# ------------------------------------------------------------------ beam search
class BeamSelection:
    """Device outputs of logits_beam_select, (batch, n) each: token and parent (int32),
    score (float32), finished (bool) and, if lengths were given, length (int32)."""

    def __init__(self, batch: int, n: int, device, length: bool):
        whole = torch.empty((3 if length else 2, batch, n), dtype=torch.int32, device=device).unbind()
        self.token, self.parent = whole[:2]
        self.length = whole[2] if length else None
        self.score = torch.empty_strided((batch, n), (n, 1), dtype=torch.float32, device=device)
        self.finished = torch.empty_strided((batch, n), (n, 1), dtype=torch.bool, device=device)


def logits_beam_select(logits: torch.Tensor, score: torch.Tensor, n: int, finished: torch.Tensor | None = None,
                       length: torch.Tensor | None = None, eos: int = -1, length_penalty: float = 0.0,
                       out: BeamSelection | None = None, ws: Workspace | None = None) -> BeamSelection:
    """The n best continuations of each batch item over its beams and the vocabulary.
    logits (batch * beams, vocab), rows at any stride, fp32, fp16 or bf16; score (batch,
    beams) float32; finished (batch, beams) bool; length (batch, beams) int32. `out` may
    hold score, finished and length themselves when n is the number of beams (a step
    in place). Ranking and special values as include/qgemv.h states."""
    L = lib()
    gpu = _gpu("logits", logits, _TYPES)
    if score.dim() != 2:
        raise ValueError("score must be (batch, beams)")
    shape = score.shape
    B, W = shape
    _int32(beams=W, n=n, eos=eos)
    _same("score", score, _F32, gpu, shape)
    _, V, ld = _rows_of("logits", logits, _TYPES, gpu, B * W, 0)
    if finished is not None:
        _same("finished", finished, _FLAGS, gpu, shape)
    if length is not None:
        _same("length", length, _I32, gpu, shape)
    if out is None:
        out = BeamSelection(B, n, logits.device, length is not None)
    else:
        for name, types in (("token", _I32), ("parent", _I32), ("score", _F32), ("finished", _FLAGS), ("length", _I32)):
            t = getattr(out, name)
            if t is not None:
                _same("out." + name, t, types, gpu, (B, n))
    xt = _TYPES[logits.dtype]
    wp, wb, keep = _scratch(ws, L.logits_beam_select_workspace_bytes(xt, B, W, V, n), logits.device)
    ci = _BeamIn(logits.data_ptr(), xt, ld, B, W, V, score.data_ptr(), _ptr(finished), _ptr(length), length_penalty, eos)
    co = _BeamOut(_ptr(out.token), _ptr(out.parent), _ptr(out.score), _ptr(out.finished), _ptr(out.length))
    _launch("logits_beam_select", gpu, ctypes.byref(ci), n, wp, wb, ctypes.byref(co))
    return out


def _row_pieces(name, shape, strides, eb):
    """(row stride, piece stride, pieces, bytes of a piece), strides in bytes, of a tensor
    whose rows (first dimension) are equally spaced contiguous pieces."""
    span, dims = 1, [(n, st) for n, st in zip(shape[1:], strides[1:]) if n != 1]
    while dims and dims[-1][1] == span:
        span *= dims.pop()[0]
    outer, step = 1, 0
    while dims:
        n, st = dims.pop()
        if outer > 1 and st != outer * step:
            raise ValueError(f"{name}: a row must be equally spaced contiguous pieces, got strides {strides}")
        step = step if outer > 1 else st
        outer *= n
    return strides[0] * eb, step * eb, outer, span * eb


def _moves(i, s, d, B, W, n):
    """The last six fields of a qg_beam_state for state i moved from s to d, or None if it
    holds nothing."""
    if s.dim() < 1 or s.shape[0] != B * W or d.dim() != s.dim() or d.shape[0] != B * n or d.shape[1:] != s.shape[1:]:
        raise ValueError(f"state {i}: shapes {tuple(s.shape)} and {tuple(d.shape)} for {B} x {W} beams and {n} parents")
    if d.dtype != s.dtype:
        raise ValueError(f"out[{i}] must be {s.dtype}, not {d.dtype}")
    if s.numel() == 0:  # nothing cached yet
        return None
    eb = s.element_size()
    sr, so, outer, span = _row_pieces(f"states[{i}]", s.shape, s.stride(), eb)
    dr, do, outer_d, span_d = _row_pieces(f"out[{i}]", d.shape, d.stride(), eb)
    if (outer, span) != (outer_d, span_d):
        # pieces of the finer of the two cuts
        fine = min(span, span_d)
        if max(span, span_d) % fine or (outer != 1 and outer_d != 1):
            raise ValueError(f"state {i}: rows of state and result are cut into pieces that do not match")
        if span > fine:
            so, outer, span = fine, outer_d, fine
        else:
            do = fine
    return sr, dr, so, do, outer, span


def beam_reorder(states, parent: torch.Tensor, out=None):
    """Rows of every state follow their parents: row b * n + j of each result is row
    b * beams + parent[b, j] of the state (first dimension batch * beams; parent int32
    (batch, n); a parent outside [0, beams) leaves the result's row as it was). In place
    without `out` (then n == beams), else into the tensors of `out`. States may be
    views (a cache's filled part) and of several shapes and types; launched in groups of
    BEAM_MAX_STATES, after all of them are checked: a refused call moves nothing.
    Returns the list of results."""
    states = list(states)
    results = states if out is None else list(out)
    if not states or len(results) != len(states):
        raise ValueError("no states given" if not states else f"{len(results)} results for {len(states)} states")
    gpu = _gpu("parent", parent, _I32)
    if parent.dim() != 2 or not parent.is_contiguous():
        raise ValueError("parent must be (batch, n) and contiguous")
    B, n = parent.shape
    first = states[0]
    if not isinstance(first, torch.Tensor) or not B or not n or first.dim() < 1 or first.shape[0] % B:
        raise ValueError(f"{tuple(parent.shape)} parents do not fit the first state")
    W = first.shape[0] // B
    _int32(beams=W, n=n)
    # states that look alike (a model's layers) are cut into pieces once
    fields, seen, moves = [], None, None
    for i, s in enumerate(states):
        d = results[i]
        if not isinstance(s, torch.Tensor) or s.get_device() != gpu:
            raise ValueError(f"states[{i}] must be a tensor on GPU {gpu}")
        look = (s.shape, s.stride(), s.dtype)
        if d is not s:
            if not isinstance(d, torch.Tensor) or d.get_device() != gpu:
                raise ValueError(f"out[{i}] must be a tensor on GPU {gpu}")
            look += (d.shape, d.stride(), d.dtype)
        if look != seen:
            moves, seen = _moves(i, s, d, B, W, n), look
        if moves is not None:
            p = s.data_ptr()
            fields += (p, p if d is s else d.data_ptr())
            fields += moves
    words = array.array("q", fields)
    at, count = words.buffer_info()[0], len(words) // 8
    groups = range(0, count, BEAM_MAX_STATES)
    if len(groups) > 1:  # (a group's own call checks it, too late for the groups before it)
        src, dst = fields[0::8], fields[1::8]
        if len(set(dst)) != count or not {s for s, d in zip(src, dst) if s != d}.isdisjoint(dst):
            raise ValueError("two states share a result, or one is another's result")
        for k in groups:
            _check("qg_beam_reorder", lib().qg_beam_reorder_check(at + k * 64, min(BEAM_MAX_STATES, count - k),
                                                                  parent.data_ptr(), B, W, n))
    for k in groups:
        _launch("qg_beam_reorder", gpu, at + k * 64, min(BEAM_MAX_STATES, count - k), parent.data_ptr(), B, W, n)
    return results


# ------------------------------------------------------------------ 8-bit floating-point rows and products
_F8 = (torch.float8_e4m3fn,)


def f8_bytes(M: int, K: int, experts: int = 1) -> int:
    return int(lib().qg_f8_bytes(M, K, experts))


def pack_f8(w: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Lay out e4m3 weights (float8_e4m3fn) for qgemm_f8, one matrix (M, K), or for
    qgemm_f8_grouped, one per expert (experts, M, K); rows contiguous, at any strides.
    Returns a uint8 buffer of f8_bytes(M, K, experts) bytes."""
    gpu = _gpu("w", w, _F8)
    if w.dim() not in (2, 3):
        raise ValueError("w must be (M, K) or (experts, M, K)")
    E = w.shape[0] if w.dim() == 3 else 1
    M, K = w.shape[-2:]
    n = f8_bytes(M, K, E)
    if n == 0:
        raise ValueError(f"no e4m3 layout for {E} matrices of {M} x {K}")
    if K > 1 and w.stride(-1) != 1:
        raise ValueError("w must have contiguous rows")
    ldw = max(w.stride(-2), K) if M > 1 else K
    each = w.stride(0) if E > 1 else 0
    if M > 1 and w.stride(-2) < K or E > 1 and each < (M - 1) * ldw + K:
        raise ValueError(f"the rows or matrices of w overlap (strides {w.stride()})")
    if out is None:
        out = torch.empty(n, dtype=torch.uint8, device=w.device)
    _same("out", out, _U8, gpu, (n,))
    _launch("qg_pack_f8", gpu, w.data_ptr(), ldw, each, out.data_ptr(), M, K, E)
    return out


def quantize_f8_rows(x: torch.Tensor, gated: bool = False, count: torch.Tensor | None = None,
                     out: torch.Tensor | None = None, scale: torch.Tensor | None = None):
    """E4m3 rows of x in fp32, fp16 or bf16 with a float32 scale per 128 values (max / 448):
    of x (N, K), or with `gated` of silu(g) * u for x (N, 2 K) = g beside u. Returns
    (q float8_e4m3fn (N, ldq), scale (N, lds)), ldq = K rounded up to 128 and lds = blocks
    rounded up to 4, zeros beyond K. count: an int32 tensor of one element on the GPU; only the
    first `count` rows are done."""
    gpu = _gpu("x", x, _TYPES)
    N, W, ldx = _rows_of("x", x, _TYPES, gpu, None, 0)
    if gated and W % 2:
        raise ValueError(f"x has {W} columns, not two halves")
    K = W // 2 if gated else W
    nb = (K + 127) // 128
    kp, sp = nb * 128, (nb + 3) // 4 * 4
    if count is not None:
        _same("count", count, _I32, gpu, (1,))
    if out is None:
        out, ldq = torch.empty_strided((N, kp), (kp, 1), dtype=torch.float8_e4m3fn, device=x.device), kp
    else:
        ldq = _rows_of("out", out, _F8, gpu, N, kp)[2]
    if scale is None:
        scale, lds = torch.empty_strided((N, sp), (sp, 1), dtype=torch.float32, device=x.device), sp
    else:
        lds = _rows_of("scale", scale, _F32, gpu, N, sp)[2]
    _launch("qg_quantize_f8_rows", gpu, x.data_ptr(), _TYPES[x.dtype], ldx, 1 if gated else 0,
            None if count is None else count.data_ptr(), N, K, out.data_ptr(), ldq, scale.data_ptr(), lds)
    return out, scale


def qgemm_f8_workspace_bytes(M: int, K: int, N: int, dtype: torch.dtype = torch.float32) -> int:
    return int(lib().qgemm_f8_workspace_bytes(M, K, N, _TYPES[dtype]))


def _f8_operands(L, w, w_scale, xq, x_scale, M, K, experts, bias, shape):
    """(gpu, rows of xq, ldx, ldxs) of a product's checked inputs; shape: () or (experts,)."""
    gpu = _gpu("w", w, _U8)
    if w.numel() != L.qg_f8_bytes(M, K, experts) or not w.is_contiguous():
        raise ValueError(f"w is not {experts} packed {M} x {K} matrices" if shape else f"w is not a packed {M} x {K} matrix")
    nb = (K + 127) // 128
    X, _, ldx = _rows_of("xq", xq, _F8, gpu, None, nb * 128)
    ldxs = _rows_of("x_scale", x_scale, _F32, gpu, X, (nb + 3) // 4 * 4)[2]
    _same("w_scale", w_scale, _F32, gpu, shape + ((M + 127) // 128, nb))
    if bias is not None:
        _same("bias", bias, _F32, gpu, shape + (M,))
    return gpu, X, ldx, ldxs


def _product_rows(Y, dtype, gpu, N, M, device):
    """(Y, type, ldy) of a product's result, allocated if need be."""
    if Y is not None:
        return Y, _TYPES[Y.dtype] if Y.dtype in _TYPES else -1, _rows_of("Y", Y, _TYPES, gpu, N, M)[2]
    if dtype not in _TYPES:
        raise ValueError(f"no output of type {dtype}")
    ldy = (M + 3) // 4 * 4
    return torch.empty_strided((N, ldy), (ldy, 1), dtype=dtype, device=device), _TYPES[dtype], ldy


def qgemm_f8(w: torch.Tensor, w_scale: torch.Tensor, xq: torch.Tensor, x_scale: torch.Tensor, M: int, K: int,
             bias: torch.Tensor | None = None, Y: torch.Tensor | None = None, dtype: torch.dtype = torch.float32,
             ws: Workspace | None = None) -> torch.Tensor:
    """Y[n, m] = sum_b x_scale[n, b] w_scale[m // 128, b] sum_{k in b} xq[n, k] wq[m, k] (+ bias[m])
    over blocks b of 128, for weights packed by pack_f8 (w_scale (ceil(M / 128), ceil(K /
    128))) and rows quantized by quantize_f8_rows. Returns Y (N, ldy) of `dtype` (fp32, fp16 or
    bf16) with Y[:, :M] written. Without ws, a call that needs a workspace (products split
    along K) allocates its own."""
    L = lib()
    gpu, N, ldx, ldxs = _f8_operands(L, w, w_scale, xq, x_scale, M, K, 1, bias, ())
    Y, yt, ldy = _product_rows(Y, dtype, gpu, N, M, w.device)
    need = L.qgemm_f8_workspace_bytes(M, K, N, yt)
    wp, wb, keep = _scratch(ws, need, w.device) if need else (None, 0, None)
    _launch("qgemm_f8", gpu, w.data_ptr(), w_scale.data_ptr(), xq.data_ptr(), ldx, x_scale.data_ptr(), ldxs,
            None if bias is None else bias.data_ptr(), Y.data_ptr(), yt, ldy, M, K, N, wp, wb)
    return Y


def qgemm_f8_grouped(w: torch.Tensor, w_scale: torch.Tensor, xq: torch.Tensor, x_scale: torch.Tensor, M: int, K: int,
                     offsets: torch.Tensor, row: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                     Y: torch.Tensor | None = None, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """Products grouped by expert: rows offsets[e] .. offsets[e + 1] of Y (int32, ascending)
    are those of qgemm_f8 with expert e's matrix (w of pack_f8 with experts, w_scale (experts,
    ceil(M / 128), ceil(K / 128)), bias (experts, M)). Row r of Y comes from row row[r] of xq (int32), or
    from row r. Returns Y (rows, ldy) with Y[offsets[0]:offsets[-1], :M] written; `rows` is
    that of `row`, or of xq."""
    L = lib()
    gpu = _gpu("offsets", offsets, _I32)
    if offsets.dim() != 1 or offsets.numel() < 2 or not offsets.is_contiguous():
        raise ValueError("offsets must be contiguous, one more than there are experts")
    E = offsets.numel() - 1
    on, X, ldx, ldxs = _f8_operands(L, w, w_scale, xq, x_scale, M, K, E, bias, (E,))
    if on != gpu:
        raise ValueError(f"offsets is on GPU {gpu}, the other operands on GPU {on}")
    N = X
    if row is not None:
        N = row.numel()
        _same("row", row, _I32, gpu, (N,))
    Y, yt, ldy = _product_rows(Y, dtype, gpu, N, M, w.device)
    p = _F8Grouped(w.data_ptr(), w_scale.data_ptr(), xq.data_ptr(), ldx, x_scale.data_ptr(), ldxs, X, _ptr(row),
                   offsets.data_ptr(), _ptr(bias), Y.data_ptr(), yt, ldy, M, K, E, N)
    _launch("qgemm_f8_grouped", gpu, ctypes.byref(p))
    return Y


# ------------------------------------------------------------------ experts
class ExpertSelection:
    """Device outputs of logits_expert_select: expert (int32), weight (float32) and position
    (int32), (N, k) each, row (int32, N * k) and offsets (int32, experts + 1)."""

    def __init__(self, N: int, E: int, k: int, device):
        self.expert, self.position = torch.empty_strided((2, N, k), (N * k, k, 1), dtype=torch.int32, device=device).unbind()
        self.weight = torch.empty_strided((N, k), (k, 1), dtype=torch.float32, device=device)
        self.row = torch.empty_strided((N * k,), (1,), dtype=torch.int32, device=device)
        self.offsets = torch.empty_strided((E + 1,), (1,), dtype=torch.int32, device=device)


def logits_expert_select(logits: torch.Tensor, k: int, normalize: bool = False, scale: float = 1.0,
                         out: ExpertSelection | None = None, ws: Workspace | None = None) -> ExpertSelection:
    """The k best of each row's expert logits (N, E) in fp32, fp16 or bf16, rows at any
    stride, their softmax weights (over all experts, or with `normalize` over the k taken, times
    `scale`), and the rows in the experts' order: what qgemm_f8_grouped (offsets, row) and
    expert_combine (position, weight) take. Ranking and special values as include/qgemv.h states."""
    L = lib()
    gpu = _gpu("logits", logits, _TYPES)
    N, E, ld = _rows_of("logits", logits, _TYPES, gpu, None, 0)
    _int32(experts=E, k=k)
    if out is None:
        if not (1 <= k <= min(E, EXPERTS_MAX_K) and N >= 1):
            raise ValueError(f"k={k} for logits of shape {tuple(logits.shape)}: it is at most the experts and {EXPERTS_MAX_K}")
        out = ExpertSelection(N, E, k, logits.device)
    else:
        for name, types, shape in (("expert", _I32, (N, k)), ("weight", _F32, (N, k)), ("position", _I32, (N, k)),
                                   ("row", _I32, (N * k,)), ("offsets", _I32, (E + 1,))):
            _same("out." + name, getattr(out, name), types, gpu, shape)
    need = L.logits_expert_select_workspace_bytes(N, E, k)
    wp, wb, keep = _scratch(ws, need, logits.device) if need else (None, 0, None)
    co = _ExpertsOut(out.expert.data_ptr(), out.weight.data_ptr(), out.position.data_ptr(), out.row.data_ptr(),
                     out.offsets.data_ptr())
    _launch("logits_expert_select", gpu, logits.data_ptr(), _TYPES[logits.dtype], ld, N, E, k, 1 if normalize else 0, scale, wp,
            wb, ctypes.byref(co))
    return out


def expert_combine(Y: torch.Tensor, position: torch.Tensor, weight: torch.Tensor, add: torch.Tensor | None = None,
                   out: torch.Tensor | None = None, dtype: torch.dtype | None = None, M: int | None = None) -> torch.Tensor:
    """out[n] = (add[n] +) sum_j weight[n, j] Y[position[n, j]] over the first M (default all) columns of
    Y, in float32, rounded once to `dtype` (default: that of add, or of Y). position int32 and
    weight float32 (N, k); positions outside Y are skipped. out may be add itself."""
    gpu = _gpu("Y", Y, _TYPES)
    R, W, ldy = _rows_of("Y", Y, _TYPES, gpu, None, M or 0)
    M = W if M is None else M
    if position.dim() != 2:
        raise ValueError("position must be (N, k)")
    N, k = position.shape
    _int32(k=k)
    _same("position", position, _I32, gpu, (N, k))
    _same("weight", weight, _F32, gpu, (N, k))
    if out is not None:
        dtype = out.dtype
    elif dtype is None:
        dtype = Y.dtype if add is None else add.dtype
    if dtype not in _TYPES:
        raise ValueError(f"no output of type {dtype}")
    ldadd = 0 if add is None else _rows_of("add", add, (dtype,), gpu, N, M)[2]
    if out is None:
        out, ldo = torch.empty_strided((N, M), (M, 1), dtype=dtype, device=Y.device), M
    else:
        ldo = _rows_of("out", out, _TYPES, gpu, N, M)[2]
    _launch("qg_expert_combine", gpu, Y.data_ptr(), _TYPES[Y.dtype], ldy, R, position.data_ptr(), weight.data_ptr(), k,
            _ptr(add), ldadd, out.data_ptr(), _TYPES[dtype], ldo, N, M)
    return out
