"""Python binding of ``libshampoo.so``: the batched block preconditioner step of
block-diagonal Shampoo on MI355X (gfx950).

Argument marshalling only.  Every step of the path runs in the library's HIP
kernels; torch supplies device memory (``data_ptr``) and the current stream.
The functions keep the C names (``shampoo_inverse_root`` ...).  Importing the
package loads the library and raises ImportError when it is missing: there is
no fallback.
"""

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libshampoo.so")

# ---------------------------------------------------------------------------
# enums (include/shampoo.h)
# ---------------------------------------------------------------------------
OK, E_INVALID, E_UNSUPPORTED, E_WORKSPACE, E_HIP, E_NONFINITE = range(6)
STATUS_NAMES = {0: "OK", 1: "E_INVALID", 2: "E_UNSUPPORTED", 3: "E_WORKSPACE", 4: "E_HIP", 5: "E_NONFINITE"}
F32, F16, BF16, F64, E4M3, E5M2 = 0, 1, 2, 3, 4, 5
CN, NDB, CHEBYSHEV = 0, 1, 2
SCALE_FROBENIUS, SCALE_POWER = 0, 1
CHEB_CLENSHAW, CHEB_PS = 0, 1
GRAFT_SGD, GRAFT_MOMENTUM, GRAFT_ADAM, GRAFT_NONE = 0, 1, 2, 3
FLAG_NONFINITE, FLAG_ZERO_SCALE, FLAG_PI_FALLBACK, FLAG_RECOMPUTED_F64, FLAG_KEPT_PREVIOUS = 1, 2, 4, 8, 16
FLAG_RESIDUAL = 32
REDUCTIONS = {"none": 0, "sum": 1, "mean": 2}
FORMATS_F8 = {"e4m3": E4M3, "e5m2": E5M2}
FALLBACKS = {"none": 0, "keep": 1, "f64": 2}

METHODS = {"cn": CN, "ndb": NDB, "chebyshev": CHEBYSHEV}
SCALINGS = {"frobenius": SCALE_FROBENIUS, "power": SCALE_POWER}
CHEB_EVALS = {"clenshaw": CHEB_CLENSHAW, "ps": CHEB_PS}
DTYPES = {"f32": F32, "f16": F16, "bf16": BF16, "f64": F64}
GRAFTS = {"sgd": GRAFT_SGD, "momentum": GRAFT_MOMENTUM, "adam": GRAFT_ADAM, "none": GRAFT_NONE}


class ShampooError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__("%s: %s" % (STATUS_NAMES.get(status, status), msg))
        self.status = status


# ---------------------------------------------------------------------------
# ctypes mirrors of the C structs
# ---------------------------------------------------------------------------
class Block(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("param", "brow", "bcol", "row0", "col0", "rows", "cols", "B")]


class Matrix(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("ld", ctypes.c_int64)]


class Param(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("ld", ctypes.c_int64), ("first_block", ctypes.c_int64)]


class RootOptsC(ctypes.Structure):
    _fields_ = [("method", ctypes.c_int32), ("scaling", ctypes.c_int32), ("compute", ctypes.c_int32),
                ("iters", ctypes.c_int32), ("iters2", ctypes.c_int32), ("pi_vectors", ctypes.c_int32),
                ("pi_iters", ctypes.c_int32), ("cheb_degree", ctypes.c_int32),
                ("cheb_points", ctypes.c_int32), ("cheb_eval", ctypes.c_int32),
                ("eps", ctypes.c_double), ("cheb_eps", ctypes.c_double),
                ("pi_start_dev", ctypes.c_void_p), ("tol", ctypes.c_double),
                ("residual_out_dev", ctypes.c_void_p), ("residual_bound", ctypes.c_double)]


class StepArgsC(ctypes.Structure):
    _fields_ = [("nparams", ctypes.c_int32), ("B", ctypes.c_int32), ("nblk", ctypes.c_int64),
                ("params_dev", ctypes.c_void_p), ("table_dev", ctypes.c_void_p),
                ("g_dt", ctypes.c_int32), ("p", ctypes.c_int32),
                ("stats_dt", ctypes.c_int32), ("fallback", ctypes.c_int32),
                ("LR", ctypes.c_void_p), ("roots", ctypes.c_void_p),
                ("beta2", ctypes.c_double), ("recompute_roots", ctypes.c_int32),
                ("root", RootOptsC),
                ("graft", ctypes.c_int32), ("graft_blockwise", ctypes.c_int32),
                ("lr", ctypes.c_float), ("momentum", ctypes.c_float),
                ("beta1", ctypes.c_float), ("graft_beta2", ctypes.c_float), ("graft_eps", ctypes.c_float),
                ("t", ctypes.c_int32), ("flags_dev", ctypes.c_void_p), ("dstack", ctypes.c_void_p),
                ("ws", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t), ("table_host", ctypes.c_void_p),
                ("precond_dt", ctypes.c_int32)]


class XentArgsC(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("targets", ctypes.c_void_p),
                ("row_scale", ctypes.c_void_p), ("loss", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("dhidden", ctypes.c_void_p), ("dweight", ctypes.c_void_p),
                ("ld_hidden", ctypes.c_int64), ("ld_weight", ctypes.c_int64),
                ("ld_dhidden", ctypes.c_int64), ("ld_dweight", ctypes.c_int64),
                ("N", ctypes.c_int64), ("V", ctypes.c_int64), ("d", ctypes.c_int64),
                ("ignore_index", ctypes.c_int64), ("panel_rows", ctypes.c_int64),
                ("dt", ctypes.c_int32), ("weight_dt", ctypes.c_int32), ("dweight_dt", ctypes.c_int32),
                ("logits_dt", ctypes.c_int32), ("reduction", ctypes.c_int32),
                ("accumulate", ctypes.c_int32), ("scale", ctypes.c_float),
                ("ws", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t)]


EXPORTS = [
    "shampoo_version", "shampoo_last_error", "shampoo_plan_blocks", "shampoo_pack_blocks",
    "shampoo_unpack_blocks", "shampoo_update_stats", "shampoo_inverse_root_workspace",
    "shampoo_inverse_root", "shampoo_inverse_root_noalloc", "shampoo_precondition_workspace",
    "shampoo_precondition",
    "shampoo_step_workspace", "shampoo_step", "shampoo_check_flags", "shampoo_timing_enable",
    "shampoo_timing_read", "shampoo_mfma_peak", "shampoo_quantize_f8", "shampoo_matmul_f8_workspace",
    "shampoo_matmul_f8", "shampoo_linear_xent_workspace", "shampoo_linear_xent",
]


def _load():
    # torch is loaded first so that the library binds to torch's HIP runtime:
    # both runtimes carry the soname libamdhip64.so.7, and whichever is loaded
    # first serves the whole process.
    import torch  # noqa: F401
    if not os.path.exists(LIB_PATH):
        raise ImportError("libshampoo.so is not built (%s); run `python -m matrix_inverse_roots_amd.build` "
                          "or __graft_entry__.build()" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    P = ctypes.POINTER
    sig = {
        "shampoo_version": ([], ctypes.c_char_p),
        "shampoo_last_error": ([], ctypes.c_char_p),
        "shampoo_plan_blocks": ([vp, vp, i32, vp, P(i64)], ctypes.c_int),
        "shampoo_pack_blocks": ([vp, i32, vp, i64, i32, ctypes.c_int, vp, vp, vp], ctypes.c_int),
        "shampoo_unpack_blocks": ([vp, vp, i64, i32, vp, i32, vp], ctypes.c_int),
        "shampoo_update_stats": ([vp, vp, ctypes.c_int, i64, i32, vp, ctypes.c_int, ctypes.c_double, vp],
                                 ctypes.c_int),
        "shampoo_inverse_root_workspace": ([i64, i32, i32, P(RootOptsC), P(sz)], ctypes.c_int),
        "shampoo_inverse_root": ([vp, vp, ctypes.c_int, i64, i32, i32, P(RootOptsC), vp, vp, vp, vp, sz, vp],
                                 ctypes.c_int),
        "shampoo_inverse_root_noalloc": ([vp, vp, ctypes.c_int, i64, i32, i32, P(RootOptsC), vp, vp, vp, vp],
                                         ctypes.c_int),
        "shampoo_precondition_workspace": ([i64, i32, ctypes.c_int, P(sz)], ctypes.c_int),
        "shampoo_precondition": ([vp, ctypes.c_int, vp, ctypes.c_int, i64, i32, vp, vp, sz, vp], ctypes.c_int),
        "shampoo_step_workspace": ([P(StepArgsC), P(sz)], ctypes.c_int),
        "shampoo_step": ([P(StepArgsC), vp], ctypes.c_int),
        "shampoo_check_flags": ([vp, i64, vp], ctypes.c_int),
        "shampoo_timing_enable": ([i32], ctypes.c_int),
        "shampoo_timing_read": ([vp, i32, P(i32)], ctypes.c_int),
        "shampoo_mfma_peak": ([ctypes.c_int, vp, vp, P(ctypes.c_double)], ctypes.c_int),
        "shampoo_quantize_f8": ([vp, ctypes.c_int, i64, i64, i64, i64, i64, ctypes.c_int, i32, vp, vp, vp, vp, vp],
                                ctypes.c_int),
        "shampoo_matmul_f8_workspace": ([i64, i64, i64, i64, P(sz)], ctypes.c_int),
        "shampoo_matmul_f8": ([vp, ctypes.c_int, vp, i32, vp, ctypes.c_int, vp, i32, i64, i64, i64, i64, vp,
                               ctypes.c_int, vp, sz, vp], ctypes.c_int),
        "shampoo_linear_xent_workspace": ([P(XentArgsC), P(sz)], ctypes.c_int),
        "shampoo_linear_xent": ([P(XentArgsC), vp], ctypes.c_int),
    }
    for name in EXPORTS:
        f = getattr(lib, name)
        f.argtypes, f.restype = sig[name]
    return lib


lib = _load()


def _check(status):
    if status != OK:
        raise ShampooError(status, lib.shampoo_last_error().decode())


def version():
    return lib.shampoo_version().decode()


# ---------------------------------------------------------------------------
# torch plumbing
# ---------------------------------------------------------------------------
def _torch():
    import torch
    return torch


def _dtype_code(t):
    torch = _torch()
    m = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16, torch.float64: F64}
    if t.dtype not in m:
        raise TypeError("unsupported dtype %s" % t.dtype)
    return m[t.dtype]


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t, name):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


@dataclass
class RootOpts:
    """Inverse-root options (mirrors shampoo_root_opts)."""
    method: str = "cn"            # "cn" | "ndb" | "chebyshev"
    scaling: str = "frobenius"    # "frobenius" | "power"
    compute: str = "f32"          # "f32" | "f16" | "f64"
    iters: int = 20
    iters2: int = 0
    pi_vectors: int = 16
    pi_iters: int = 10
    cheb_degree: int = 16
    cheb_points: int = 0
    cheb_eval: str = "clenshaw"   # "clenshaw" | "ps" (Paterson-Stockmeyer split)
    eps: float = 0.0
    cheb_eps: Optional[float] = None   # defaults to eps
    pi_start: object = None       # device float32 [pi_vectors, B]
    tol: float = 0.0              # CN / NDB: stop once ||M - I||_F <= tol (0: run iters; f16 checks the half copy)
    residual_out: object = None   # device float32 [n]: ||X^p A_s - I||_F / sqrt(v) per matrix
    residual_bound: float = 0.0   # > 0: FLAG_RESIDUAL where the residual exceeds it

    def c(self):
        return RootOptsC(METHODS[self.method], SCALINGS[self.scaling], DTYPES[self.compute],
                         int(self.iters), int(self.iters2), int(self.pi_vectors), int(self.pi_iters),
                         int(self.cheb_degree), int(self.cheb_points), CHEB_EVALS[self.cheb_eval], float(self.eps),
                         float(self.eps if self.cheb_eps is None else self.cheb_eps),
                         None if self.pi_start is None else self.pi_start.data_ptr(), float(self.tol),
                         None if self.residual_out is None else self.residual_out.data_ptr(),
                         float(self.residual_bound))


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------
def shampoo_plan_blocks(shapes2d, block_sizes):
    """Block table (host int32 numpy [nblk, 8]) for 2-D shapes and block sizes."""
    shapes = np.ascontiguousarray(np.asarray(shapes2d, dtype=np.int64).reshape(-1, 2))
    bs = np.ascontiguousarray(np.asarray(block_sizes, dtype=np.int32).reshape(-1))
    if shapes.shape[0] != bs.shape[0]:
        raise ValueError("one block size per parameter")
    n = ctypes.c_int64(0)
    _check(lib.shampoo_plan_blocks(shapes.ctypes.data, bs.ctypes.data, shapes.shape[0], None, ctypes.byref(n)))
    out = np.zeros((n.value, 8), dtype=np.int32)
    cap = ctypes.c_int64(n.value)
    if n.value:
        _check(lib.shampoo_plan_blocks(shapes.ctypes.data, bs.ctypes.data, shapes.shape[0], out.ctypes.data,
                                       ctypes.byref(cap)))
    return out


def table_to_device(table, device="cuda"):
    torch = _torch()
    return torch.from_numpy(np.ascontiguousarray(table, dtype=np.int32)).to(device)


def matrices_to_device(mats, device="cuda"):
    """Device array of shampoo_matrix for a list of 2-D row-major tensors."""
    torch = _torch()
    rows = []
    for m in mats:
        if m.dim() != 2 or m.stride(1) != 1:
            raise ValueError("matrices must be 2-D with unit column stride")
        rows.append([m.data_ptr(), m.shape[0], m.shape[1], m.stride(0)])
    return torch.tensor(rows, dtype=torch.int64).reshape(-1, 4).to(device)


def shampoo_pack_blocks(mats, table_dev, B, stack, stack_t=None, stream=None):
    """Pack 2-D matrices (list of device tensors of one dtype) into [nblk, B, B]."""
    _dev(stack, "stack")
    _dev(stack_t, "stack_t")
    desc = matrices_to_device(mats, stack.device)
    nblk = table_dev.shape[0]
    _check(lib.shampoo_pack_blocks(_ptr(desc), len(mats), _ptr(table_dev), nblk, int(B), _dtype_code(stack),
                                   _ptr(stack), _ptr(stack_t), _stream(stream)))
    return desc


def shampoo_unpack_blocks(stack, table_dev, B, outs, stream=None):
    _dev(stack, "stack")
    desc = matrices_to_device(outs, stack.device)
    _check(lib.shampoo_unpack_blocks(_ptr(stack), _ptr(table_dev), table_dev.shape[0], int(B), _ptr(desc),
                                     len(outs), _stream(stream)))
    return desc


def shampoo_update_stats(gstack, gstack_t, LR, beta2, stream=None):
    """L, R (the two halves of LR, float32 or float64) updated from a block
    stack and its transpose."""
    for t, n in ((gstack, "gstack"), (gstack_t, "gstack_t"), (LR, "LR")):
        _dev(t, n)
    nblk, B = gstack.shape[0], gstack.shape[1]
    _check(lib.shampoo_update_stats(_ptr(gstack), _ptr(gstack_t), _dtype_code(gstack), nblk, B, _ptr(LR),
                                    _dtype_code(LR), float(beta2), _stream(stream)))


def shampoo_inverse_root_workspace(n, B, p, opts):
    b = ctypes.c_size_t(0)
    oc = opts.c()
    _check(lib.shampoo_inverse_root_workspace(int(n), int(B), int(p), ctypes.byref(oc), ctypes.byref(b)))
    return b.value


def shampoo_inverse_root(inp, out, p, opts, valid=None, scale_out=None, flags=None, ws=None, stream=None):
    """out = (inp + eps I)^(-1/p) for a stack inp [n, B, B] (float32 or float64)."""
    torch = _torch()
    for t, nm in ((inp, "inp"), (out, "out"), (valid, "valid"), (scale_out, "scale_out"), (flags, "flags")):
        _dev(t, nm)
    n, B = inp.shape[0], inp.shape[1]
    if out.dtype != inp.dtype or out.shape != inp.shape:
        raise ValueError("out must match inp")
    if ws is None:
        nb = shampoo_inverse_root_workspace(n, B, p, opts)
        ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=inp.device)
    oc = opts.c()
    _check(lib.shampoo_inverse_root(_ptr(inp), _ptr(out), _dtype_code(inp), n, B, int(p), ctypes.byref(oc),
                                    _ptr(valid), _ptr(scale_out), _ptr(flags), _ptr(ws), ws.numel(),
                                    _stream(stream)))
    return out


def shampoo_inverse_root_noalloc(inp, out, p, opts, valid=None, scale_out=None, flags=None, stream=None):
    """shampoo_inverse_root with the library's own fixed device scratch
    (no workspace, no allocation); calls on one device must not overlap."""
    for t, nm in ((inp, "inp"), (out, "out"), (valid, "valid"), (scale_out, "scale_out"), (flags, "flags")):
        _dev(t, nm)
    n, B = inp.shape[0], inp.shape[1]
    if out.dtype != inp.dtype or out.shape != inp.shape:
        raise ValueError("out must match inp")
    oc = opts.c()
    _check(lib.shampoo_inverse_root_noalloc(_ptr(inp), _ptr(out), _dtype_code(inp), n, B, int(p), ctypes.byref(oc),
                                            _ptr(valid), _ptr(scale_out), _ptr(flags), _stream(stream)))
    return out


def shampoo_precondition(roots, gstack, dstack, ws=None, stream=None):
    """dstack = Lr G Rr per block; roots float32 or float64 [2 nblk, B, B]."""
    torch = _torch()
    for t, nm in ((roots, "roots"), (gstack, "gstack"), (dstack, "dstack")):
        _dev(t, nm)
    nblk, B = gstack.shape[0], gstack.shape[1]
    if ws is None:
        b = ctypes.c_size_t(0)
        _check(lib.shampoo_precondition_workspace(nblk, B, _dtype_code(roots), ctypes.byref(b)))
        ws = torch.empty(max(b.value, 1), dtype=torch.uint8, device=gstack.device)
    _check(lib.shampoo_precondition(_ptr(roots), _dtype_code(roots), _ptr(gstack), _dtype_code(gstack), nblk, B,
                                    _ptr(dstack), _ptr(ws), ws.numel(), _stream(stream)))


def shampoo_step_workspace(args):
    b = ctypes.c_size_t(0)
    _check(lib.shampoo_step_workspace(ctypes.byref(args), ctypes.byref(b)))
    return b.value


def shampoo_step(args, stream=None):
    """One full step over one stack; ``args`` is a StepArgsC (see optimizer.ShampooStack)."""
    _check(lib.shampoo_step(ctypes.byref(args), _stream(stream)))


def shampoo_check_flags(flags, stream=None):
    """Synchronises the stream; True if no matrix is flagged."""
    st = lib.shampoo_check_flags(_ptr(flags), flags.numel(), _stream(stream))
    if st == E_NONFINITE:
        return False
    _check(st)
    return True


def shampoo_timing_enable(capacity):
    _check(lib.shampoo_timing_enable(int(capacity)))


def shampoo_timing_read(capacity):
    """Durations (ms) of the batched-product launches recorded since enabling."""
    buf = (ctypes.c_float * max(int(capacity), 1))()
    n = ctypes.c_int32(0)
    _check(lib.shampoo_timing_read(buf, int(capacity), ctypes.byref(n)))
    return [buf[i] for i in range(n.value)]


def shampoo_mfma_peak(dtype, stream=None):
    """Measured dense matrix-core TFLOP/s for dtype "f32", "f64", "f16" or "bf16"."""
    import torch
    sink = torch.zeros(16, dtype=torch.float32, device="cuda")
    out = ctypes.c_double(0.0)
    _check(lib.shampoo_mfma_peak(DTYPES[dtype], ctypes.c_void_p(sink.data_ptr()), _stream(stream),
                                 ctypes.byref(out)))
    return out.value


# ---------------------------------------------------------------------------
# 8-bit block-scaled products
# ---------------------------------------------------------------------------
def _on_device(*tensors):
    """The common device of these tensors; ValueError unless they are device tensors of one device."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("expected device tensors")
        if dev is None:
            dev = t.device
        elif t.get_device() != dev.index:
            raise ValueError("tensors are on different devices")
    return dev


def _own_stream(stream, dev):
    if stream is not None and stream.device.index != dev.index:
        raise ValueError("stream of %s for tensors on %s" % (stream.device, dev))


def _launch(fn, dev, stream, *args):
    """fn(*args, stream) with ``dev`` current, on ``stream`` or the current one of that device."""
    _own_stream(stream, dev)
    torch = _torch()
    if torch.cuda.current_device() == dev.index:
        if stream is None:
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            handle = raw(dev.index) if raw is not None else torch.cuda.current_stream().cuda_stream
        else:
            handle = stream.cuda_stream
        _check(fn(*args, handle))
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, (stream if stream is not None else torch.cuda.current_stream()).cuda_stream))


def _empty(shape, dtype, dev, stream):
    """Device memory that belongs to the stream that will use it, so that the
    allocator hands it on only behind that stream's work."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _own_stream(stream, dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _up(x, m):
    return -(-x // m) * m


_FLOAT_CODES = {}


def _float_codes():
    """Types that are quantised, and that products write."""
    if not _FLOAT_CODES:
        torch = _torch()
        _FLOAT_CODES.update({torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16})
    return _FLOAT_CODES


def _f8_code(t):
    torch = _torch()
    if t.dtype == torch.float8_e4m3fn:
        return E4M3
    if t.dtype == torch.float8_e5m2:
        return E5M2
    raise TypeError("expected a float8_e4m3fn or float8_e5m2 tensor, got %s" % t.dtype)


def shampoo_quantize_f8(x, fmt="e4m3", block_rows=1, transpose=False, out=None, stream=None):
    """x [rows, cols] or [n, rows, cols] (float32, float16 or bfloat16, unit
    column stride) as 8-bit floating point with a power-of-two scale for each
    block of 128 columns of ``block_rows`` (1 or 128) rows.

    Returns (q, scale): q float8 [.., rows, cols rounded up to 128], zeros
    behind the columns; scale float8_e8m0fnu [.., ceil(rows / block_rows),
    blocks rounded up to 4], ones behind the blocks.  transpose=True
    quantises the transpose (blocks along x's rows) instead, "both" returns
    ((q, scale), (q_t, scale_t)) from one reading of x.  ``out``: tensors to
    write to, as returned."""
    torch = _torch()
    code = FORMATS_F8.get(fmt)
    if code is None:
        raise ValueError("fmt must be one of %s" % sorted(FORMATS_F8))
    if block_rows != 1 and block_rows != 128:
        raise ValueError("block_rows must be 1 or 128")
    if transpose is not False and transpose is not True and transpose != "both":
        raise ValueError("transpose must be False, True or 'both'")
    dim = x.dim()
    if dim not in (2, 3):
        raise ValueError("x must have 2 or 3 dimensions")
    dt = _float_codes().get(x.dtype)
    if dt is None:
        raise TypeError("unsupported dtype %s" % x.dtype)
    dev = _on_device(x)
    n, rows, cols = x.shape if dim == 3 else (1,) + tuple(x.shape)
    ld, apart = cols, 0
    if n and rows and cols:
        strides = x.stride()
        if cols > 1 and strides[-1] != 1:
            raise ValueError("x must have unit column stride")
        ld = strides[-2] if rows > 1 else cols
        apart = strides[0] if n > 1 else 0
        if ld < cols or apart < 0:
            raise ValueError("x must not overlap itself (row stride %d, %d columns)" % (ld, cols))
    kind = torch.float8_e4m3fn if code == E4M3 else torch.float8_e5m2

    def pair(r, k, given):
        K = _up(k, 128)
        shape, held = (r, K), (r if block_rows == 1 else -(-r // 128), _up(K // 128, 4))
        if dim == 3:
            shape, held = (n,) + shape, (n,) + held
        if given is None:
            return _empty(shape, kind, dev, stream), _empty(held, torch.float8_e8m0fnu, dev, stream)
        for t, s, d in zip(given, (shape, held), (kind, torch.float8_e8m0fnu)):
            _dev(t, "out")
            if tuple(t.shape) != s or t.dtype != d or t.device != dev:
                raise ValueError("out must be a %s tensor of shape %s on %s" % (d, s, dev))
        return tuple(given)

    q = s = qt = st = plain = turned = None
    if transpose is not True:
        plain = pair(rows, cols, out[0] if out is not None and transpose else out)
        q, s = plain[0].data_ptr(), plain[1].data_ptr()
    if transpose:
        turned = pair(cols, rows, out[1] if out is not None and transpose == "both" else out)
        qt, st = turned[0].data_ptr(), turned[1].data_ptr()
    _launch(lib.shampoo_quantize_f8, dev, stream, x.data_ptr(), dt, n, rows, cols, ld, apart, code, block_rows, q, s, qt, st)
    return (plain, turned) if transpose == "both" else turned if transpose else plain


def shampoo_matmul_f8_workspace(n, M, N, K):
    b = ctypes.c_size_t(0)
    _check(lib.shampoo_matmul_f8_workspace(int(n), int(M), int(N), int(K), ctypes.byref(b)))
    return b.value


def shampoo_matmul_f8(a, a_scale, b, b_scale, c, ws=None, stream=None):
    """c = a b^T of quantised matrices (as ``shampoo_quantize_f8`` returns
    them): a [M, K] or [n, M, K], b [N, K] or [n, N, K] in any mix of the two
    formats, c [M, N] or [n, M, N] float32, float16 or bfloat16.  A linear
    layer y = x W^T and its gradients dx = dy W, dW = dy^T x are three of
    these, on the operands quantised along each product's own inner side."""
    torch = _torch()
    dev = _on_device(a, a_scale, b, b_scale, c, ws)
    for t, nm in ((a, "a"), (a_scale, "a_scale"), (b, "b"), (b_scale, "b_scale"), (c, "c")):
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % nm)
    dim = a.dim()
    if dim not in (2, 3) or b.dim() != dim or c.dim() != dim or a_scale.dim() != dim or b_scale.dim() != dim:
        raise ValueError("a, b, c and the scales must all have 2, or all 3, dimensions")
    cdt = _float_codes().get(c.dtype)
    if cdt is None:
        raise TypeError("unsupported result dtype %s" % c.dtype)
    n, M, K = a.shape if dim == 3 else (1,) + tuple(a.shape)
    N = b.shape[-2]
    lead = (n,) if dim == 3 else ()
    if tuple(b.shape) != lead + (N, K) or tuple(c.shape) != lead + (M, N):
        raise ValueError("shapes do not match: a %s, b %s, c %s" % (tuple(a.shape), tuple(b.shape), tuple(c.shape)))

    def block_rows(t, s, rows):
        if s.dtype != torch.float8_e8m0fnu and s.dtype != torch.uint8:
            raise TypeError("scales must be float8_e8m0fnu")
        shape, Ks = tuple(s.shape), _up(K // 128, 4)
        if shape == lead + (rows, Ks):
            return 1
        if shape == lead + (-(-rows // 128), Ks):
            return 128
        raise ValueError("scales of shape %s do not fit %s" % (shape, tuple(t.shape)))

    arb, brb = block_rows(a, a_scale, M), block_rows(b, b_scale, N)
    room = 0
    if ws is None:
        need = shampoo_matmul_f8_workspace(n, M, N, K)
        ws = _empty(need, torch.uint8, dev, stream) if need else None
    if ws is not None:
        room = ws.numel() * ws.element_size()
    _launch(lib.shampoo_matmul_f8, dev, stream, a.data_ptr(), _f8_code(a), a_scale.data_ptr(), arb, b.data_ptr(),
            _f8_code(b), b_scale.data_ptr(), brb, n, M, N, K, c.data_ptr(), cdt,
            None if ws is None else ws.data_ptr(), room)
    return c


# ---------------------------------------------------------------------------
# softmax cross entropy of a projection
# ---------------------------------------------------------------------------
def _rows2d(t, name, shape, dtypes):
    if t is None:
        return 0
    if tuple(t.shape) != shape or t.dtype not in dtypes:
        raise ValueError("%s must be a %s tensor of shape %s, got %s %s" % (
            name, " or ".join(str(d) for d in dtypes), shape, t.dtype, tuple(t.shape)))
    if t.numel() and shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s must have unit column stride" % name)
    ld = t.stride(0) if shape[0] > 1 else shape[1]
    if t.numel() and ld < shape[1]:
        raise ValueError("%s must not overlap itself" % name)
    return ld


def _xent_args(hidden, weight, targets, loss, lse, dhidden, dweight, row_scale, ignore_index, reduction, scale, accumulate,
               panel_rows, logits_dtype=None):
    torch = _torch()
    if reduction not in REDUCTIONS:
        raise ValueError("reduction must be one of %s" % sorted(REDUCTIONS))
    if hidden.dim() != 2 or weight.dim() != 2:
        raise ValueError("hidden and weight must have 2 dimensions")
    N, d = hidden.shape
    V = weight.shape[0]
    if hidden.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("unsupported dtype %s (float32, bfloat16)" % hidden.dtype)
    ldh = _rows2d(hidden, "hidden", (N, d), (hidden.dtype,))
    ldw = _rows2d(weight, "weight", (V, d), (hidden.dtype, torch.float32))
    lddh = _rows2d(dhidden, "dhidden", (N, d), (hidden.dtype,))
    lddw = _rows2d(dweight, "dweight", (V, d), (hidden.dtype, torch.float32))
    for t, name, dtype in ((targets, "targets", torch.int64), (row_scale, "row_scale", torch.float32),
                           (lse, "lse", torch.float32)):
        if t is not None and (t.dtype != dtype or tuple(t.shape) != (N,) or not t.is_contiguous()):
            raise ValueError("%s must be a contiguous %s tensor of shape (%d,)" % (name, dtype, N))
    shape = (N,) if reduction == "none" else ()
    if loss is not None and (loss.dtype != torch.float32 or tuple(loss.shape) != shape or not loss.is_contiguous()):
        raise ValueError("loss must be a contiguous float32 tensor of shape %s" % (shape,))

    if logits_dtype not in (None, hidden.dtype, torch.float8_e4m3fn):
        raise ValueError("logits_dtype must be None, hidden's dtype or torch.float8_e4m3fn")
    if logits_dtype == torch.float8_e4m3fn and hidden.dtype != torch.bfloat16:
        raise ValueError("8-bit logits need bfloat16 hidden")

    def at(t):
        return None if t is None else t.data_ptr()

    return XentArgsC(at(hidden), at(weight), at(targets), at(row_scale), at(loss), at(lse), at(dhidden), at(dweight),
                     max(ldh, d), max(ldw, d), max(lddh, d), max(lddw, d), N, V, d, int(ignore_index), int(panel_rows),
                     _dtype_code(hidden), _dtype_code(weight), _dtype_code(dweight) if dweight is not None else _dtype_code(hidden),
                     E4M3 if logits_dtype == torch.float8_e4m3fn else _dtype_code(hidden),
                     REDUCTIONS[reduction], 1 if accumulate else 0, float(scale), None, 0)


def shampoo_linear_xent_workspace(hidden, weight, targets, dhidden=None, dweight=None, panel_rows=0, logits_dtype=None):
    """Workspace bytes of ``shampoo_linear_xent`` with these tensors."""
    b = ctypes.c_size_t(0)
    args = _xent_args(hidden, weight, targets, None, None, dhidden, dweight, None, -100, "mean", 1.0, False, panel_rows,
                      logits_dtype)
    _check(lib.shampoo_linear_xent_workspace(ctypes.byref(args), ctypes.byref(b)))
    return b.value


def shampoo_linear_xent(hidden, weight, targets, loss=None, lse=None, dhidden=None, dweight=None, row_scale=None,
                        ignore_index=-100, reduction="mean", scale=1.0, accumulate=False, panel_rows=0, logits_dtype=None,
                        ws=None, stream=None):
    """Softmax cross entropy of the projection hidden weight^T against
    ``targets``; returns the loss.  Alone it keeps no logits; with gradients
    the exponentials of a panel of rows, in hidden's type.

    hidden [N, d] and weight [V, d] (float32 or bfloat16, unit column
    stride; a float32 weight beside bfloat16 hidden is rounded to bfloat16),
    targets int64 [N]; rows with target ``ignore_index`` count for
    nothing.  reduction: "mean" over the other rows, "sum" or "none".
    row_scale float32 [N] and scale multiply each row's loss before the
    reduction; with "none" the losses come as they are, and row_scale times
    scale is the gradient that arrives at them.  dhidden, dweight: tensors that
    receive the gradients; dweight may be float32 beside bfloat16 inputs, and
    accumulate=True adds to it.  lse:
    receives log sum exp of each row.  panel_rows bounds the rows whose
    exponentials the workspace holds at a time (0: up to 2 GiB of them).
    logits_dtype=torch.float8_e4m3fn (bfloat16 hidden only) quantises hidden
    and weight as ``shampoo_quantize_f8`` does and takes the logits from their
    8-bit product; the gradients' products stay in bfloat16."""
    torch = _torch()
    dev = _on_device(hidden, weight, targets, loss, lse, dhidden, dweight, row_scale, ws)
    if loss is None:
        loss = _empty((hidden.shape[0],) if reduction == "none" else (), torch.float32, dev, stream)
    args = _xent_args(hidden, weight, targets, loss, lse, dhidden, dweight, row_scale, ignore_index, reduction, scale,
                      accumulate, panel_rows, logits_dtype)
    if ws is None:
        b = ctypes.c_size_t(0)
        _check(lib.shampoo_linear_xent_workspace(ctypes.byref(args), ctypes.byref(b)))
        ws = _empty(max(b.value, 1), torch.uint8, dev, stream)
    args.ws, args.ws_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    _launch(lib.shampoo_linear_xent, dev, stream, ctypes.byref(args))
    return loss


from .optimizer import Shampoo, ShampooStack  # noqa: E402  (needs the binding above)
