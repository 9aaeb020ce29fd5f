"""Streaming log-domain Sinkhorn on AMD Instinct MI355X (gfx950).

Thin ctypes binding over the C ABI in ``include/sk.h`` (libsk.so): argument
marshalling only.  Every step of the computation runs in the library's HIP
kernels; PyTorch provides device memory and the current stream.  There is no
CPU fallback: if libsk.so is missing or cannot be loaded, every call raises.

Tensor contract (SinkSLOT README, Tensor Contract): x (n, d) and y (m, d)
float32 point clouds, optional nonnegative weights a (n,), b (m,) -- uniform
if omitted, used exactly as given, sum(a) must equal sum(b) (ValueError
otherwise), zeros legal -- all on the same CUDA/HIP device.  float64 inputs
raise ValueError: the kernels are float32-only.  The cost is
C_ij = |x_i - y_j|^2 with no 1/2 factor; eps is measured against it.
Potentials are returned in cost units (f, g), not divided by eps.

The scores_* functions take a score matrix instead of clouds, (n, m) float32,
bfloat16 or float16 with any row stride: balancing potentials and routing of a
router's scores, log-probabilities of a head's, and their gradients.

No function here takes part in autograd: inputs are read and outputs written by
their addresses, so a result carries no graph, also where an input requires a
gradient, and a tensor written into (``out``, ``grad``, ``g``, ...) keeps its version.
A trainer wraps a forward and its gradient in a ``torch.autograd.Function``.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libsk.so")

SK_OK = 0
_STATUS_NAMES = {
    0: "SK_OK", 1: "SK_ERR_NULL", 2: "SK_ERR_SHAPE", 3: "SK_ERR_UNSUPPORTED_D", 4: "SK_ERR_EPS",
    5: "SK_ERR_ITERS", 6: "SK_ERR_CHECK_EVERY", 7: "SK_ERR_NEG_WEIGHT", 8: "SK_ERR_MASS_MISMATCH",
    9: "SK_ERR_EMPTY_MEASURE", 10: "SK_ERR_NONFINITE", 11: "SK_ERR_WORKSPACE", 12: "SK_ERR_HIP",
    13: "SK_ERR_VARIANT", 14: "SK_ERR_STOP", 15: "SK_ERR_CAPTURE", 16: "SK_ERR_LR", 17: "SK_ERR_SCRATCH",
    18: "SK_ERR_DTYPE", 19: "SK_ERR_ROUTE", 20: "SK_ERR_OVERLAP",
}
_VALUE_ERRORS = {1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 13, 14, 15, 16, 17, 18, 19, 20}
NOALLOC_SCRATCH_BYTES = 64 << 20  # SK_NOALLOC_SCRATCH_BYTES of include/sk.h

# SinkSLOT README, API Reference: variant and stop_mode names
VARIANTS = {"alternating": 0, "symmetric": 1}
STOP_MODES = {"fixed": 0, "marginal": 1, "potential": 2}

# operators on a given score matrix: element types (sk_dtype), score functions and where the choice is made
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
SCORE_FNS = {"softmax": 0, "sigmoid": 1}
SELECT_ON = {"score": 0, "logit": 1}

# C ABI: (name, restype, argtypes)
_vp, _i64, _i32, _f32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "sk_abi_version": (ctypes.c_int, []),
    "sk_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "sk_workspace_bytes": (_sz, [_i64, _i64, _i32]),
    "sk_check_inputs": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _vp, _sz, _vp]),
    "sk_solve": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _f32, _i32, _vp, _vp, _i32, _vp, _vp, _sz,
                                _vp]),
    "sk_solve_warm": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _f32, _i32, _vp, _vp, _vp, _i32, _vp,
                                     _vp, _sz, _vp]),
    "sk_solve_noalloc": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _f32, _i32, _vp, _vp, _i32, _vp,
                                        _vp]),
    "sk_primal_cost": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _f32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "sk_cost": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _f32, _vp, _vp]),
    "sk_marginal_residual": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _f32, _vp, _vp, _vp, _vp, _sz,
                                            _vp]),
    "sk_grad_x": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _f32, _vp, _vp, _vp, _sz, _vp]),
    "sk_solve_ex": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _f32, _i32, _f32, _i32, _f32, _i32, _i32,
                                   _vp, _vp, ctypes.POINTER(_i32), ctypes.POINTER(_i32), ctypes.POINTER(_f32), _vp,
                                   _sz, _vp]),
    "sk_dual_cost": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _f32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "sk_divergence_workspace_bytes": (_sz, [_i64, _i64, _i32]),
    "sk_divergence": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _f32, _i32, _f32, _i32, _vp, _vp, _sz,
                                     _vp]),
    "sk_gradient_flow": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _f32, _i32, _i32, _f32, _vp, _vp, _vp,
                                        _vp, _vp, _sz, _vp]),
    "sk_transport_workspace_bytes": (_sz, [_i64, _i64, _i32]),
    "sk_transport": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _f32, _vp, _vp, _i32, _vp, _i32, _vp, _vp,
                                    _sz, _vp]),
    "sk_hvp": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _f32, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _sz,
                              _vp]),
    "sk_fs2_workspace_bytes": (_sz, [_i64, _i64, _i32, _i32, _i32]),
    "sk_fs2_solve": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _f32, _i32, _f32, _f32, _i32, _i32, _f32,
                                    _i32, _i32, _i32, _i32, _vp, _vp, ctypes.POINTER(_i32), ctypes.POINTER(_f32), _vp,
                                    _vp, _vp, _sz, _vp]),
    "sk_scores_solve_workspace_bytes": (_sz, [_i64, _i64]),
    "sk_scores_solve": (ctypes.c_int, [_vp, _i32, _i64, _i64, _i64, _vp, _vp, _f32, _i32, _vp, _vp, _vp, _vp, _sz,
                                       _vp]),
    "sk_scores_route": (ctypes.c_int, [_vp, _i32, _i64, _i64, _i64, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                       _f32, _vp, _vp, _vp, _vp]),
    "sk_scores_route_grad": (ctypes.c_int, [_vp, _i32, _i64, _i64, _i64, _i32, _vp, _vp, _i32, _i32, _f32, _vp, _i64,
                                            _vp]),
    "sk_scores_logprobs_workspace_bytes": (_sz, [_i32, _i64, _i64, _i32]),
    "sk_scores_logprobs": (ctypes.c_int, [_vp, _i32, _i64, _i64, _i64, _f32, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                          _vp, _sz, _vp]),
    "sk_scores_logprobs_grad": (ctypes.c_int, [_vp, _i32, _i64, _i64, _i64, _f32, _vp, _vp, _vp, _i32, _vp, _vp, _vp,
                                               _vp, _vp, _vp, _i64, _vp]),
    "sk_timing_enable": (ctypes.c_int, [ctypes.c_int]),
    "sk_timing_read": (ctypes.c_int, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64),
                                      ctypes.POINTER(ctypes.c_double)]),
}

_lock = threading.Lock()
_lib = None


class SinkhornError(RuntimeError):
    """A HIP failure inside the library."""


def load_library(path: str | None = None):
    """Load libsk.so (raises if it is missing: there is no fallback path)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"libsk.so not found at {p}; build it with "
                               "`python -m streaming_sinkhorn_solver_amd.build`")
        lib = ctypes.CDLL(p)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        if path is None:
            _lib = lib
        return lib


def status_string(code: int) -> str:
    return load_library().sk_status_string(int(code)).decode()


def _raise(code: int, where: str):
    if code == SK_OK:
        return
    msg = f"{where}: {_STATUS_NAMES.get(code, code)} ({status_string(code)})"
    if code in _VALUE_ERRORS:
        raise ValueError(msg)
    raise SinkhornError(msg)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _buf(t, shape, dtype, device, name: str) -> torch.Tensor:
    """A caller-supplied output (checked: dtype, device, shape, contiguous) or a new one."""
    shape = tuple(int(k) for k in shape)
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be a {dtype} tensor on {device}")
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {shape} (got {tuple(t.shape)})")
    return t


def _in(t, shape, device, name: str) -> torch.Tensor:
    """A float32 input of the given shape on the device, made contiguous."""
    shape = tuple(int(k) for k in shape)
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.device != device:
        raise ValueError(f"{name} must be a float32 tensor on {device}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape} (got {tuple(t.shape)})")
    return t.contiguous()


def _at_least(t, count: int, dtype, device, name: str) -> torch.Tensor:
    """A caller-supplied contiguous buffer of at least count elements (dtype, device checked)."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on {device}")
    if t.numel() < count:
        raise ValueError(f"{name} must hold at least {count} values")
    return t


def _ws(ws, device, make) -> torch.Tensor:
    """A caller-supplied workspace (a contiguous uint8 tensor on the device; the library checks its
    size and alignment) or a new one from make()."""
    if ws is None:
        return make()
    if not isinstance(ws, torch.Tensor) or ws.dtype != torch.uint8 or ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous uint8 tensor on {device}")
    return ws


def _as_problem(x, y, a, b):
    if not isinstance(x, torch.Tensor) or not isinstance(y, torch.Tensor):
        raise TypeError("x and y must be torch tensors")
    if x.dtype != torch.float32 or y.dtype != torch.float32:
        raise ValueError("the kernels are float32-only (got %s, %s)" % (x.dtype, y.dtype))
    if x.dim() != 2 or y.dim() != 2 or x.shape[1] != y.shape[1]:
        raise ValueError("x must be (n, d) and y (m, d) with the same d")
    if x.device.type != "cuda" or y.device != x.device:
        raise ValueError("x and y must be on the same GPU device")
    n, d = x.shape
    m = y.shape[0]
    if a is None:
        a = torch.full((n,), 1.0 / n, dtype=torch.float32, device=x.device)
    if b is None:
        b = torch.full((m,), 1.0 / m, dtype=torch.float32, device=x.device)
    for name, w, k in (("a", a, n), ("b", b, m)):
        if w.dtype != torch.float32:
            raise ValueError(f"{name} must be float32 (got {w.dtype})")
        if w.shape != (k,) or w.device != x.device:
            raise ValueError(f"{name} must have shape ({k},) on {x.device}")
    return x.contiguous(), y.contiguous(), a.contiguous(), b.contiguous(), n, m, d


def workspace_bytes(n: int, m: int, d: int) -> int:
    return int(load_library().sk_workspace_bytes(n, m, d))


def workspace(n: int, m: int, d: int, device) -> torch.Tensor:
    """A workspace tensor for problems of this size (uint8, 256-byte aligned by torch's allocator)."""
    nb = workspace_bytes(n, m, d)
    if nb == 0:
        raise ValueError(f"invalid problem size n={n} m={m} d={d}")
    ws = torch.empty(nb, dtype=torch.uint8, device=device)
    if ws.data_ptr() % 256:
        raise RuntimeError("allocator returned a workspace that is not 256-byte aligned")
    return ws


def check_inputs(x, y, a=None, b=None, ws: torch.Tensor | None = None) -> None:
    """Validate the data (finite, nonnegative weights, equal nonzero masses); raises ValueError."""
    lib = load_library()
    x, y, a, b, n, m, d = _as_problem(x, y, a, b)
    ws = _ws(ws, x.device, lambda: workspace(n, m, d, x.device))
    _raise(lib.sk_check_inputs(_ptr(x), _ptr(y), _ptr(a), _ptr(b), n, m, d, _ptr(ws), ws.numel(),
                               _stream(x.device)), "sk_check_inputs")


def solve(x, y, a=None, b=None, *, eps: float, n_iters: int, check_every: int = 0,
          ws: torch.Tensor | None = None, f: torch.Tensor | None = None, g: torch.Tensor | None = None,
          trace: torch.Tensor | None = None, check: bool = True):
    """Fixed-count alternating log-domain Sinkhorn from g = 0.

    Returns (f, g, resid_trace); resid_trace holds n_iters // check_every
    marginal residuals (empty when check_every == 0).  Outputs are enqueued on
    the current stream.
    """
    lib = load_library()
    x, y, a, b, n, m, d = _as_problem(x, y, a, b)
    ws = _ws(ws, x.device, lambda: workspace(n, m, d, x.device))
    if check:
        check_inputs(x, y, a, b, ws)
    f = _buf(f, (n,), torch.float32, x.device, "f")
    g = _buf(g, (m,), torch.float32, x.device, "g")
    nt = n_iters // check_every if check_every > 0 else 0
    if trace is None:
        trace = torch.empty(max(nt, 0), dtype=torch.float32, device=x.device)
    else:
        trace = _at_least(trace, nt, torch.float32, x.device, "trace")
    _raise(lib.sk_solve(_ptr(x), _ptr(y), _ptr(a), _ptr(b), n, m, d, float(eps), int(n_iters), _ptr(f), _ptr(g),
                        int(check_every), _ptr(trace) if nt > 0 else None, _ptr(ws), ws.numel(),
                        _stream(x.device)), "sk_solve")
    return f, g, trace


def solve_warm(x, y, a=None, b=None, *, eps: float, n_iters: int, g_init: torch.Tensor, check_every: int = 0,
               ws: torch.Tensor | None = None, f: torch.Tensor | None = None, g: torch.Tensor | None = None,
               trace: torch.Tensor | None = None, check: bool = True):
    """The fixed-count solve of ``solve`` started from g = g_init (m,) instead of 0; g_init may be g itself
    (continued in place).  Returns (f, g, resid_trace)."""
    lib = load_library()
    x, y, a, b, n, m, d = _as_problem(x, y, a, b)
    ws = _ws(ws, x.device, lambda: workspace(n, m, d, x.device))
    if check:
        check_inputs(x, y, a, b, ws)
    g_init = _in(g_init, (m,), x.device, "g_init")
    f = _buf(f, (n,), torch.float32, x.device, "f")
    g = _buf(g, (m,), torch.float32, x.device, "g")
    nt = n_iters // check_every if check_every > 0 else 0
    if trace is None:
        trace = torch.empty(max(nt, 0), dtype=torch.float32, device=x.device)
    else:
        trace = _at_least(trace, nt, torch.float32, x.device, "trace")
    _raise(lib.sk_solve_warm(_ptr(x), _ptr(y), _ptr(a), _ptr(b), n, m, d, float(eps), int(n_iters), _ptr(g_init),
                             _ptr(f), _ptr(g), int(check_every), _ptr(trace) if nt > 0 else None, _ptr(ws),
                             ws.numel(), _stream(x.device)), "sk_solve_warm")
    return f, g, trace


def primal_cost(x, y, a, b, f, g, *, eps: float, ws: torch.Tensor | None = None,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """[<P,C> + eps KL(P | a x b), <P,C>] of the plan at (f, g), as a 2-element float64 tensor."""
    lib = load_library()
    x, y, a, b, n, m, d = _as_problem(x, y, a, b)
    ws = _ws(ws, x.device, lambda: transport_workspace(n, m, d, x.device))
    f, g = _potentials(f, g, n, m, x.device)
    out = _buf(out, (2,), torch.float64, x.device, "out")
    _raise(lib.sk_primal_cost(_ptr(x), _ptr(y), _ptr(a), _ptr(b), n, m, d, float(eps), _ptr(f), _ptr(g), _ptr(out),
                              _ptr(ws), ws.numel(), _stream(x.device)), "sk_primal_cost")
    return out


def solve_noalloc(x, y, a=None, b=None, *, eps: float, n_iters: int, f: torch.Tensor, g: torch.Tensor,
                  check_every: int = 0, trace: torch.Tensor | None = None):
    """sk_solve_noalloc: the fixed-count solve of ``solve`` in the library's static device scratch, with
    caller-supplied outputs (f (n,), g (m,) and, when check_every > 0, trace of n_iters // check_every
    floats).  Nothing is allocated, so the data checks of ``check_inputs`` (which need a workspace) are not
    run here; call it beforehand if the data may be invalid.  Problems whose workspace would exceed
    NOALLOC_SCRATCH_BYTES raise ValueError.  Calls whose work overlaps on one GPU race (one scratch per GPU).
    """
    lib = load_library()
    x, y, a, b, n, m, d = _as_problem(x, y, a, b)
    f = _buf(f, (n,), torch.float32, x.device, "f")
    g = _buf(g, (m,), torch.float32, x.device, "g")
    nt = n_iters // check_every if check_every > 0 else 0
    if nt > 0:
        trace = _at_least(trace, nt, torch.float32, x.device, "trace")
    _raise(lib.sk_solve_noalloc(_ptr(x), _ptr(y), _ptr(a), _ptr(b), n, m, d, float(eps), int(n_iters), _ptr(f),
                                _ptr(g), int(check_every), _ptr(trace) if nt > 0 else None, _stream(x.device)),
           "sk_solve_noalloc")
    return f, g, trace


def solve_ex(x, y, a=None, b=None, *, eps: float, variant: str = "alternating", alpha: float = 0.5,
             stop_mode: str = "fixed", stop_tol: float = 1e-6, max_iter: int = 200, check_every: int = 5,
             ws: torch.Tensor | None = None, f: torch.Tensor | None = None, g: torch.Tensor | None = None,
             check: bool = True):
    """Sinkhorn with update variant ("alternating" | "symmetric" with blend alpha) and stop rule
    ("fixed" | "marginal" | "potential"; max_iter is the iteration count or cap).

    Returns (f, g, iters_run, converged, final_viol); converged and final_viol
    are None under stop_mode="fixed" (then nothing synchronises and the
    outputs are enqueued on the current stream).
    """
    lib = load_library()
    if variant not in VARIANTS or stop_mode not in STOP_MODES:
        raise ValueError(f"variant must be one of {list(VARIANTS)}, stop_mode one of {list(STOP_MODES)}")
    x, y, a, b, n, m, d = _as_problem(x, y, a, b)
    ws = _ws(ws, x.device, lambda: workspace(n, m, d, x.device))
    if check:
        check_inputs(x, y, a, b, ws)
    f = _buf(f, (n,), torch.float32, x.device, "f")
    g = _buf(g, (m,), torch.float32, x.device, "g")
    it, conv, viol = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_float()
    _raise(lib.sk_solve_ex(_ptr(x), _ptr(y), _ptr(a), _ptr(b), n, m, d, float(eps), VARIANTS[variant],
                           float(alpha), STOP_MODES[stop_mode], float(stop_tol), int(max_iter), int(check_every),
                           _ptr(f), _ptr(g), ctypes.byref(it), ctypes.byref(conv), ctypes.byref(viol), _ptr(ws),
                           ws.numel(), _stream(x.device)), "sk_solve_ex")
    if stop_mode == "fixed":
        return f, g, it.value, None, None
    return f, g, it.value, bool(conv.value), viol.value


def dual_cost(x, y, a, b, f, g, *, eps: float, ws: torch.Tensor | None = None,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """<a,f> + <b,g> - eps (sum_ij P_ij - sum(a) sum(b)) at any potentials (1-element float64 tensor)."""
    lib = load_library()
    x, y, a, b, n, m, d = _as_problem(x, y, a, b)
    ws = _ws(ws, x.device, lambda: workspace(n, m, d, x.device))
    f, g = _potentials(f, g, n, m, x.device)
    out = _buf(out, (1,), torch.float64, x.device, "out")
    _raise(lib.sk_dual_cost(_ptr(x), _ptr(y), _ptr(a), _ptr(b), n, m, d, float(eps), _ptr(f), _ptr(g), _ptr(out),
                            _ptr(ws), ws.numel(), _stream(x.device)), "sk_dual_cost")
    return out


def divergence_workspace(n: int, m: int, d: int, device) -> torch.Tensor:
    nb = int(load_library().sk_divergence_workspace_bytes(n, m, d))
    if nb == 0:
        raise ValueError(f"invalid problem size n={n} m={m} d={d}")
    ws = torch.empty(nb, dtype=torch.uint8, device=device)
    if ws.data_ptr() % 256:
        raise RuntimeError("allocator returned a workspace that is not 256-byte aligned")
    return ws


def divergence(x, y, a=None, b=None, *, eps: float, n_iters: int, variant: str = "alternating",
               alpha: float = 0.5, ws: torch.Tensor | None = None, out: torch.Tensor | None = None,
               check: bool = True) -> torch.Tensor:
    """Debiased divergence OT(x,y) - OT(x,x)/2 - OT(y,y)/2 after n_iters iterations per term.

    Returns a 4-element float64 device tensor [S, OT(x,y), OT(x,x), OT(y,y)].
    """
    lib = load_library()
    if variant not in VARIANTS:
        raise ValueError(f"variant must be one of {list(VARIANTS)}")
    x, y, a, b, n, m, d = _as_problem(x, y, a, b)
    if check:
        check_inputs(x, y, a, b)
    ws = _ws(ws, x.device, lambda: divergence_workspace(n, m, d, x.device))
    out = _buf(out, (4,), torch.float64, x.device, "out")
    _raise(lib.sk_divergence(_ptr(x), _ptr(y), _ptr(a), _ptr(b), n, m, d, float(eps), VARIANTS[variant],
                             float(alpha), int(n_iters), _ptr(out), _ptr(ws), ws.numel(), _stream(x.device)),
           "sk_divergence")
    return out


def gradient_flow(x, y, a=None, b=None, *, eps: float, n_iters: int, n_steps: int, lr: float,
                  ws: torch.Tensor | None = None, f: torch.Tensor | None = None, g: torch.Tensor | None = None,
                  grad: torch.Tensor | None = None, cost_trace: torch.Tensor | None = None, check: bool = True):
    """n_steps of x <- x - lr * grad_x, each at a fresh n_iters-iteration solve; x is updated in place.

    Returns (x, f, g, grad, cost_trace): f, g, grad of the last step, cost_trace (float64, n_steps) of
    every step."""
    lib = load_library()
    x_in = x
    x, y, a, b, n, m, d = _as_problem(x, y, a, b)
    if x.data_ptr() != x_in.data_ptr():
        raise ValueError("x is updated in place and must be contiguous")
    ws = _ws(ws, x.device, lambda: workspace(n, m, d, x.device))
    if check:
        check_inputs(x, y, a, b, ws)
    f = _buf(f, (n,), torch.float32, x.device, "f")
    g = _buf(g, (m,), torch.float32, x.device, "g")
    grad = _buf(grad, (n, d), torch.float32, x.device, "grad")
    if cost_trace is None:
        cost_trace = torch.empty(max(n_steps, 1), dtype=torch.float64, device=x.device)
    else:
        cost_trace = _at_least(cost_trace, n_steps, torch.float64, x.device, "cost_trace")
    _raise(lib.sk_gradient_flow(_ptr(x), _ptr(y), _ptr(a), _ptr(b), n, m, d, float(eps), int(n_iters), int(n_steps),
                                float(lr), _ptr(f), _ptr(g), _ptr(grad), _ptr(cost_trace), _ptr(ws), ws.numel(),
                                _stream(x.device)), "sk_gradient_flow")
    return x, f, g, grad, cost_trace[:n_steps]


def transport_workspace(n: int, m: int, d: int, device) -> torch.Tensor:
    nb = int(load_library().sk_transport_workspace_bytes(n, m, d))
    if nb == 0:
        raise ValueError(f"invalid problem size n={n} m={m} d={d}")
    ws = torch.empty(nb, dtype=torch.uint8, device=device)
    if ws.data_ptr() % 256:
        raise RuntimeError("allocator returned a workspace that is not 256-byte aligned")
    return ws


def _potentials(f, g, n, m, device):
    return _in(f, (n,), device, "f"), _in(g, (m,), device, "g")


def transport(x, y, a, b, f, g, v, *, eps: float, transpose: bool = False, ws: torch.Tensor | None = None,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """P v (v: (m,) or (m, k)) or, with transpose, P^T v (v: (n,) or (n, k)), with
    P_ij = a_i b_j exp((f_i + g_j - C_ij)/eps)."""
    lib = load_library()
    x, y, a, b, n, m, d = _as_problem(x, y, a, b)
    f, g = _potentials(f, g, n, m, x.device)
    rows_in, rows_out = (n, m) if transpose else (m, n)
    vec = v.dim() == 1
    v2 = v.reshape(-1, 1) if vec else v
    if v2.dim() != 2 or v2.shape[0] != rows_in:
        raise ValueError(f"v must have {rows_in} rows")
    k = v2.shape[1]
    v2 = _in(v2, (rows_in, k), x.device, "v")
    ws = _ws(ws, x.device, lambda: transport_workspace(n, m, d, x.device))
    out = _buf(out, (rows_out, k), torch.float32, x.device, "out")
    _raise(lib.sk_transport(_ptr(x), _ptr(y), _ptr(a), _ptr(b), n, m, d, float(eps), _ptr(f), _ptr(g),
                            1 if transpose else 0, _ptr(v2), k, _ptr(out), _ptr(ws), ws.numel(), _stream(x.device)),
           "sk_transport")
    return out.reshape(-1) if vec else out


def hvp(x, y, a, b, f, g, v, *, eps: float, cg_iters: int = 50, ws: torch.Tensor | None = None,
        out: torch.Tensor | None = None, cg_resid: torch.Tensor | None = None):
    """Hessian-vector product of OT_eps(x, y) in x at the plan of (f, g); v and the result are (n, d).

    Returns (H v, cg_resid) with cg_resid a 1-element device tensor."""
    lib = load_library()
    x, y, a, b, n, m, d = _as_problem(x, y, a, b)
    f, g = _potentials(f, g, n, m, x.device)
    v = _in(v, (n, d), x.device, "v")
    ws = _ws(ws, x.device, lambda: transport_workspace(n, m, d, x.device))
    out = _buf(out, (n, d), torch.float32, x.device, "out")
    cg_resid = _buf(cg_resid, (1,), torch.float32, x.device, "cg_resid")
    _raise(lib.sk_hvp(_ptr(x), _ptr(y), _ptr(a), _ptr(b), n, m, d, float(eps), _ptr(f), _ptr(g), _ptr(v),
                      int(cg_iters), _ptr(out), _ptr(cg_resid), _ptr(ws), ws.numel(), _stream(x.device)), "sk_hvp")
    return out, cg_resid


def fs2_solve(x, y, a=None, b=None, *, eps: float, block: int = 512, tol: float = 1e-4, delta: float = 1e-6,
              coarse_iters: int = 20, max_rounds: int = 10, coarse_gain: float = 0.1, n_sample: int = 1024,
              max_iters: int = 1000, check_every: int = 10, screen_every: int = 10, ws: torch.Tensor | None = None,
              f: torch.Tensor | None = None, g: torch.Tensor | None = None, return_perm: bool = False,
              check: bool = True):
    """Two-stage block-sparse solver (d <= 8).  Returns (f, g, info); info holds rounds, fine_iters,
    kept (block pairs at the last screening), kept_fraction, converged, residual, last_check and,
    with return_perm, the Morton orders perm_x, perm_y (device int32)."""
    lib = load_library()
    x, y, a, b, n, m, d = _as_problem(x, y, a, b)
    if check:
        check_inputs(x, y, a, b)
    def make_ws():
        nb = int(lib.sk_fs2_workspace_bytes(n, m, d, int(block), int(n_sample)))
        if nb == 0:
            raise ValueError(f"invalid arguments for the block-sparse solver (n={n} m={m} d={d} block={block})")
        return torch.empty(nb, dtype=torch.uint8, device=x.device)

    ws = _ws(ws, x.device, make_ws)
    f = _buf(f, (n,), torch.float32, x.device, "f")
    g = _buf(g, (m,), torch.float32, x.device, "g")
    px = torch.empty(n, dtype=torch.int32, device=x.device) if return_perm else None
    py = torch.empty(m, dtype=torch.int32, device=x.device) if return_perm else None
    ii = (ctypes.c_int32 * 4)()
    ff = (ctypes.c_float * 2)()
    _raise(lib.sk_fs2_solve(_ptr(x), _ptr(y), _ptr(a), _ptr(b), n, m, d, float(eps), int(block), float(tol),
                            float(delta), int(coarse_iters), int(max_rounds), float(coarse_gain), int(n_sample),
                            int(max_iters), int(check_every), int(screen_every), _ptr(f), _ptr(g), ii, ff, _ptr(px),
                            _ptr(py), _ptr(ws), ws.numel(), _stream(x.device)), "sk_fs2_solve")
    nbx, nby = (n + block - 1) // block, (m + block - 1) // block
    info = dict(rounds=ii[0], fine_iters=ii[1], kept=ii[2], kept_fraction=ii[2] / (nbx * nby), converged=bool(ii[3]),
                residual=ff[0], last_check=ff[1])
    if return_perm:
        info["perm_x"], info["perm_y"] = px, py
    return f, g, info


def cost(a, b, f, g, *, eps: float, out: torch.Tensor | None = None) -> torch.Tensor:
    """<a,f> + <b,g> - eps sum(b)(1 - sum(a)) in float64 (a 1-element device tensor)."""
    lib = load_library()
    if not isinstance(a, torch.Tensor) or a.device.type != "cuda":
        raise ValueError("a must be a float32 GPU tensor")
    n, m = a.numel(), b.numel()
    a, b = _in(a, (n,), a.device, "a"), _in(b, (m,), a.device, "b")
    f, g = _in(f, (n,), a.device, "f"), _in(g, (m,), a.device, "g")
    out = _buf(out, (1,), torch.float64, a.device, "out")
    _raise(lib.sk_cost(_ptr(a), _ptr(b), _ptr(f), _ptr(g), n, m, float(eps), _ptr(out), _stream(a.device)),
           "sk_cost")
    return out


def marginal_residual(x, y, a, b, f, g, *, eps: float, ws: torch.Tensor | None = None) -> torch.Tensor:
    """[max|P1-a|, max|P^T1-b|, sum|P1-a|, sum|P^T1-b|] at (f, g), as a 4-element float32 tensor."""
    lib = load_library()
    x, y, a, b, n, m, d = _as_problem(x, y, a, b)
    ws = _ws(ws, x.device, lambda: workspace(n, m, d, x.device))
    out = torch.empty(4, dtype=torch.float32, device=x.device)
    f, g = _potentials(f, g, n, m, x.device)
    _raise(lib.sk_marginal_residual(_ptr(x), _ptr(y), _ptr(a), _ptr(b), n, m, d, float(eps), _ptr(f), _ptr(g),
                                    _ptr(out), _ptr(ws), ws.numel(), _stream(x.device)), "sk_marginal_residual")
    return out


def grad_x(x, y, a, b, g, *, eps: float, ws: torch.Tensor | None = None,
           out: torch.Tensor | None = None) -> torch.Tensor:
    """grad_i = 2 a_i (x_i - sum_j w_ij y_j), w_i. = softmax_j((g_j - C_ij)/eps + log b_j)."""
    lib = load_library()
    x, y, a, b, n, m, d = _as_problem(x, y, a, b)
    ws = _ws(ws, x.device, lambda: workspace(n, m, d, x.device))
    g = _in(g, (m,), x.device, "g")
    out = _buf(out, (n, d), torch.float32, x.device, "out")
    _raise(lib.sk_grad_x(_ptr(x), _ptr(y), _ptr(a), _ptr(b), n, m, d, float(eps), _ptr(g), _ptr(out), _ptr(ws),
                         ws.numel(), _stream(x.device)), "sk_grad_x")
    return out


def _scores(scores):
    """A score matrix as (tensor, dtype code, n, m, row stride): (n, m) float32, bfloat16 or float16 on a GPU, any
    row stride; scores whose neighbours in a row do not lie next to each other are copied."""
    if not isinstance(scores, torch.Tensor):
        raise TypeError("scores must be a torch tensor")
    code = DTYPES.get(scores.dtype)
    if code is None:
        raise ValueError(f"scores must be float32, bfloat16 or float16 (got {scores.dtype})")
    if scores.dim() != 2:
        raise ValueError(f"scores must be (n, m) (got shape {tuple(scores.shape)})")
    if scores.device.type != "cuda":
        raise ValueError("scores must be on a GPU device")
    n, m = scores.shape
    ld = scores.stride(0)
    if (m > 1 and scores.stride(1) != 1) or (n > 1 and ld < m):
        scores = scores.contiguous()
        ld = m
    return scores, code, n, m, max(ld, m)


def _grad_buf(grad, scores):
    """The gradient of a score matrix: a caller's (n, m) tensor of its type with contiguous rows, or a new one."""
    if grad is None:
        return torch.empty(scores.shape, dtype=scores.dtype, device=scores.device)
    n, m = scores.shape
    if not isinstance(grad, torch.Tensor) or grad.dtype != scores.dtype or grad.device != scores.device:
        raise ValueError(f"grad must be a {scores.dtype} tensor on {scores.device}")
    if grad.shape != scores.shape or (m > 1 and grad.stride(1) != 1) or (n > 1 and grad.stride(0) < m):
        raise ValueError(f"grad must be ({n}, {m}) with contiguous rows (got {tuple(grad.shape)})")
    return grad


def _vec(t, n, dtype, device, name):
    """An optional (n,) input (or of shape n, a tuple), contiguous."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be a {dtype} tensor on {device}")
    if tuple(t.shape) != (n if isinstance(n, tuple) else (n,)):
        raise ValueError(f"{name} must have shape {n if isinstance(n, tuple) else (n,)} (got {tuple(t.shape)})")
    return t.contiguous()


def _addr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _out(t, shape, dtype, device, name: str) -> torch.Tensor:
    """_buf, without its checks where there is nothing to check (a call on a few rows is bound by the host)."""
    return torch.empty(shape, dtype=dtype, device=device) if t is None else _buf(t, shape, dtype, device, name)


def _call(name: str, device, *args):
    """Calls an entry point on the scores' device and its current stream (the last argument)."""
    fn = getattr(_lib or load_library(), name)
    # the handle alone: a Stream object for it costs as much host time as a third of a small call
    stream = torch._C._cuda_getCurrentRawStream(device.index)
    if torch.cuda.current_device() == device.index:
        code = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            code = fn(*args, stream)
    if code:
        _raise(code, name)


def scores_solve_workspace(n: int, m: int, device) -> torch.Tensor:
    """A workspace tensor for scores_solve on an (n, m) score matrix."""
    nb = int(load_library().sk_scores_solve_workspace_bytes(n, m))
    if nb == 0:
        raise ValueError(f"invalid problem size n={n} m={m} (n >= 1, 1 <= m <= 1024)")
    return torch.empty(nb, dtype=torch.uint8, device=device)


def scores_solve(scores, a=None, b=None, *, eps: float, n_iters: int, g_init: torch.Tensor | None = None,
                 ws: torch.Tensor | None = None, f: torch.Tensor | None = None, g: torch.Tensor | None = None,
                 check: bool = True):
    """Sinkhorn potentials (f (n,), g (m,)) of a given score matrix (cost -scores), from g_init or 0.

    For a router, rows are tokens (a: zero for padding) and columns experts (b: their capacities); a and b default
    to uniform weights.  g (plus eps * log b where b is not uniform) is the bias for balance that ``scores_route``
    takes with select_on="logit".  g_init may be g itself.  An expert is best switched off by b = 0: a column masked by
    -inf in every row is summed anew in every iteration.  With check, given weights are validated as in
    ``check_inputs`` (this waits for the stream)."""
    s, code, n, m, ld = _scores(scores)
    a, b = _vec(a, n, torch.float32, s.device, "a"), _vec(b, m, torch.float32, s.device, "b")
    if check and (a is not None or b is not None):
        aa = torch.full((n,), 1.0 / n, dtype=torch.float32, device=s.device) if a is None else a
        bb = torch.full((m,), 1.0 / m, dtype=torch.float32, device=s.device) if b is None else b
        with torch.cuda.device(s.device):
            check_inputs(aa[:, None], bb[:, None], aa, bb)
    g_init = _vec(g_init, m, torch.float32, s.device, "g_init")
    ws = _ws(ws, s.device, lambda: scores_solve_workspace(n, m, s.device))
    f = _out(f, (n,), torch.float32, s.device, "f")
    g = _out(g, (m,), torch.float32, s.device, "g")
    _call("sk_scores_solve", s.device, s.data_ptr(), code, n, m, ld, _addr(a), _addr(b), float(eps), int(n_iters),
          _addr(g_init), _addr(f), _addr(g), _addr(ws), ws.numel())
    return f, g


class Routing(NamedTuple):
    """Chosen experts (n, k) int32, their weights (n, k) float32, and rows per expert (m,) int32 or None."""
    idx: torch.Tensor
    weights: torch.Tensor
    counts: torch.Tensor | None


def scores_route(scores, k: int, *, score_fn: str = "softmax", bias: torch.Tensor | None = None,
                 select_on: str = "score", n_group: int = 1, topk_group: int = 1, group_top: int = 1,
                 renorm: bool = True, scale: float = 1.0, counts: bool = False,
                 out: Routing | None = None) -> Routing:
    """The k experts of every row of a score matrix and their weights.

    The choice is by softmax or sigmoid of the scores (select_on="score"), or by the scores themselves ("logit"),
    plus bias (m,), in the order of these values in float64 (without a bias in that of the scores themselves); with
    n_group > 1 inside the topk_group best groups of columns (by the sum of a group's group_top largest values).  The
    weights are the softmax or sigmoid at the choice, divided by their sum with renorm, times scale.  ``out``: a Routing of earlier buffers to write into."""
    if score_fn not in SCORE_FNS or select_on not in SELECT_ON:
        raise ValueError(f"score_fn must be one of {list(SCORE_FNS)}, select_on one of {list(SELECT_ON)}")
    s, code, n, m, ld = _scores(scores)
    k = int(k)
    if not 1 <= k <= m:
        raise ValueError(f"k must be between 1 and the {m} columns (got {k})")
    bias = _vec(bias, m, torch.float32, s.device, "bias")
    o_idx, o_weights, o_counts = out or (None, None, None)
    idx = _out(o_idx, (n, k), torch.int32, s.device, "out.idx")
    weights = _out(o_weights, (n, k), torch.float32, s.device, "out.weights")
    cnt = _out(o_counts, (m,), torch.int32, s.device, "out.counts") if counts else None
    _call("sk_scores_route", s.device, s.data_ptr(), code, n, m, ld, SCORE_FNS[score_fn], _addr(bias),
          SELECT_ON[select_on], int(n_group), int(topk_group), int(group_top), k, int(bool(renorm)), float(scale),
          idx.data_ptr(), weights.data_ptr(), _addr(cnt))
    return Routing(idx, weights, cnt)


def scores_route_grad(scores, idx, d_weights, *, score_fn: str = "softmax", renorm: bool = True, scale: float = 1.0,
                      grad: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of ``scores_route``'s weights in the scores, for the choice idx (n, k) held fixed; grad may be scores
    itself."""
    if score_fn not in SCORE_FNS:
        raise ValueError(f"score_fn must be one of {list(SCORE_FNS)}")
    s, code, n, m, ld = _scores(scores)
    if not isinstance(idx, torch.Tensor) or idx.dim() != 2 or idx.shape[0] != n:
        raise ValueError(f"idx must be an ({n}, k) int32 tensor")
    k = idx.shape[1]
    idx = _vec(idx, (n, k), torch.int32, s.device, "idx")
    d_weights = _vec(d_weights, (n, k), torch.float32, s.device, "d_weights")
    if d_weights is None:
        raise ValueError("d_weights must be given")
    grad = _grad_buf(grad, s)
    _call("sk_scores_route_grad", s.device, s.data_ptr(), code, n, m, ld, SCORE_FNS[score_fn], idx.data_ptr(),
          d_weights.data_ptr(), k, int(bool(renorm)), float(scale), grad.data_ptr(), max(grad.stride(0), m))
    return grad


class Logprobs(NamedTuple):
    """Of each row: log-probability of its target (or None), log-sum-exp, entropy (or None), the largest entries'
    columns and log-probabilities (or None), and (maximum, log sum) for the gradient."""
    logp: torch.Tensor | None
    lse: torch.Tensor
    entropy: torch.Tensor | None
    top_idx: torch.Tensor | None
    top_logp: torch.Tensor | None
    stats: torch.Tensor


def scores_logprobs_workspace(dtype: torch.dtype, n: int, m: int, top: int, device) -> torch.Tensor:
    """A workspace tensor for scores_logprobs on an (n, m) score matrix of this dtype."""
    nb = int(load_library().sk_scores_logprobs_workspace_bytes(DTYPES.get(dtype, -1), n, m, top))
    if nb == 0:
        raise ValueError(f"invalid arguments for scores_logprobs (dtype={dtype} n={n} m={m} top={top}: top <= 64, "
                         "top <= m, and m <= 2**20 where top > 0)")
    return torch.empty(nb, dtype=torch.uint8, device=device)


def scores_logprobs(scores, targets: torch.Tensor | None = None, *, eps: float = 1.0, top: int = 0,
                    entropy: bool = False, ws: torch.Tensor | None = None, out: Logprobs | None = None) -> Logprobs:
    """Log-probabilities of targets (n,) int64 (negative: no token given) under softmax(scores / eps), with the rows'
    log-sum-exp, their entropy and the ``top`` largest alternatives, in one read of the scores.  ``out``: a Logprobs
    of earlier buffers to write into."""
    s, code, n, m, ld = _scores(scores)
    top = int(top)
    dev = s.device
    targets = _vec(targets, n, torch.int64, dev, "targets")
    ws = _ws(ws, dev, lambda: scores_logprobs_workspace(s.dtype, n, m, top, dev))
    o_logp, o_lse, o_ent, o_idx, o_top, o_stats = out or (None,) * 6
    f32 = torch.float32
    logp = None if targets is None else _out(o_logp, (n,), f32, dev, "out.logp")
    lse = _out(o_lse, (n,), f32, dev, "out.lse")
    ent = _out(o_ent, (n,), f32, dev, "out.entropy") if entropy else None
    top_idx = _out(o_idx, (n, top), torch.int32, dev, "out.top_idx") if top > 0 else None
    top_logp = _out(o_top, (n, top), f32, dev, "out.top_logp") if top > 0 else None
    stats = _out(o_stats, (n, 2), f32, dev, "out.stats")
    _call("sk_scores_logprobs", dev, s.data_ptr(), code, n, m, ld, float(eps), _addr(targets), top, _addr(logp),
          lse.data_ptr(), _addr(ent), _addr(top_idx), _addr(top_logp), stats.data_ptr(), ws.data_ptr(), ws.numel())
    return Logprobs(logp, lse, ent, top_idx, top_logp, stats)


def scores_logprobs_grad(scores, targets: torch.Tensor | None, fwd: Logprobs, *, eps: float = 1.0,
                         d_logp: torch.Tensor | None = None, d_lse: torch.Tensor | None = None,
                         d_entropy: torch.Tensor | None = None, d_top: torch.Tensor | None = None,
                         grad: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of ``scores_logprobs`` in the scores from the gradients of its outputs (each optional; d_top is that
    of top_logp); fwd is its result for the same scores, targets and eps.  grad may be scores itself; for a window of
    padded rows a grad of the same row stride is written fastest (a new one is contiguous)."""
    s, code, n, m, ld = _scores(scores)
    dev = s.device
    targets = _vec(targets, n, torch.int64, dev, "targets")
    stats = _in(fwd.stats, (n, 2), dev, "fwd.stats")
    if d_logp is not None and targets is None:
        raise ValueError("d_logp needs targets")
    if d_entropy is not None and fwd.entropy is None:
        raise ValueError("d_entropy needs the forward's entropy")
    if d_top is not None and fwd.top_idx is None:
        raise ValueError("d_top needs the forward's top_idx")
    top = 0 if d_top is None else fwd.top_idx.shape[1]
    ent = None if d_entropy is None else _vec(fwd.entropy, n, torch.float32, dev, "fwd.entropy")
    top_idx = None if d_top is None else _vec(fwd.top_idx, (n, top), torch.int32, dev, "fwd.top_idx")
    d_logp, d_lse = _vec(d_logp, n, torch.float32, dev, "d_logp"), _vec(d_lse, n, torch.float32, dev, "d_lse")
    d_entropy = _vec(d_entropy, n, torch.float32, dev, "d_entropy")
    d_top = _vec(d_top, (n, top), torch.float32, dev, "d_top")
    grad = _grad_buf(grad, s)
    _call("sk_scores_logprobs_grad", dev, s.data_ptr(), code, n, m, ld, float(eps), _addr(targets), stats.data_ptr(),
          _addr(ent), top, _addr(top_idx), _addr(d_logp), _addr(d_lse), _addr(d_entropy), _addr(d_top), grad.data_ptr(),
          max(grad.stride(0), m))
    return grad


def timing_enable(enable: bool = True, stride: int = 1) -> None:
    """Start (reset) or stop event timing of the streamed-pass kernels; every
    stride-th pass launch is timed."""
    if stride < 1:
        raise ValueError("stride must be >= 1")
    _raise(load_library().sk_timing_enable(int(stride) if enable else 0), "sk_timing_enable")


def timing_read() -> tuple[float, int, float]:
    """(total kernel ms, launches, pairs evaluated) since timing_enable(True)."""
    ms, n, pairs = ctypes.c_double(), ctypes.c_int64(), ctypes.c_double()
    _raise(load_library().sk_timing_read(ctypes.byref(ms), ctypes.byref(n), ctypes.byref(pairs)), "sk_timing_read")
    return ms.value, n.value, pairs.value


__all__ = ["timing_enable", "timing_read", "solve", "solve_ex", "gradient_flow", "transport", "hvp", "fs2_solve",
           "transport_workspace", "cost", "dual_cost", "divergence",
           "divergence_workspace", "marginal_residual", "grad_x", "check_inputs", "workspace", "workspace_bytes",
           "load_library", "status_string", "SinkhornError", "LIB_PATH", "SIGNATURES", "VARIANTS", "STOP_MODES",
           "solve_noalloc", "NOALLOC_SCRATCH_BYTES", "solve_warm", "primal_cost",
           "scores_solve", "scores_solve_workspace", "scores_route", "scores_route_grad", "Routing", "scores_logprobs",
           "scores_logprobs_grad", "scores_logprobs_workspace", "Logprobs", "DTYPES", "SCORE_FNS", "SELECT_ON"]
