"""Python binding of libswimba.so: the same entry points as include/swimba.h,
taking torch tensors.  Argument marshalling only -- every step of the
computation runs in the HIP kernels; torch provides device memory and the
current stream.  There is no fallback: without the built library every call
raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libswimba.so")

F32, BF16 = 0, 1
OK, EINVAL, EUNSUPPORTED, EWORKSPACE, EHIP, ESCRATCH = 0, -1, -2, -3, -4, -5
# fixed chunk-workspace buffer of swimba_scan_noalloc (SWIMBA_NOALLOC_SCRATCH_BYTES)
NOALLOC_SCRATCH_BYTES = 64 << 20
CARRY = {"auto": 0, "rewalk": 1, "fixup": 2}
A_DIAGONAL, A_SCALAR = 0, 1  # A [E, D, N] or [E, D] (one transition per channel)
DISC_EULER, DISC_ZOH = 0, 1  # input term Delta B x, or zero-order hold
N_STATE = 16

_vp = ctypes.c_void_p
_ci = ctypes.c_int


class ScanArgs(ctypes.Structure):
    _fields_ = [("B", _ci), ("L", _ci), ("D", _ci), ("N", _ci), ("E", _ci), ("k", _ci),
                ("in_dtype", _ci), ("y_dtype", _ci),
                ("x", _vp), ("dt_raw", _vp), ("Bm", _vp), ("Cm", _vp),
                ("idx", _vp), ("gate", _vp), ("A", _vp), ("dt_bias", _vp), ("Dskip", _vp),
                ("h0", _vp), ("y", _vp), ("h_final", _vp),
                ("chunk", _ci), ("carry", _ci), ("phase_events", _vp), ("a_form", _ci),
                ("disc", _ci)]


class StepArgs(ctypes.Structure):
    _fields_ = [("B", _ci), ("D", _ci), ("N", _ci), ("E", _ci), ("k", _ci),
                ("in_dtype", _ci), ("y_dtype", _ci),
                ("x", _vp), ("dt_raw", _vp), ("Bm", _vp), ("Cm", _vp),
                ("Wr", _vp), ("idx", _vp), ("gate", _vp), ("idx_out", _vp), ("gate_out", _vp),
                ("A", _vp), ("dt_bias", _vp), ("Dskip", _vp), ("state", _vp), ("y", _vp),
                ("a_form", _ci), ("disc", _ci)]


class GradArgs(ctypes.Structure):
    _fields_ = [("fwd", ScanArgs), ("dy", _vp), ("dy_dtype", _ci), ("dh_final", _vp),
                ("dx", _vp), ("ddt_raw", _vp), ("dBm", _vp), ("dCm", _vp), ("dgate", _vp),
                ("dA", _vp), ("ddt_bias", _vp), ("dDskip", _vp), ("dh0", _vp)]


class StreamArgs(ctypes.Structure):
    _fields_ = [("B", _ci), ("L", _ci), ("D", _ci), ("N", _ci), ("k", _ci),
                ("in_dtype", _ci), ("y_dtype", _ci),
                ("X", _vp), ("dt_raw", _vp), ("Bs", _vp), ("Cs", _vp), ("gate", _vp),
                ("A", _vp), ("dt_bias", _vp), ("h0", _vp), ("y", _vp), ("h_final", _vp),
                ("chunk", _ci), ("carry", _ci), ("phase_events", _vp)]


class LinearAttentionArgs(ctypes.Structure):
    _fields_ = [("B", _ci), ("L", _ci), ("H", _ci), ("G", _ci), ("N", _ci), ("P", _ci),
                ("in_dtype", _ci), ("y_dtype", _ci), ("decay_form", _ci),
                ("q", _vp), ("k", _vp), ("v", _vp), ("log_decay", _vp), ("h0", _vp),
                ("y", _vp), ("h_final", _vp)]


class LinearAttentionGradArgs(ctypes.Structure):
    _fields_ = [("fwd", LinearAttentionArgs), ("dy", _vp), ("dh_final", _vp),
                ("grad_dtype", _ci), ("dq", _vp), ("dk", _vp), ("dv", _vp), ("dlog_decay", _vp),
                ("dh0", _vp)]


class LinearAttentionStepArgs(ctypes.Structure):
    _fields_ = [("B", _ci), ("H", _ci), ("G", _ci), ("N", _ci), ("P", _ci),
                ("in_dtype", _ci), ("y_dtype", _ci), ("decay_form", _ci),
                ("q", _vp), ("k", _vp), ("v", _vp), ("log_decay", _vp), ("state", _vp),
                ("state_out", _vp), ("y", _vp)]


class DeltaRuleArgs(ctypes.Structure):
    _fields_ = [("B", _ci), ("L", _ci), ("H", _ci), ("G", _ci), ("N", _ci), ("P", _ci),
                ("in_dtype", _ci), ("y_dtype", _ci), ("decay_form", _ci),
                ("q", _vp), ("k", _vp), ("v", _vp), ("log_decay", _vp), ("beta", _vp),
                ("h0", _vp), ("y", _vp), ("h_final", _vp)]


class DeltaRuleGradArgs(ctypes.Structure):
    _fields_ = [("fwd", DeltaRuleArgs), ("dy", _vp), ("dh_final", _vp), ("grad_dtype", _ci),
                ("dq", _vp), ("dk", _vp), ("dv", _vp), ("dlog_decay", _vp), ("dbeta", _vp),
                ("dh0", _vp)]


class DeltaRuleStepArgs(ctypes.Structure):
    _fields_ = [("B", _ci), ("H", _ci), ("G", _ci), ("N", _ci), ("P", _ci),
                ("in_dtype", _ci), ("y_dtype", _ci), ("decay_form", _ci),
                ("q", _vp), ("k", _vp), ("v", _vp), ("log_decay", _vp), ("beta", _vp),
                ("state", _vp), ("state_out", _vp), ("y", _vp)]


class NormRotateArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("Hq", _ci), ("Hk", _ci), ("N", _ci), ("R", _ci),
                ("in_dtype", _ci), ("out_dtype", _ci), ("norm", _ci), ("pairs", _ci),
                ("eps", ctypes.c_float), ("q_scale", ctypes.c_float),
                ("q", _vp), ("k", _vp), ("q_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("wq", _vp), ("wk", _vp), ("positions", _vp),
                ("rates", _vp), ("q_out", _vp), ("k_out", _vp)]


class NormRotateGradArgs(ctypes.Structure):
    _fields_ = [("fwd", NormRotateArgs), ("dq_out", _vp), ("dk_out", _vp), ("grad_dtype", _ci),
                ("dq", _vp), ("dk", _vp), ("dwq", _vp), ("dwk", _vp)]


class SwimbaError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__("%s failed: %s (%d)" % (fn, status_string(status), status))
        self.status = status


_lib = None


def load(path: str | None = None):
    """Load libswimba.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    so = path or LIB_PATH
    if not os.path.exists(so):
        raise ImportError("libswimba.so is not built (%s); run __graft_entry__.build() or "
                          "python parameter_space_moe_amd/build.py" % so)
    lib = ctypes.CDLL(so)
    lib.swimba_route.argtypes = [_vp, _ci, _vp, ctypes.c_int64, _ci, _ci, _ci, _vp, _vp, _vp]
    lib.swimba_route.restype = _ci
    lib.swimba_scan_workspace_size.argtypes = [ctypes.POINTER(ScanArgs), _ci]
    lib.swimba_scan_workspace_size.restype = ctypes.c_size_t
    for fn in (lib.swimba_scan, lib.swimba_scan_separate, lib.swimba_scan_slots,
               lib.swimba_scan_all_experts):
        fn.argtypes = [ctypes.POINTER(ScanArgs), _vp, ctypes.c_size_t, _vp]
        fn.restype = _ci
    lib.swimba_scan_noalloc.argtypes = [ctypes.POINTER(ScanArgs), _vp]
    lib.swimba_scan_noalloc.restype = _ci
    lib.swimba_scan_plan.argtypes = [ctypes.POINTER(ScanArgs), _ci, ctypes.POINTER(_ci),
                                     ctypes.POINTER(_ci)]
    lib.swimba_scan_plan.restype = _ci
    lib.swimba_scan_streams_workspace_size.argtypes = [ctypes.POINTER(StreamArgs)]
    lib.swimba_scan_streams_workspace_size.restype = ctypes.c_size_t
    lib.swimba_scan_streams_plan.argtypes = [ctypes.POINTER(StreamArgs), ctypes.POINTER(_ci),
                                             ctypes.POINTER(_ci)]
    lib.swimba_scan_streams_plan.restype = _ci
    lib.swimba_scan_streams.argtypes = [ctypes.POINTER(StreamArgs), _vp, ctypes.c_size_t, _vp]
    lib.swimba_scan_streams.restype = _ci
    lib.swimba_scan_backward_workspace_size.argtypes = [ctypes.POINTER(GradArgs)]
    lib.swimba_scan_backward_workspace_size.restype = ctypes.c_size_t
    lib.swimba_scan_backward.argtypes = [ctypes.POINTER(GradArgs), _vp, ctypes.c_size_t, _vp]
    lib.swimba_scan_backward.restype = _ci
    lib.swimba_step.argtypes = [ctypes.POINTER(StepArgs), _vp]
    lib.swimba_step.restype = _ci
    _i64, _sz = ctypes.c_int64, ctypes.c_size_t
    lib.swimba_sort_tokens_workspace_size.argtypes = [_i64, _ci, _ci]
    lib.swimba_sort_tokens_workspace_size.restype = _sz
    lib.swimba_sort_tokens.argtypes = [_vp, _i64, _ci, _ci, _vp, _vp, _vp, _vp, _sz, _vp]
    lib.swimba_sort_tokens.restype = _ci
    lib.swimba_dispatch_tokens.argtypes = [_vp, _ci, _vp, _i64, _ci, _ci, _vp, _vp]
    lib.swimba_dispatch_tokens.restype = _ci
    lib.swimba_combine_tokens.argtypes = [_vp, _ci, _vp, _vp, _i64, _ci, _ci, _vp, _ci, _vp]
    lib.swimba_combine_tokens.restype = _ci
    lib.swimba_combine_tokens_backward.argtypes = [_vp, _ci, _vp, _vp, _vp, _ci, _i64, _ci, _ci,
                                                   _vp, _ci, _vp, _vp]
    lib.swimba_combine_tokens_backward.restype = _ci
    lib.swimba_route_backward_workspace_size.argtypes = [_i64, _ci, _ci]
    lib.swimba_route_backward_workspace_size.restype = _sz
    lib.swimba_route_backward.argtypes = [_vp, _ci, _vp, _vp, _vp, _vp, _i64, _ci, _ci, _ci, _vp,
                                          _ci, _vp, _vp, _sz, _vp]
    lib.swimba_route_backward.restype = _ci
    for fn, args in ((lib.swimba_linear_attention, LinearAttentionArgs),
                     (lib.swimba_linear_attention_backward, LinearAttentionGradArgs),
                     (lib.swimba_delta_rule, DeltaRuleArgs),
                     (lib.swimba_delta_rule_backward, DeltaRuleGradArgs),
                     (lib.swimba_norm_rotate_backward, NormRotateGradArgs)):
        fn.argtypes = [ctypes.POINTER(args), _vp, _sz, _vp]
        fn.restype = _ci
    for fn, args in ((lib.swimba_linear_attention_workspace_size, LinearAttentionArgs),
                     (lib.swimba_linear_attention_backward_workspace_size,
                      LinearAttentionGradArgs),
                     (lib.swimba_delta_rule_workspace_size, DeltaRuleArgs),
                     (lib.swimba_delta_rule_backward_workspace_size, DeltaRuleGradArgs),
                     (lib.swimba_norm_rotate_backward_workspace_size, NormRotateGradArgs)):
        fn.argtypes = [ctypes.POINTER(args)]
        fn.restype = _sz
    for fn, args in ((lib.swimba_linear_attention_step, LinearAttentionStepArgs),
                     (lib.swimba_delta_rule_step, DeltaRuleStepArgs),
                     (lib.swimba_norm_rotate, NormRotateArgs)):
        fn.argtypes = [ctypes.POINTER(args), _vp]
        fn.restype = _ci
    lib.swimba_status_string.argtypes = [_ci]
    lib.swimba_status_string.restype = ctypes.c_char_p
    if path is None:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().swimba_status_string(status).decode()


def _check(fn, rc):
    if rc != OK:
        raise SwimbaError(fn, rc)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError("expected float32 or bfloat16, got %s" % t.dtype)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, shape=None, dtype=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _hold(stream, *tensors):
    """Temporaries allocated here for a call on the caller's stream: the
    caching allocator must not hand them out again before that stream's
    work has run (allocation is ordered on the current stream only)."""
    if stream is not None:
        for t in tensors:
            t.record_stream(stream)


def route(x: torch.Tensor, Wr: torch.Tensor, k: int, idx=None, gate=None, stream=None):
    """Top-k router: x [..., D] (f32/bf16), Wr [D, E] f32 -> idx [..., k] int32,
    gate [..., k] f32 (include/swimba.h: swimba_route)."""
    _need(x, "x")
    D = x.shape[-1]
    E = Wr.shape[1] if Wr.dim() == 2 else -1
    _need(Wr, "Wr", (D, E), torch.float32, x.device)
    T = x.numel() // D if D else 0
    lead = tuple(x.shape[:-1])
    if idx is None:
        idx = torch.empty(lead + (k,), dtype=torch.int32, device=x.device)
    if gate is None:
        gate = torch.empty(lead + (k,), dtype=torch.float32, device=x.device)
    _need(idx, "idx", lead + (k,), torch.int32, x.device)
    _need(gate, "gate", lead + (k,), torch.float32, x.device)
    rc = load().swimba_route(_ptr(x), _dt(x), _ptr(Wr), T, D, E, k, _ptr(idx), _ptr(gate),
                             _stream(stream))
    _check("swimba_route", rc)
    return idx, gate


def _scan_args(x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, h0, y, h_final, chunk, carry,
               design, phase_events, need_y=True, zoh=False):
    _need(x, "x")
    if x.dim() != 3:
        raise ValueError("x must be [B, L, D]")
    B, L, D = x.shape
    E = A.shape[0]
    N = Bm.shape[2] if Bm.dim() == 3 else -1
    k = idx.shape[2] if idx.dim() == 3 else -1
    dev = x.device
    _need(dt_raw, "dt_raw", (B, L, D), x.dtype, dev)
    _need(Bm, "Bm", (B, L, N), x.dtype, dev)
    _need(Cm, "Cm", (B, L, N), x.dtype, dev)
    _need(idx, "idx", (B, L, k), torch.int32, dev)
    _need(gate, "gate", (B, L, k), torch.float32, dev)
    scalar_a = A.dim() == 2
    _need(A, "A", (E, D) if scalar_a else (E, D, N), torch.float32, dev)
    _need(dt_bias, "dt_bias", (E, D), torch.float32, dev)
    _need(Dskip, "Dskip", (E, D), torch.float32, dev)
    sshape = _state_shape(design, B, E, k, D, N)
    if h0 is not None:
        _need(h0, "h0", sshape, torch.float32, dev)
    if need_y:
        _need(y, "y", (B, L, D), None, dev)
    if h_final is not None:
        _need(h_final, "h_final", sshape, torch.float32, dev)
    a = ScanArgs()
    a.B, a.L, a.D, a.N, a.E, a.k = B, L, D, N, E, k
    a.in_dtype, a.y_dtype = _dt(x), (_dt(y) if y is not None else _dt(x))
    a.x, a.dt_raw, a.Bm, a.Cm = _ptr(x), _ptr(dt_raw), _ptr(Bm), _ptr(Cm)
    a.idx, a.gate, a.A, a.dt_bias, a.Dskip = _ptr(idx), _ptr(gate), _ptr(A), _ptr(dt_bias), \
        _ptr(Dskip)
    a.h0, a.y, a.h_final = _ptr(h0), _ptr(y), _ptr(h_final)
    a.chunk = int(chunk)
    a.carry = CARRY[carry] if isinstance(carry, str) else int(carry)
    a.phase_events = phase_events
    a.a_form = A_SCALAR if scalar_a else A_DIAGONAL
    a.disc = DISC_ZOH if zoh else DISC_EULER
    return a


# Which scan (SWIMBA_DESIGN_* in include/swimba.h); a bool `separate` reads as
# MIXED (False) or SEPARATE (True).
DESIGN_MIXED, DESIGN_SEPARATE, DESIGN_SLOTS, DESIGN_ALL_EXPERTS = 0, 1, 2, 3
_SCAN_FN = {DESIGN_MIXED: "swimba_scan", DESIGN_SEPARATE: "swimba_scan_separate",
            DESIGN_SLOTS: "swimba_scan_slots", DESIGN_ALL_EXPERTS: "swimba_scan_all_experts"}


def _state_shape(design, B, E, k, D, N=N_STATE):
    """h0 / h_final shape: one state per (b, d), per (b, expert, d) or per
    (b, slot, d)."""
    design = int(design)
    if design in (DESIGN_SEPARATE, DESIGN_ALL_EXPERTS):
        return (B, E, D, N)
    if design == DESIGN_SLOTS:
        return (B, k, D, N)
    return (B, D, N)


def workspace_size(args: ScanArgs, design) -> int:
    return int(load().swimba_scan_workspace_size(ctypes.byref(args), int(design)))


def _scan(design, x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, h0=None, y=None,
          h_final=None, y_dtype=None, want_state=True, chunk=0, carry="auto", workspace=None,
          stream=None, phase_events=None, zoh=False):
    design = int(design)
    if y is None:
        y = torch.empty(x.shape, dtype=y_dtype or x.dtype, device=x.device)
    if h_final is None and want_state:
        shape = _state_shape(design, x.shape[0], A.shape[0], idx.shape[-1], x.shape[2])
        h_final = torch.empty(shape, dtype=torch.float32, device=x.device)
    a = _scan_args(x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, h0, y, h_final, chunk, carry,
                   design, phase_events, zoh=zoh)
    lib = load()
    need = workspace_size(a, design)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
        _hold(stream, workspace)
    name = _SCAN_FN[design]
    rc = getattr(lib, name)(ctypes.byref(a), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(name, rc)
    return y, h_final


def scan(x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, h0=None, **kw):
    """Parameter-space-mixed scan (include/swimba.h: swimba_scan).  A is
    [E,D,16], or [E,D] for one transition per channel (the scalar form).
    Returns (y [B,L,D], h_final [B,D,16] or None)."""
    return _scan(False, x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, h0, **kw)


def scan_noalloc(x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, h0=None, y=None,
                 h_final=None, y_dtype=None, want_state=True, chunk=0, carry="auto",
                 stream=None, zoh=False):
    """The mixed scan with its chunk workspace in the library's fixed buffer
    (include/swimba.h: swimba_scan_noalloc): no workspace is allocated for
    the call.  Outputs y and h_final are allocated here unless given.
    Returns (y [B,L,D], h_final [B,D,16] or None)."""
    if y is None:
        y = torch.empty(x.shape, dtype=y_dtype or x.dtype, device=x.device)
    if h_final is None and want_state:
        h_final = torch.empty((x.shape[0], x.shape[2], N_STATE), dtype=torch.float32,
                              device=x.device)
    a = _scan_args(x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, h0, y, h_final, chunk, carry,
                   DESIGN_MIXED, None, zoh=zoh)
    rc = load().swimba_scan_noalloc(ctypes.byref(a), _stream(stream))
    _check("swimba_scan_noalloc", rc)
    return y, h_final


def scan_separate(x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, h0=None, **kw):
    """Separate design (include/swimba.h: swimba_scan_separate).  Returns
    (y [B,L,D], h_final [B,E,D,16] or None)."""
    return _scan(DESIGN_SEPARATE, x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, h0, **kw)


def scan_slots(x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, h0=None, **kw):
    """Separate trajectories per routing slot (include/swimba.h:
    swimba_scan_slots).  Returns (y [B,L,D], h_final [B,k,D,16] or None)."""
    return _scan(DESIGN_SLOTS, x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, h0, **kw)


def scan_all_experts(x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, h0=None, **kw):
    """Separate trajectories where every expert advances at every token
    (include/swimba.h: swimba_scan_all_experts).  Returns (y [B,L,D],
    h_final [B,E,D,16] or None)."""
    return _scan(DESIGN_ALL_EXPERTS, x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, h0, **kw)


def _grad_args(x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, dy, h0, dh_final, chunk,
               out):
    a = _scan_args(x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, h0, None, None, chunk,
                   "auto", False, None, need_y=False)
    B, L, D = x.shape
    E, k = A.shape[0], idx.shape[2]
    N = Bm.shape[2]
    dev = x.device
    _need(dy, "dy", (B, L, D), None, dev)
    if dh_final is not None:
        _need(dh_final, "dh_final", (B, D, N), torch.float32, dev)
    shapes = {"dx": (B, L, D), "ddt_raw": (B, L, D), "dBm": (B, L, N), "dCm": (B, L, N),
              "dgate": (B, L, k), "dA": tuple(A.shape), "ddt_bias": (E, D), "dDskip": (E, D),
              "dh0": (B, D, N)}
    for name, shape in shapes.items():
        if out.get(name) is not None:
            _need(out[name], name, shape, torch.float32, dev)
    g = GradArgs()
    g.fwd = a
    g.dy, g.dy_dtype, g.dh_final = _ptr(dy), _dt(dy), _ptr(dh_final)
    for name in shapes:
        setattr(g, name, _ptr(out.get(name)))
    return g


def scan_backward(x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, dy, h0=None, dh_final=None,
                  chunk=0, want_dh0=True, out=None, workspace=None, stream=None):
    """Gradients of the mixed scan (include/swimba.h: swimba_scan_backward) for
    dL/dy = dy (and dL/dh_final).  Returns a dict of fp32 tensors: dx,
    ddt_raw [B,L,D]; dBm, dCm [B,L,16]; dgate [B,L,k]; dA [E,D,16]; ddt_bias,
    dDskip [E,D]; dh0 [B,D,16] (when want_dh0)."""
    B, L, D = x.shape
    E, k, N = A.shape[0], idx.shape[2], N_STATE
    dev = x.device
    out = dict(out or {})
    shapes = {"dx": (B, L, D), "ddt_raw": (B, L, D), "dBm": (B, L, N), "dCm": (B, L, N),
              "dgate": (B, L, k), "dA": tuple(A.shape), "ddt_bias": (E, D), "dDskip": (E, D)}
    if want_dh0:
        shapes["dh0"] = (B, D, N)
    for name, shape in shapes.items():
        if out.get(name) is None:
            out[name] = torch.empty(shape, dtype=torch.float32, device=dev)
    g = _grad_args(x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, dy, h0, dh_final, chunk, out)
    lib = load()
    need = int(lib.swimba_scan_backward_workspace_size(ctypes.byref(g)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        _hold(stream, workspace)
    rc = lib.swimba_scan_backward(ctypes.byref(g), _ptr(workspace), workspace.numel(),
                                  _stream(stream))
    _check("swimba_scan_backward", rc)
    return out


class PreparedBackward:
    """swimba_scan_backward marshalled once (see PreparedScan)."""

    def __init__(self, x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, dy, out, h0=None,
                 dh_final=None, chunk=0, workspace=None, stream=None):
        self.args = _grad_args(x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, dy, h0, dh_final,
                               chunk, out)
        lib = load()
        need = int(lib.swimba_scan_backward_workspace_size(ctypes.byref(self.args)))
        self.workspace = workspace if workspace is not None else torch.empty(
            max(need, 1), dtype=torch.uint8, device=x.device)
        self._keep = (x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, dy, h0, dh_final, out)
        self._fn = lib.swimba_scan_backward
        self._ref = ctypes.byref(self.args)
        self._ws = self.workspace.data_ptr()
        self._wsn = self.workspace.numel()
        self.stream = _stream(stream)

    def __call__(self):
        rc = self._fn(self._ref, self._ws, self._wsn, self.stream)
        if rc != OK:
            raise SwimbaError("swimba_scan_backward", rc)


def _shape_args(x, A, idx, chunk, y_dtype):
    B, L, D = x.shape
    a = ScanArgs()
    a.B, a.L, a.D, a.N, a.E, a.k = B, L, D, N_STATE, A.shape[0], idx.shape[2]
    a.a_form = A_SCALAR if A.dim() == 2 else A_DIAGONAL
    a.in_dtype = _dt(x)
    a.y_dtype = a.in_dtype if y_dtype is None else (BF16 if y_dtype == torch.bfloat16 else F32)
    a.chunk = chunk
    return a


def scan_workspace_bytes(x, A, idx, separate=False, chunk=0, y_dtype=None):
    """Workspace bytes the scan named by `separate` (a DESIGN_* value, or a
    bool for mixed / separate) needs for these shapes."""
    return workspace_size(_shape_args(x, A, idx, chunk, y_dtype), separate)


def scan_plan(x, A, idx, separate=False, chunk=0):
    """(tokens per chunk, number of chunks) the scan will use (swimba_scan_plan);
    `separate` as in scan_workspace_bytes."""
    c, n = _ci(), _ci()
    rc = load().swimba_scan_plan(ctypes.byref(_shape_args(x, A, idx, chunk, None)),
                                 int(separate), ctypes.byref(c), ctypes.byref(n))
    _check("swimba_scan_plan", rc)
    return c.value, n.value


class PreparedScan:
    """A scan call marshalled once (argument struct, workspace) for callers
    that issue the same call repeatedly; __call__ goes straight to the C ABI."""

    def __init__(self, separate, x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, h0=None,
                 y=None, h_final=None, chunk=0, carry="auto", workspace=None, stream=None,
                 zoh=False):
        # separate: a DESIGN_* value, or a bool for mixed / separate
        design = int(separate)
        self.args = _scan_args(x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, h0, y, h_final,
                               chunk, carry, design, None, zoh=zoh)
        need = workspace_size(self.args, design)
        self.workspace = workspace if workspace is not None else torch.empty(
            max(need, 1), dtype=torch.uint8, device=x.device)
        self._keep = (x, dt_raw, Bm, Cm, idx, gate, A, dt_bias, Dskip, h0, y, h_final)
        lib = load()
        self._name = _SCAN_FN[design]
        self._fn = getattr(lib, self._name)
        self._ref = ctypes.byref(self.args)
        self._ws = self.workspace.data_ptr()
        self._wsn = self.workspace.numel()
        self.stream = _stream(stream)

    def __call__(self, phase_events=None):
        self.args.phase_events = phase_events
        rc = self._fn(self._ref, self._ws, self._wsn, self.stream)
        if rc != OK:
            raise SwimbaError(self._name, rc)


def _stream_args(X, dt_raw, Bs, Cs, gate, A, dt_bias, h0, y, h_final, chunk, carry,
                 phase_events):
    _need(X, "X")
    if X.dim() != 4:
        raise ValueError("X must be [B, L, k, D]")
    B, L, k, D = X.shape
    N = A.shape[1] if A.dim() == 2 else -1
    dev = X.device
    _need(dt_raw, "dt_raw", (B, L, D), X.dtype, dev)
    _need(Bs, "Bs", (B, L, k, N), X.dtype, dev)
    _need(Cs, "Cs", (B, L, k, N), X.dtype, dev)
    _need(gate, "gate", (B, L, k), torch.float32, dev)
    _need(A, "A", (D, N), torch.float32, dev)
    _need(dt_bias, "dt_bias", (D,), torch.float32, dev)
    if h0 is not None:
        _need(h0, "h0", (B, D, N), torch.float32, dev)
    _need(y, "y", (B, L, D), None, dev)
    if h_final is not None:
        _need(h_final, "h_final", (B, D, N), torch.float32, dev)
    a = StreamArgs()
    a.B, a.L, a.D, a.N, a.k = B, L, D, N, k
    a.in_dtype, a.y_dtype = _dt(X), _dt(y)
    a.X, a.dt_raw, a.Bs, a.Cs, a.gate = _ptr(X), _ptr(dt_raw), _ptr(Bs), _ptr(Cs), _ptr(gate)
    a.A, a.dt_bias, a.h0, a.y, a.h_final = _ptr(A), _ptr(dt_bias), _ptr(h0), _ptr(y), \
        _ptr(h_final)
    a.chunk = int(chunk)
    a.carry = CARRY[carry] if isinstance(carry, str) else int(carry)
    a.phase_events = phase_events
    return a


def scan_streams(X, dt_raw, Bs, Cs, gate, A, dt_bias, h0=None, y=None, h_final=None,
                 y_dtype=None, want_state=True, chunk=0, carry="auto", workspace=None,
                 stream=None, phase_events=None):
    """Stream-mixed scan (include/swimba.h: swimba_scan_streams).  X [B,L,k,D];
    dt_raw [B,L,D]; Bs, Cs [B,L,k,16]; gate [B,L,k] f32; A [D,16], dt_bias [D]
    f32.  Returns (y [B,L,D], h_final [B,D,16] or None)."""
    B, L, k, D = X.shape
    if y is None:
        y = torch.empty((B, L, D), dtype=y_dtype or X.dtype, device=X.device)
    if h_final is None and want_state:
        h_final = torch.empty((B, D, N_STATE), dtype=torch.float32, device=X.device)
    a = _stream_args(X, dt_raw, Bs, Cs, gate, A, dt_bias, h0, y, h_final, chunk, carry,
                     phase_events)
    lib = load()
    need = int(lib.swimba_scan_streams_workspace_size(ctypes.byref(a)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=X.device)
        _hold(stream, workspace)
    rc = lib.swimba_scan_streams(ctypes.byref(a), _ptr(workspace), workspace.numel(),
                                 _stream(stream))
    _check("swimba_scan_streams", rc)
    return y, h_final


def scan_streams_plan(X, chunk=0):
    """(tokens per chunk, number of chunks) of swimba_scan_streams for X [B,L,k,D]."""
    a = StreamArgs()
    a.B, a.L, a.k, a.D = X.shape
    a.N = N_STATE
    a.in_dtype = a.y_dtype = _dt(X)
    a.chunk = chunk
    c, n = _ci(), _ci()
    rc = load().swimba_scan_streams_plan(ctypes.byref(a), ctypes.byref(c), ctypes.byref(n))
    _check("swimba_scan_streams_plan", rc)
    return c.value, n.value


class PreparedStreams:
    """swimba_scan_streams marshalled once (see PreparedScan)."""

    def __init__(self, X, dt_raw, Bs, Cs, gate, A, dt_bias, h0=None, y=None, h_final=None,
                 chunk=0, carry="auto", workspace=None, stream=None):
        self.args = _stream_args(X, dt_raw, Bs, Cs, gate, A, dt_bias, h0, y, h_final, chunk,
                                 carry, None)
        lib = load()
        need = int(lib.swimba_scan_streams_workspace_size(ctypes.byref(self.args)))
        self.workspace = workspace if workspace is not None else torch.empty(
            max(need, 1), dtype=torch.uint8, device=X.device)
        self._keep = (X, dt_raw, Bs, Cs, gate, A, dt_bias, h0, y, h_final)
        self._fn = lib.swimba_scan_streams
        self._ref = ctypes.byref(self.args)
        self._ws = self.workspace.data_ptr()
        self._wsn = self.workspace.numel()
        self.stream = _stream(stream)

    def __call__(self, phase_events=None):
        self.args.phase_events = phase_events
        rc = self._fn(self._ref, self._ws, self._wsn, self.stream)
        if rc != OK:
            raise SwimbaError("swimba_scan_streams", rc)


class PreparedRoute:
    """swimba_route marshalled once (see PreparedScan)."""

    def __init__(self, x, Wr, k, idx, gate, stream=None):
        _need(x, "x")
        D = x.shape[-1]
        E = Wr.shape[1]
        _need(Wr, "Wr", (D, E), torch.float32, x.device)
        lead = tuple(x.shape[:-1])
        _need(idx, "idx", lead + (k,), torch.int32, x.device)
        _need(gate, "gate", lead + (k,), torch.float32, x.device)
        self._keep = (x, Wr, idx, gate)
        self._a = (x.data_ptr(), _dt(x), Wr.data_ptr(), x.numel() // D, D, E, k, idx.data_ptr(),
                   gate.data_ptr(), _stream(stream))
        self._fn = load().swimba_route

    def __call__(self):
        rc = self._fn(*self._a)
        if rc != OK:
            raise SwimbaError("swimba_route", rc)


def _step_args(x, dt_raw, Bm, Cm, A, dt_bias, Dskip, state, Wr, k, idx, gate, y, idx_out,
               gate_out, y_dtype, zoh=False):
    _need(x, "x")
    B, D = x.shape
    E = A.shape[0]
    N = Bm.shape[1] if Bm.dim() == 2 else -1
    dev = x.device
    _need(dt_raw, "dt_raw", (B, D), x.dtype, dev)
    _need(Bm, "Bm", (B, N), x.dtype, dev)
    _need(Cm, "Cm", (B, N), x.dtype, dev)
    scalar_a = A.dim() == 2
    _need(A, "A", (E, D) if scalar_a else (E, D, N), torch.float32, dev)
    _need(dt_bias, "dt_bias", (E, D), torch.float32, dev)
    _need(Dskip, "Dskip", (E, D), torch.float32, dev)
    _need(state, "state", (B, D, N), torch.float32, dev)
    if idx is not None:
        k = idx.shape[1]
        _need(idx, "idx", (B, k), torch.int32, dev)
        _need(gate, "gate", (B, k), torch.float32, dev)
    else:
        if Wr is None or k is None:
            raise ValueError("step needs Wr and k, or idx and gate")
        _need(Wr, "Wr", (D, E), torch.float32, dev)
    if y is None:
        y = torch.empty((B, D), dtype=y_dtype or x.dtype, device=dev)
    _need(y, "y", (B, D), None, dev)
    if idx_out is not None:
        _need(idx_out, "idx_out", (B, k), torch.int32, dev)
    if gate_out is not None:
        _need(gate_out, "gate_out", (B, k), torch.float32, dev)
    a = StepArgs()
    a.B, a.D, a.N, a.E, a.k = B, D, N, E, k
    a.in_dtype, a.y_dtype = _dt(x), _dt(y)
    a.x, a.dt_raw, a.Bm, a.Cm = _ptr(x), _ptr(dt_raw), _ptr(Bm), _ptr(Cm)
    a.Wr, a.idx, a.gate = _ptr(Wr), _ptr(idx), _ptr(gate)
    a.idx_out, a.gate_out = _ptr(idx_out), _ptr(gate_out)
    a.A, a.dt_bias, a.Dskip, a.state, a.y = _ptr(A), _ptr(dt_bias), _ptr(Dskip), _ptr(state), \
        _ptr(y)
    a.a_form = A_SCALAR if scalar_a else A_DIAGONAL
    a.disc = DISC_ZOH if zoh else DISC_EULER
    return a, y


def step(x, dt_raw, Bm, Cm, A, dt_bias, Dskip, state, Wr=None, k=None, idx=None, gate=None,
         y=None, idx_out=None, gate_out=None, y_dtype=None, stream=None, zoh=False):
    """One decode step (include/swimba.h: swimba_step).  x, dt_raw [B,D];
    Bm, Cm [B,16]; state [B,D,16] f32 updated in place.  Routing from Wr [D,E]
    with top-k, or forced idx/gate [B,k].  Returns y [B,D]."""
    a, y = _step_args(x, dt_raw, Bm, Cm, A, dt_bias, Dskip, state, Wr, k, idx, gate, y, idx_out,
                      gate_out, y_dtype, zoh)
    rc = load().swimba_step(ctypes.byref(a), _stream(stream))
    _check("swimba_step", rc)
    return y


class PreparedStep:
    """swimba_step marshalled once for fixed tensors (a decode loop that keeps
    its buffers calls the C ABI directly, without per-call checks)."""

    def __init__(self, x, dt_raw, Bm, Cm, A, dt_bias, Dskip, state, Wr=None, k=None, idx=None,
                 gate=None, y=None, idx_out=None, gate_out=None, y_dtype=None, stream=None,
                 zoh=False):
        self.args, self.y = _step_args(x, dt_raw, Bm, Cm, A, dt_bias, Dskip, state, Wr, k, idx,
                                       gate, y, idx_out, gate_out, y_dtype, zoh)
        self._keep = (x, dt_raw, Bm, Cm, A, dt_bias, Dskip, state, Wr, idx, gate, idx_out,
                      gate_out)
        self._ref = ctypes.byref(self.args)
        self._fn = load().swimba_step
        self.stream = _stream(stream)

    def __call__(self):
        rc = self._fn(self._ref, self.stream)
        if rc != OK:
            raise SwimbaError("swimba_step", rc)
        return self.y


def _fits(t, name, shape, dtype, dev):
    """_need for calls where latency counts: one expression when all is well."""
    if not (isinstance(t, torch.Tensor) and t.device == dev and t.shape == shape
            and (dtype is None or t.dtype == dtype) and t.is_contiguous()):
        _need(t, name, shape, dtype, dev)


def _current(dev):
    """The handle of `dev`'s current stream."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _new(t, name, shape, dtype, dev):
    """The caller's output buffer, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _fits(t, name, shape, dtype, dev)
    return t


def _workspace(given, need, dev):
    """The caller's workspace, or one of `need` bytes for this call: (tensor or None,
    address, bytes)."""
    if given is None:
        if need == 0:
            return None, None, 0
        given = torch.empty(need, dtype=torch.uint8, device=dev)
    elif not given.is_cuda or given.device != dev or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % dev)
    return given, given.data_ptr(), given.numel() * given.element_size()


def _placed(fn):
    """Runs `fn` on its first tensor's device and on the stream asked for: with
    stream=s everything `fn` allocates belongs to s (a caller that uses the
    results on another stream waits for s there and records them, as for any
    tensor made on a side stream)."""

    name = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        first = args[0] if args else kw.get(name)
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            raise ValueError("%s: %s must be a device tensor" % (fn.__name__, name))
        dev = first.device
        if stream is not None:
            if stream.device != dev:
                raise ValueError("stream is on %s, the tensors on %s" % (stream.device, dev))
            with torch.cuda.stream(stream):
                return fn(*args, **kw)
        if dev.index != torch.cuda.current_device():
            with torch.cuda.device(dev):
                return fn(*args, **kw)
        return fn(*args, **kw)

    return call


# ---- tokens by expert ----


@_placed
def sort_tokens(idx, E, order=None, pos=None, offsets=None, workspace=None):
    """Slots sorted by expert (include/swimba.h: swimba_sort_tokens).  idx
    [..., k] int32, values outside [0, E) without an expert.  Returns (order
    [T*k], pos like idx, offsets [E+1]), int32."""
    _need(idx, "idx", None, torch.int32)
    if idx.dim() < 1 or idx.shape[-1] < 1:
        raise ValueError("idx must be [..., k]")
    dev, k = idx.device, idx.shape[-1]
    T = idx.numel() // k
    order = _new(order, "order", (T * k,), torch.int32, dev)
    pos = _new(pos, "pos", tuple(idx.shape), torch.int32, dev)
    offsets = _new(offsets, "offsets", (E + 1,), torch.int32, dev)
    lib = load()
    ws, wp, wn = _workspace(workspace, lib.swimba_sort_tokens_workspace_size(T, E, k), dev)
    rc = lib.swimba_sort_tokens(_ptr(idx), T, E, k, _ptr(order), _ptr(pos), _ptr(offsets), wp, wn,
                                _current(dev))
    _check("swimba_sort_tokens", rc)
    return order, pos, offsets


def _pos_shape(pos, dev):
    if not isinstance(pos, torch.Tensor) or pos.dim() < 1 or pos.shape[-1] < 1:
        raise ValueError("pos must be a tensor [..., k]")
    shape = pos.shape
    _fits(pos, "pos", shape, torch.int32, dev)
    k = shape[-1]
    return tuple(shape[:-1]), pos.numel() // k, k


@_placed
def dispatch_tokens(x, pos, rows=None):
    """rows[pos[t, j]] = x[t] (include/swimba.h: swimba_dispatch_tokens).  x
    [..., D], pos [..., k] from sort_tokens; returns rows [T*k, D].  Rows that no
    slot has are left as they were (unwritten memory where `rows` is not given)."""
    dev = x.device
    lead, T, k = _pos_shape(pos, dev)
    D = x.shape[-1] if x.dim() else 0
    _fits(x, "x", lead + (D,), None, dev)
    rows = _new(rows, "rows", (T * k, D), x.dtype, dev)
    rc = load().swimba_dispatch_tokens(_ptr(x), _dt(x), _ptr(pos), T, D, k, _ptr(rows),
                                       _current(dev))
    _check("swimba_dispatch_tokens", rc)
    return rows


@_placed
def combine_tokens(rows, pos, gate=None, y=None, y_dtype=None):
    """y[t] = sum_j gate[t, j] rows[pos[t, j]] (include/swimba.h:
    swimba_combine_tokens).  rows [T*k, D], pos and gate [..., k]; gate None: ones.
    Returns y [..., D]."""
    dev = rows.device
    lead, T, k = _pos_shape(pos, dev)
    D = rows.shape[-1] if rows.dim() else 0
    _fits(rows, "rows", (T * k, D), None, dev)
    if gate is not None:
        _fits(gate, "gate", lead + (k,), torch.float32, dev)
    if y is None:
        y = torch.empty(lead + (D,), dtype=y_dtype or rows.dtype, device=dev)
    else:
        _fits(y, "y", lead + (D,), None, dev)
    rc = load().swimba_combine_tokens(_ptr(rows), _dt(rows), _ptr(pos), _ptr(gate), T, D, k,
                                      _ptr(y), _dt(y), _current(dev))
    _check("swimba_combine_tokens", rc)
    return y


@_placed
def dispatch_tokens_backward(drows, pos, dx=None, grad_dtype=None):
    """The gradient of dispatch_tokens: the sum of a token's rows' gradients
    (combine_tokens without gates).  Returns dx [..., D], by default of drows'
    dtype."""
    return combine_tokens(drows, pos, None, y=dx, y_dtype=grad_dtype)


@_placed
def combine_tokens_backward(rows, pos, gate, dy, drows=None, dgate=None, grad_dtype=None):
    """Gradients of combine_tokens (include/swimba.h:
    swimba_combine_tokens_backward).  Returns (drows [T*k, D], by default of rows'
    dtype, and dgate [..., k] f32).  Rows of drows that no slot has are left as
    they were (unwritten memory where it is not given)."""
    dev = rows.device
    lead, T, k = _pos_shape(pos, dev)
    D = rows.shape[-1] if rows.dim() else 0
    _fits(rows, "rows", (T * k, D), None, dev)
    _fits(gate, "gate", lead + (k,), torch.float32, dev)
    _fits(dy, "dy", lead + (D,), None, dev)
    if drows is None:
        drows = torch.empty((T * k, D), dtype=grad_dtype or rows.dtype, device=dev)
    _fits(drows, "drows", (T * k, D), None, dev)
    dgate = _new(dgate, "dgate", lead + (k,), torch.float32, dev)
    rc = load().swimba_combine_tokens_backward(
        _ptr(rows), _dt(rows), _ptr(pos), _ptr(gate), _ptr(dy), _dt(dy), T, D, k, _ptr(drows),
        _dt(drows), _ptr(dgate), _current(dev))
    _check("swimba_combine_tokens_backward", rc)
    return drows, dgate


@_placed
def route_backward(x, Wr, idx, gate, dgate, dx=None, dWr=None, grad_dtype=torch.float32,
                   workspace=None):
    """Gradients of route's gates (include/swimba.h: swimba_route_backward) for
    dL/dgate = dgate [..., k].  Returns (dx [..., D] of grad_dtype, dWr [D, E] f32)."""
    _need(x, "x")
    dev, D = x.device, x.shape[-1]
    E = Wr.shape[1] if Wr.dim() == 2 else -1
    _need(Wr, "Wr", (D, E), torch.float32, dev)
    lead = tuple(x.shape[:-1])
    k = idx.shape[-1] if idx.dim() else 0
    _need(idx, "idx", lead + (k,), torch.int32, dev)
    _need(gate, "gate", lead + (k,), torch.float32, dev)
    _need(dgate, "dgate", lead + (k,), torch.float32, dev)
    T = x.numel() // D if D else 0
    if dx is None:
        dx = torch.empty(x.shape, dtype=grad_dtype, device=dev)
    _need(dx, "dx", tuple(x.shape), None, dev)
    dWr = _new(dWr, "dWr", (D, E), torch.float32, dev)
    lib = load()
    need = lib.swimba_route_backward_workspace_size(T, D, E)
    ws, wp, wn = _workspace(workspace, need, dev)
    rc = lib.swimba_route_backward(_ptr(x), _dt(x), _ptr(Wr), _ptr(idx), _ptr(gate), _ptr(dgate),
                                   T, D, E, k, _ptr(dx), _dt(dx), _ptr(dWr), wp, wn,
                                   _current(dev))
    _check("swimba_route_backward", rc)
    return dx, dWr


# ---- linear attention with a decay per head ----

DECAY_HEAD, DECAY_TOKEN = 0, 1  # log_decay [H], or one per token and head


def _linear_attention_args(q, k, v, log_decay, h0, y, h_final, need_y=True):
    _need(v, "v")
    if v.dim() != 4:
        raise ValueError("v must be [B, L, H, P]")
    B, L, H, P = v.shape
    dev = v.device
    _need(q, "q", None, v.dtype, dev)
    if q.dim() != 4:
        raise ValueError("q must be [B, L, G, N]")
    G, N = q.shape[2:]
    _need(q, "q", (B, L, G, N))
    _fits(k, "k", (B, L, G, N), v.dtype, dev)
    a = LinearAttentionArgs()
    a.decay_form = DECAY_HEAD if log_decay.dim() == 1 else DECAY_TOKEN
    _need(log_decay, "log_decay", (H,) if a.decay_form == DECAY_HEAD else (B, L, H),
          torch.float32, dev)
    if h0 is not None:
        _fits(h0, "h0", (B, H, N, P), torch.float32, dev)
    if need_y:
        _fits(y, "y", (B, L, H, P), None, dev)
    if h_final is not None:
        _fits(h_final, "h_final", (B, H, N, P), torch.float32, dev)
    a.B, a.L, a.H, a.G, a.N, a.P = B, L, H, G, N, P
    a.in_dtype = _dt(v)
    a.y_dtype = _dt(y) if y is not None else a.in_dtype
    a.q, a.k, a.v, a.log_decay, a.h0 = _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(h0)
    a.y, a.h_final = _ptr(y), _ptr(h_final)
    return a


@_placed
def linear_attention(q, k, v, log_decay, h0=None, y=None, h_final=None, y_dtype=None,
                     want_state=True, workspace=None):
    """Linear attention with a decay per head (include/swimba.h:
    swimba_linear_attention).  q, k [B,L,G,N], v [B,L,H,P] (f32 or bf16, H a multiple
    of G); log_decay [H] or [B,L,H] f32; h0 [B,H,N,P] f32.  Returns (y [B,L,H,P],
    h_final [B,H,N,P] f32 or None)."""
    if not (isinstance(v, torch.Tensor) and v.dim() == 4 and q.dim() == 4):
        raise ValueError("q must be [B, L, G, N] and v [B, L, H, P]")
    if y is None:
        y = torch.empty(v.shape, dtype=y_dtype or v.dtype, device=v.device)
    if h_final is None and want_state:
        h_final = torch.empty((v.shape[0], v.shape[2], q.shape[-1], v.shape[3]),
                              dtype=torch.float32, device=v.device)
    a = _linear_attention_args(q, k, v, log_decay, h0, y, h_final)
    lib, ref = load(), ctypes.byref(a)
    need = lib.swimba_linear_attention_workspace_size(ref) if workspace is None else 0
    ws, wp, wn = _workspace(workspace, need, v.device)
    _check("swimba_linear_attention", lib.swimba_linear_attention(ref, wp, wn, _current(v.device)))
    return y, h_final


def linear_attention_workspace_bytes(q, k, v, log_decay):
    """Workspace bytes linear_attention needs for these shapes."""
    a = _linear_attention_args(q, k, v, log_decay, None, None, None, need_y=False)
    with torch.cuda.device(v.device):
        return int(load().swimba_linear_attention_workspace_size(ctypes.byref(a)))


@_placed
def linear_attention_backward(q, k, v, log_decay, dy, h0=None, dh_final=None, want_dh0=True,
                              grad_dtype=torch.float32, out=None, workspace=None):
    """Gradients of linear_attention (include/swimba.h:
    swimba_linear_attention_backward) for dL/dy = dy (of v's dtype) and
    dL/dh_final.  Returns a dict: dq, dk [B,L,G,N], dv [B,L,H,P] of grad_dtype;
    dlog_decay like log_decay and dh0 [B,H,N,P] (when want_dh0), f32."""
    a = _linear_attention_args(q, k, v, log_decay, h0, None, None, need_y=False)
    dev = v.device
    _need(dy, "dy", tuple(v.shape), v.dtype, dev)
    state = (a.B, a.H, a.N, a.P)
    if dh_final is not None:
        _need(dh_final, "dh_final", state, torch.float32, dev)
    out = dict(out or {})
    shapes = {"dq": q.shape, "dk": k.shape, "dv": v.shape, "dlog_decay": log_decay.shape}
    if want_dh0:
        shapes["dh0"] = state
    res = {}
    for name, shape in shapes.items():
        dt = grad_dtype if name in ("dq", "dk", "dv") else torch.float32
        res[name] = _new(out.get(name), name, tuple(shape), dt, dev)
    g = LinearAttentionGradArgs()
    g.fwd = a
    g.dy, g.dh_final, g.grad_dtype = _ptr(dy), _ptr(dh_final), _dt(res["dq"])
    for name in res:
        setattr(g, name, _ptr(res[name]))
    lib, ref = load(), ctypes.byref(g)
    need = lib.swimba_linear_attention_backward_workspace_size(ref) if workspace is None else 0
    ws, wp, wn = _workspace(workspace, need, dev)
    _check("swimba_linear_attention_backward",
           lib.swimba_linear_attention_backward(ref, wp, wn, _current(dev)))
    return res


def _linear_attention_step_args(q, k, v, log_decay, state, state_out, y, y_dtype):
    _need(v, "v")
    if v.dim() != 3:
        raise ValueError("v must be [B, H, P]")
    B, H, P = v.shape
    dev = v.device
    _need(q, "q", None, v.dtype, dev)
    if q.dim() != 3:
        raise ValueError("q must be [B, G, N]")
    G, N = q.shape[1:]
    _need(q, "q", (B, G, N))
    _fits(k, "k", (B, G, N), v.dtype, dev)
    form = DECAY_HEAD if log_decay.dim() == 1 else DECAY_TOKEN
    _need(log_decay, "log_decay", (H,) if form == DECAY_HEAD else (B, H), torch.float32, dev)
    _fits(state, "state", (B, H, N, P), torch.float32, dev)
    if state_out is not None:
        _fits(state_out, "state_out", (B, H, N, P), torch.float32, dev)
    if y is None:
        y = torch.empty((B, H, P), dtype=y_dtype or v.dtype, device=dev)
    _fits(y, "y", (B, H, P), None, dev)
    a = LinearAttentionStepArgs()
    a.B, a.H, a.G, a.N, a.P = B, H, G, N, P
    a.in_dtype, a.y_dtype, a.decay_form = _dt(v), _dt(y), form
    a.q, a.k, a.v, a.log_decay = _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay)
    a.state, a.state_out, a.y = _ptr(state), _ptr(state_out), _ptr(y)
    return a, y


@_placed
def linear_attention_step(q, k, v, log_decay, state, state_out=None, y=None, y_dtype=None):
    """One decode step of linear_attention (include/swimba.h:
    swimba_linear_attention_step).  q, k [B,G,N], v [B,H,P]; log_decay [H] or [B,H]
    f32; state [B,H,N,P] f32, updated in place unless state_out is given.
    Returns y [B,H,P]."""
    a, y = _linear_attention_step_args(q, k, v, log_decay, state, state_out, y, y_dtype)
    _check("swimba_linear_attention_step",
           load().swimba_linear_attention_step(ctypes.byref(a), _current(v.device)))
    return y


class PreparedLinearAttentionStep:
    """swimba_linear_attention_step marshalled once for fixed tensors (see
    PreparedStep).  Each call goes to the device's current stream (a capturing one
    records it), or to `stream` if that is given."""

    _name = "swimba_linear_attention_step"

    def __init__(self, q, k, v, log_decay, state, state_out=None, y=None, y_dtype=None,
                 stream=None):
        self.args, self.y = _linear_attention_step_args(q, k, v, log_decay, state, state_out, y,
                                                        y_dtype)
        self._prepare((q, k, v, log_decay, state, state_out), v.device, stream)

    def _prepare(self, keep, dev, stream):
        self._keep = keep
        self._ref = ctypes.byref(self.args)
        self._fn = getattr(load(), self._name)
        self._dev = dev.index
        if stream is not None and stream.device != dev:
            raise ValueError("stream is on %s, the tensors on %s" % (stream.device, dev))
        self.stream = None if stream is None else stream.cuda_stream

    def __call__(self):
        stream = self.stream
        if stream is None:
            stream = torch._C._cuda_getCurrentRawStream(self._dev)
        if self._dev != torch.cuda.current_device():
            with torch.cuda.device(self._dev):
                rc = self._fn(self._ref, stream)
        else:
            rc = self._fn(self._ref, stream)
        if rc != OK:
            raise SwimbaError(self._name, rc)
        return self.y


# ---- the gated delta rule ----


def _delta_rule_args(q, k, v, log_decay, beta, h0, y, h_final, need_y=True):
    la = _linear_attention_args(q, k, v, log_decay, h0, y, h_final, need_y)
    _fits(beta, "beta", (la.B, la.L, la.H), torch.float32, v.device)
    a = DeltaRuleArgs()
    for name, _ in LinearAttentionArgs._fields_:
        setattr(a, name, getattr(la, name))
    a.beta = _ptr(beta)
    return a


@_placed
def delta_rule(q, k, v, log_decay, beta, h0=None, y=None, h_final=None, y_dtype=None,
               want_state=True, workspace=None):
    """The gated delta rule (include/swimba.h: swimba_delta_rule).  q, k [B,L,G,N], v
    [B,L,H,P] (f32 or bf16, H a multiple of G); log_decay [H] or [B,L,H] f32; beta
    [B,L,H] f32; h0 [B,H,N,P] f32.  Returns (y [B,L,H,P], h_final [B,H,N,P] f32 or
    None)."""
    if not (isinstance(v, torch.Tensor) and v.dim() == 4 and q.dim() == 4):
        raise ValueError("q must be [B, L, G, N] and v [B, L, H, P]")
    if y is None:
        y = torch.empty(v.shape, dtype=y_dtype or v.dtype, device=v.device)
    if h_final is None and want_state:
        h_final = torch.empty((v.shape[0], v.shape[2], q.shape[-1], v.shape[3]),
                              dtype=torch.float32, device=v.device)
    a = _delta_rule_args(q, k, v, log_decay, beta, h0, y, h_final)
    lib, ref = load(), ctypes.byref(a)
    need = lib.swimba_delta_rule_workspace_size(ref) if workspace is None else 0
    ws, wp, wn = _workspace(workspace, need, v.device)
    _check("swimba_delta_rule", lib.swimba_delta_rule(ref, wp, wn, _current(v.device)))
    return y, h_final


def delta_rule_workspace_bytes(q, k, v, log_decay, beta):
    """Workspace bytes delta_rule needs for these shapes."""
    a = _delta_rule_args(q, k, v, log_decay, beta, None, None, None, need_y=False)
    with torch.cuda.device(v.device):
        return int(load().swimba_delta_rule_workspace_size(ctypes.byref(a)))


def delta_rule_backward_workspace_bytes(q, k, v, log_decay, beta):
    """Workspace bytes delta_rule_backward needs for these shapes."""
    g = DeltaRuleGradArgs()
    g.fwd = _delta_rule_args(q, k, v, log_decay, beta, None, None, None, need_y=False)
    with torch.cuda.device(v.device):
        return int(load().swimba_delta_rule_backward_workspace_size(ctypes.byref(g)))


@_placed
def delta_rule_backward(q, k, v, log_decay, beta, dy, h0=None, dh_final=None, want_dh0=True,
                        grad_dtype=torch.float32, out=None, workspace=None):
    """Gradients of delta_rule (include/swimba.h: swimba_delta_rule_backward) for dL/dy
    = dy (of v's dtype) and dL/dh_final.  Returns a dict: dq, dk [B,L,G,N], dv
    [B,L,H,P] of grad_dtype; dlog_decay like log_decay, dbeta [B,L,H] and dh0
    [B,H,N,P] (when want_dh0), f32."""
    a = _delta_rule_args(q, k, v, log_decay, beta, h0, None, None, need_y=False)
    dev = v.device
    _need(dy, "dy", tuple(v.shape), v.dtype, dev)
    state = (a.B, a.H, a.N, a.P)
    if dh_final is not None:
        _need(dh_final, "dh_final", state, torch.float32, dev)
    out = dict(out or {})
    shapes = {"dq": q.shape, "dk": k.shape, "dv": v.shape, "dlog_decay": log_decay.shape,
              "dbeta": beta.shape}
    if want_dh0:
        shapes["dh0"] = state
    res = {}
    for name, shape in shapes.items():
        dt = grad_dtype if name in ("dq", "dk", "dv") else torch.float32
        res[name] = _new(out.get(name), name, tuple(shape), dt, dev)
    g = DeltaRuleGradArgs()
    g.fwd = a
    g.dy, g.dh_final, g.grad_dtype = _ptr(dy), _ptr(dh_final), _dt(res["dq"])
    for name in res:
        setattr(g, name, _ptr(res[name]))
    lib, ref = load(), ctypes.byref(g)
    need = lib.swimba_delta_rule_backward_workspace_size(ref) if workspace is None else 0
    ws, wp, wn = _workspace(workspace, need, dev)
    _check("swimba_delta_rule_backward",
           lib.swimba_delta_rule_backward(ref, wp, wn, _current(dev)))
    return res


def _delta_rule_step_args(q, k, v, log_decay, beta, state, state_out, y, y_dtype):
    la, y = _linear_attention_step_args(q, k, v, log_decay, state, state_out, y, y_dtype)
    _fits(beta, "beta", (la.B, la.H), torch.float32, v.device)
    a = DeltaRuleStepArgs()
    for name, _ in LinearAttentionStepArgs._fields_:
        setattr(a, name, getattr(la, name))
    a.beta = _ptr(beta)
    return a, y


@_placed
def delta_rule_step(q, k, v, log_decay, beta, state, state_out=None, y=None, y_dtype=None):
    """One decode step of delta_rule (include/swimba.h: swimba_delta_rule_step).  q, k
    [B,G,N], v [B,H,P]; log_decay [H] or [B,H] f32; beta [B,H] f32; state [B,H,N,P]
    f32, updated in place unless state_out is given.  Returns y [B,H,P]."""
    a, y = _delta_rule_step_args(q, k, v, log_decay, beta, state, state_out, y, y_dtype)
    _check("swimba_delta_rule_step",
           load().swimba_delta_rule_step(ctypes.byref(a), _current(v.device)))
    return y


class PreparedDeltaRuleStep(PreparedLinearAttentionStep):
    """swimba_delta_rule_step marshalled once for fixed tensors (see
    PreparedLinearAttentionStep)."""

    _name = "swimba_delta_rule_step"

    def __init__(self, q, k, v, log_decay, beta, state, state_out=None, y=None, y_dtype=None,
                 stream=None):
        self.args, self.y = _delta_rule_step_args(q, k, v, log_decay, beta, state, state_out, y,
                                                  y_dtype)
        self._prepare((q, k, v, log_decay, beta, state, state_out), v.device, stream)


# ---- norms of queries and keys, with their rotation ----

NORM = {"rms": 0, "l2": 1}
PAIRS = {"halves": 0, "neighbours": 1}


def _token_rows(t, name):
    """(tokens, heads, N, stride of a token) of a tensor [..., heads, N] whose tokens are
    equally far apart, each dense."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if t.dim() < 2:
        raise ValueError("%s must be [..., heads, N]" % name)
    heads, N = t.shape[-2:]
    if t.is_contiguous() and heads * N:
        return t.numel() // (heads * N), heads, N, heads * N
    lead, strides = t.shape[:-2], t.stride()
    T = 1
    for n in lead:
        T *= n
    if T * heads * N == 0:
        return T, heads, N, heads * N
    if (N > 1 and strides[-1] != 1) or (heads > 1 and strides[-2] != N):
        raise ValueError("%s: the heads of a token must be contiguous" % name)
    stride = far = None
    for n, step in zip(reversed(lead), reversed(strides[:-2])):
        if n == 1:
            continue
        if stride is None:
            stride, far = step, step * n
        elif step == far:
            far *= n
        else:
            raise ValueError("%s: tokens must be equally far apart" % name)
    stride = heads * N if stride is None else stride
    if stride < heads * N:
        raise ValueError("%s: tokens overlap" % name)
    return T, heads, N, stride


def _norm_rotate_args(q, k, wq, wk, positions, rates, norm, pairs, eps, q_scale):
    a = NormRotateArgs()
    a.T, a.Hq, a.N, a.q_stride = _token_rows(q, "q")
    T, a.Hk, N, a.k_stride = _token_rows(k, "k")
    dev, lead = q.device, q.shape[:-2]
    if k.shape[:-2] != lead or N != a.N or k.dtype != q.dtype or k.device != dev:
        raise ValueError("k must have the tokens, the head size, the dtype and the device of q")
    for name, t in (("wq", wq), ("wk", wk)):
        if t is not None:
            _fits(t, name, (N,), torch.float32, dev)
    if (positions is None) != (rates is None):
        raise ValueError("positions and rates belong together")
    if positions is not None:
        _need(rates, "rates", None, torch.float32, dev)
        if rates.dim() != 1:
            raise ValueError("rates must be [R / 2]")
        _fits(positions, "positions", lead, torch.int32, dev)
        a.R = 2 * rates.numel()
    if norm not in NORM or pairs not in PAIRS:
        raise ValueError("norm is one of %s, pairs of %s" % (sorted(NORM), sorted(PAIRS)))
    a.in_dtype = a.out_dtype = _dt(q)
    a.norm, a.pairs, a.eps, a.q_scale = NORM[norm], PAIRS[pairs], eps, q_scale
    a.q, a.k, a.wq, a.wk = _ptr(q), _ptr(k), _ptr(wq), _ptr(wk)
    a.positions, a.rates = _ptr(positions), _ptr(rates)
    return a


@_placed
def norm_rotate(q, k, wq=None, wk=None, positions=None, rates=None, norm="rms", pairs="halves",
                eps=1e-6, q_scale=1.0, q_out=None, k_out=None, out_dtype=None):
    """Norms of queries and keys for each head with the rotation of their positions
    (include/swimba.h: swimba_norm_rotate).  q [..., Hq, N], k [..., Hk, N] (f32 or
    bf16; tokens may lie apart, as parts of one projection's rows); wq, wk [N] f32;
    positions [...] int32 with rates [R/2] f32, or neither (no rotation).  norm:
    "rms" or "l2"; pairs: "halves" or "neighbours".  Returns (q_out, k_out), dense."""
    a = _norm_rotate_args(q, k, wq, wk, positions, rates, norm, pairs, eps, q_scale)
    dt = out_dtype or (q_out.dtype if q_out is not None else q.dtype)
    q_out = _new(q_out, "q_out", q.shape, dt, q.device)
    k_out = _new(k_out, "k_out", k.shape, dt, q.device)
    a.out_dtype, a.q_out, a.k_out = _dt(q_out), _ptr(q_out), _ptr(k_out)
    _check("swimba_norm_rotate", load().swimba_norm_rotate(ctypes.byref(a), _current(q.device)))
    return q_out, k_out


def norm_rotate_backward_workspace_bytes(q, k, wq=None, wk=None, positions=None, rates=None):
    """Workspace bytes norm_rotate_backward needs for these shapes and weights."""
    g = NormRotateGradArgs()
    g.fwd = _norm_rotate_args(q, k, wq, wk, positions, rates, "rms", "halves", 1e-6, 1.0)
    g.dwq, g.dwk = _ptr(wq), _ptr(wk)  # (only whether they are there)
    with torch.cuda.device(q.device):
        return int(load().swimba_norm_rotate_backward_workspace_size(ctypes.byref(g)))


@_placed
def norm_rotate_backward(q, k, dq_out, dk_out, wq=None, wk=None, positions=None, rates=None,
                         norm="rms", pairs="halves", eps=1e-6, q_scale=1.0,
                         grad_dtype=torch.float32, out=None, workspace=None):
    """Gradients of norm_rotate (include/swimba.h: swimba_norm_rotate_backward) for dL/dq_out
    and dL/dk_out (dense, of q's dtype).  Returns a dict: dq, dk like q and k, of
    grad_dtype; dwq and dwk [N] f32, None where that weight is not given."""
    a = _norm_rotate_args(q, k, wq, wk, positions, rates, norm, pairs, eps, q_scale)
    dev = q.device
    _need(dq_out, "dq_out", tuple(q.shape), q.dtype, dev)
    _need(dk_out, "dk_out", tuple(k.shape), k.dtype, dev)
    out = dict(out or {})
    res = {"dq": _new(out.get("dq"), "dq", tuple(q.shape), grad_dtype, dev),
           "dk": _new(out.get("dk"), "dk", tuple(k.shape), grad_dtype, dev)}
    for name, w in (("dwq", wq), ("dwk", wk)):
        res[name] = None if w is None else _new(out.get(name), name, (a.N,), torch.float32, dev)
    g = NormRotateGradArgs()
    g.fwd = a
    g.dq_out, g.dk_out, g.grad_dtype = _ptr(dq_out), _ptr(dk_out), _dt(res["dq"])
    for name in res:
        setattr(g, name, _ptr(res[name]))
    lib, ref = load(), ctypes.byref(g)
    need = lib.swimba_norm_rotate_backward_workspace_size(ref) if workspace is None else 0
    ws, wp, wn = _workspace(workspace, need, dev)
    _check("swimba_norm_rotate_backward",
           lib.swimba_norm_rotate_backward(ref, wp, wn, _current(dev)))
    return res
