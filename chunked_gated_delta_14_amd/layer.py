"""Binding of the operators around the recurrence (see include/gdr.h): the short
causal convolution, the decay gate, the single-token recurrence and the norm with
gate and residual.

Like the rest of the binding this only marshals arguments.  A problem object holds
the input tensors of a call and its C struct; it is built (and its tensors
checked) once and used for any number of calls on those tensors, so the calls of
a training step or a serving loop cost one C call each.  A tensor that does not
fit raises GdrError with GDR_ERR_INVALID_ARG before anything is enqueued.  Calls
run on the device of the problem's tensors, on `stream` or that device's current
stream; keeping a tensor that was allocated on another stream is the caller's part
(`Tensor.record_stream`), as in the rest of the binding.
"""
from __future__ import annotations

import ctypes

import numpy as np

from . import GDR_GDN, GDR_KDA, GdrError, _check, lib, plan_chunks

GDR_BF16, GDR_F32 = 0, 1
GDR_ACT_NONE, GDR_ACT_SILU, GDR_ACT_SIGMOID = 0, 1, 2
GDR_GATE_SOFTPLUS, GDR_GATE_SIGMOID = 0, 1
GDR_RES_NONE, GDR_RES_BEFORE, GDR_RES_AFTER = 0, 1, 2

_i32, _i64, _u32, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_float, ctypes.c_void_p


class _CConv(ctypes.Structure):
    _fields_ = [("T", _i32), ("N", _i32), ("C", _i32), ("W", _i32), ("dtype", _i32), ("w_dtype", _i32),
                ("activation", _i32), ("n_chunks", _i32), ("x_stride", _i64), ("x", _vp), ("weight", _vp), ("bias", _vp),
                ("s0", _vp), ("chunk_table", _vp)]


class _CGate(ctypes.Structure):
    _fields_ = [("T", _i32), ("H", _i32), ("D", _i32), ("dtype", _i32), ("kind", _i32), ("floor", _f32),
                ("x_stride", _i64), ("x", _vp), ("a_log", _vp), ("bias", _vp)]


class _CStep(ctypes.Structure):
    _fields_ = [("T", _i32), ("N", _i32), ("H_qk", _i32), ("H_v", _i32), ("K", _i32), ("V", _i32), ("n_slots", _i32),
                ("input_flags", _u32), ("scale", _f32), ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64),
                ("q", _vp), ("k", _vp), ("v", _vp), ("g", _vp), ("beta", _vp), ("cu_seqlens", _vp), ("slots", _vp),
                ("state", _vp)]


class _CNorm(ctypes.Structure):
    _fields_ = [("T", _i32), ("H", _i32), ("D", _i32), ("dtype", _i32), ("res_dtype", _i32), ("w_dtype", _i32),
                ("activation", _i32), ("placement", _i32), ("scale", _f32), ("eps", _f32), ("x_stride", _i64),
                ("gate_stride", _i64), ("x", _vp), ("weight", _vp), ("gate", _vp), ("residual", _vp), ("s", _vp)]


def declare(L) -> None:
    """Argument types of the layer entry points on the loaded library."""
    P = ctypes.POINTER
    for name, args in (
        ("gdr_conv_fwd", [P(_CConv), _vp, _i64, _vp, _vp]),
        ("gdr_conv_bwd", [P(_CConv), _vp, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _vp]),
        ("gdr_conv_step", [P(_CConv), _vp, _i64, _vp, _vp, _i32, _vp]),
        ("gdr_gate_fwd", [P(_CGate), _vp, _vp]),
        ("gdr_gate_bwd", [P(_CGate), _vp, _vp, _i64, _vp, _vp, _vp, _i64, _vp]),
        ("gdr_kda_step", [P(_CStep), _vp, _vp]),
        ("gdr_gdn_step", [P(_CStep), _vp, _vp]),
        ("gdr_norm_fwd", [P(_CNorm), _vp, _vp]),
        ("gdr_norm_bwd", [P(_CNorm), _vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp]),
    ):
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, _i32
    for name, n in (("gdr_conv_workspace_bytes", 4), ("gdr_gate_workspace_bytes", 4), ("gdr_norm_workspace_bytes", 3)):
        fn = getattr(L, name)
        fn.argtypes, fn.restype = [_i32] * n, _i64


def _bad(detail: str):
    raise GdrError(1, detail)


def _sizes(*sizes):
    """The C structs and calls hold sizes with 32 bits, and ctypes would cut larger ones without a word."""
    for n in sizes:
        if not -(1 << 31) <= n < 1 << 31:
            _bad("a size of %d is past 32 bits" % n)


def _dtype_code(dtype, name):
    import torch

    if dtype == torch.bfloat16:
        return GDR_BF16
    if dtype == torch.float32:
        return GDR_F32
    _bad("%s must be bfloat16 or float32, not %s" % (name, dtype))


def _need(t, name, shape=None, dtype=None, device=None, contiguous=True):
    """Check one tensor argument of a call."""
    if t.shape == shape and t.dtype is dtype and t.device == device and (not contiguous or t.is_contiguous()):
        return t
    if dtype is not None and t.dtype is not dtype:
        _bad("%s must be %s, not %s" % (name, dtype, t.dtype))
    if shape is not None and t.shape != shape:
        _bad("%s must be of shape %s, not %s" % (name, shape, tuple(t.shape)))
    if device is not None and t.device != device:
        _bad("%s must be on %s, not %s" % (name, device, t.device))
    if contiguous and not t.is_contiguous():
        _bad("%s must be contiguous" % name)
    return t


def _rows(t, name, shape, dtype, device):
    """A tensor of token rows: everything inside a row contiguous, any row stride.  Returns the stride in elements."""
    if t.shape == shape and t.dtype is dtype and t.device == device and shape[0] > 1 and t.is_contiguous():
        return t.stride(0) or 1
    _need(t, name, shape, dtype, device, contiguous=False)
    inner = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != inner and t.numel():
            _bad("the rows of %s must be contiguous" % name)
        inner *= size
    if t.shape[0] < 2:
        return max(inner, 1)
    if t.stride(0) < inner:
        _bad("the rows of %s overlap" % name)
    return t.stride(0)


def _p(t):
    return None if t is None else t.data_ptr()


def _call(prob, stream, name, *args):
    """Call an entry point on the problem's device and on `stream` (None: that device's current stream)."""
    import torch

    dev = prob.device.index
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)  # what current_stream(dev).cuda_stream reads, without the object
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    fn = getattr(lib(), name)
    if torch.cuda.current_device() == dev:
        status = fn(prob.cstruct, *args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(prob.cstruct, *args, stream)
    if status:
        _check(status)


def _bytes(r) -> int:
    if r < 0:
        _check(-r)
    return int(r)


class _Base:
    def alloc_workspace(self):
        """A workspace of this problem's backward."""
        import torch

        return torch.empty(max(self.workspace_bytes(), 256), dtype=torch.uint8, device=self.device)

    def _device_of(self, t, name):
        if t.device.type != "cuda":
            _bad("%s must be on a GPU" % name)
        self.device = t.device

    def _workspace(self, ws):
        _need(ws, "workspace", device=self.device)
        return ws.data_ptr(), ws.numel() * ws.element_size()


class Plan:
    """A packed batch's chunk table on the device, shared by the convolutions of that batch.

    cu_seqlens: host sequence or tensor of N+1 ints."""

    def __init__(self, cu_seqlens, device="cuda"):
        import torch

        cu = np.asarray(cu_seqlens.cpu() if hasattr(cu_seqlens, "cpu") else cu_seqlens, dtype=np.int32)
        table, self.n_chunks = plan_chunks(cu)
        self.N, self.T = len(cu) - 1, int(cu[-1])
        self.table = torch.from_numpy(table.copy()).to(device)


class ConvProblem(_Base):
    """The short convolution over a packed batch.

    x: bf16 or fp32 [T, C], rows at any stride; weight: [C, W], bias: [C] or None (both bf16 or fp32);
    plan: the batch's Plan, or a Problem built from the same cu_seqlens; s0: [N, W-1, C] in x's dtype, or None."""

    def __init__(self, x, weight, plan, bias=None, s0=None, activation=GDR_ACT_SILU):
        self._device_of(x, "x")
        dev = self.device
        if x.dim() != 2 or weight.dim() != 2:
            _bad("x must be [T, C] and weight [C, W]")
        self.T, self.C, self.W, self.N = int(x.shape[0]), int(x.shape[1]), int(weight.shape[1]), plan.N
        _sizes(self.T, self.C, self.W)
        self.dtype, self.n_chunks = _dtype_code(x.dtype, "x"), plan.n_chunks
        if plan.T != self.T:
            _bad("the plan holds %d tokens, x %d" % (plan.T, self.T))
        stride = _rows(x, "x", None, None, dev)
        _need(weight, "weight", (self.C, self.W), None, dev)
        w_dtype = _dtype_code(weight.dtype, "weight")
        if bias is not None:
            _need(bias, "bias", (self.C,), weight.dtype, dev)
        if s0 is not None:
            _need(s0, "s0", (self.N, self.W - 1, self.C), x.dtype, dev)
        _need(plan.table, "the plan's table", None, None, dev)
        self.x, self.weight, self.bias, self.s0, self.plan = x, weight, bias, s0, plan
        self._c = _CConv(self.T, self.N, self.C, self.W, self.dtype, w_dtype, int(activation), self.n_chunks, stride, _p(x),
                         _p(weight), _p(bias), _p(s0), _p(plan.table))
        self.cstruct = ctypes.byref(self._c)

    def workspace_bytes(self) -> int:
        return conv_workspace_bytes(self.n_chunks, self.C, self.W, self.dtype)


def conv_workspace_bytes(n_chunks, C, W, dtype) -> int:
    _sizes(n_chunks, C, W)
    return _bytes(lib().gdr_conv_workspace_bytes(n_chunks, C, W, dtype))


def conv_fwd(prob, y, st=None, stream=None):
    """y: [T, C] in x's dtype, rows at any stride; st: [N, W-1, C] final rows, or None."""
    dt = prob.x.dtype
    stride = _rows(y, "y", (prob.T, prob.C), dt, prob.device)
    if st is not None:
        _need(st, "st", (prob.N, prob.W - 1, prob.C), dt, prob.device)
    _call(prob, stream, "gdr_conv_fwd", _p(y), stride, _p(st))


def conv_bwd(prob, dy, dst, dx, dw, dbias, ds0, workspace, stream=None):
    """dy, dx: [T, C] in x's dtype, rows at any stride; dst, ds0: [N, W-1, C] or None;
    dw: fp32 [C, W]; dbias: fp32 [C] or None."""
    import torch

    dt, dev = prob.x.dtype, prob.device
    dy_stride = _rows(dy, "dy", (prob.T, prob.C), dt, dev)
    dx_stride = _rows(dx, "dx", (prob.T, prob.C), dt, dev)
    for t, name in ((dst, "dst"), (ds0, "ds0")):
        if t is not None:
            _need(t, name, (prob.N, prob.W - 1, prob.C), dt, dev)
    _need(dw, "dw", (prob.C, prob.W), torch.float32, dev)
    if dbias is not None:
        _need(dbias, "dbias", (prob.C,), torch.float32, dev)
    ws, nbytes = prob._workspace(workspace)
    _call(prob, stream, "gdr_conv_bwd", _p(dy), dy_stride, _p(dst), _p(dx), dx_stride, _p(dw), _p(dbias), _p(ds0), ws, nbytes)


class ConvStep(_Base):
    """The short convolution for one token of each of N sequences.

    x: [N, C], rows at any stride; weight, bias: as ConvProblem; state: [n_slots, W-1, C] in x's dtype, updated in
    place; slots: int32 [N] on the device, the sequences' distinct slots (outside [0, n_slots): row skipped), or None."""

    def __init__(self, x, weight, state, slots=None, bias=None, activation=GDR_ACT_SILU):
        import torch

        self._device_of(x, "x")
        dev = self.device
        if x.dim() != 2 or weight.dim() != 2 or state.dim() != 3:
            _bad("x must be [N, C], weight [C, W] and state [n_slots, W-1, C]")
        self.N, self.C, self.W, self.n_slots = int(x.shape[0]), int(x.shape[1]), int(weight.shape[1]), int(state.shape[0])
        _sizes(self.N, self.C, self.W, self.n_slots)
        stride = _rows(x, "x", None, None, dev)
        _need(weight, "weight", (self.C, self.W), None, dev)
        if bias is not None:
            _need(bias, "bias", (self.C,), weight.dtype, dev)
        _need(state, "state", (self.n_slots, self.W - 1, self.C), x.dtype, dev)
        if slots is not None:
            _need(slots, "slots", (self.N,), torch.int32, dev)
        self.x, self.weight, self.bias, self.state, self.slots = x, weight, bias, state, slots
        self._c = _CConv(self.N, self.N, self.C, self.W, _dtype_code(x.dtype, "x"), _dtype_code(weight.dtype, "weight"), int(activation), 0,
                         stride, _p(x), _p(weight), _p(bias), None, None)
        self.cstruct = ctypes.byref(self._c)


def conv_step(prob, y, stream=None):
    """y: [N, C] in x's dtype, rows at any stride.  Updates prob.state."""
    stride = _rows(y, "y", (prob.N, prob.C), prob.x.dtype, prob.device)
    _call(prob, stream, "gdr_conv_step", _p(y), stride, _p(prob.state), _p(prob.slots), prob.n_slots)


class GateProblem(_Base):
    """The decay gate.  x: bf16 or fp32, [T, H] (D = 1) or [T, H * 128] or [T, H, 128] (D = 128), rows at any stride;
    a_log: fp32 [H]; bias: fp32 [H * D] values in any shape, or None; floor in [-8, 0)."""

    def __init__(self, x, a_log, bias=None, kind=GDR_GATE_SOFTPLUS, floor=-5.0):
        import torch

        self._device_of(x, "x")
        dev = self.device
        if a_log.dim() != 1 or x.dim() not in (2, 3):
            _bad("a_log must be [H] and x [T, H * D] or [T, H, D]")
        self.T, self.H = int(x.shape[0]), int(a_log.shape[0])
        width = int(x.shape[1]) * (int(x.shape[2]) if x.dim() == 3 else 1)
        if self.H < 1 or width % self.H or (x.dim() == 3 and x.shape[1] != self.H):
            _bad("x must be [T, H * D] or [T, H, D] with a_log's H")
        self.D = width // self.H
        _sizes(self.T, self.H, self.D)
        self.dtype = _dtype_code(x.dtype, "x")
        stride = _rows(x, "x", None, None, dev)
        _need(a_log, "a_log", None, torch.float32, dev)
        if bias is not None:
            _need(bias, "bias", None, torch.float32, dev)
            if bias.numel() != width:
                _bad("bias must hold H * D values")
        self.x, self.a_log, self.bias = x, a_log, bias
        self._c = _CGate(self.T, self.H, self.D, self.dtype, int(kind), float(floor), stride, _p(x), _p(a_log), _p(bias))
        self.cstruct = ctypes.byref(self._c)

    def workspace_bytes(self) -> int:
        return gate_workspace_bytes(self.T, self.H, self.D, self.dtype)


def gate_workspace_bytes(T, H, D, dtype) -> int:
    _sizes(T, H, D)
    return _bytes(lib().gdr_gate_workspace_bytes(T, H, D, dtype))


def _gate_values(t, name, prob):
    import torch

    _need(t, name, None, torch.float32, prob.device)
    if t.numel() != prob.T * prob.H * prob.D:
        _bad("%s must hold T * H * D values" % name)


def gate_fwd(prob, g, stream=None):
    """g: fp32, T * H * D values (the recurrence's [T, H, 128] or [T, H])."""
    _gate_values(g, "g", prob)
    _call(prob, stream, "gdr_gate_fwd", _p(g))


def gate_bwd(prob, dg, dx, da_log, dbias, workspace, stream=None):
    """dg: fp32, T * H * D values; dx: as x, rows at any stride; da_log: fp32 [H]; dbias: fp32, H * D values, or None."""
    import torch

    dev = prob.device
    _gate_values(dg, "dg", prob)
    stride = _rows(dx, "dx", tuple(prob.x.shape), prob.x.dtype, dev)
    _need(da_log, "da_log", (prob.H,), torch.float32, dev)
    if dbias is not None:
        _need(dbias, "dbias", None, torch.float32, dev)
        if dbias.numel() != prob.H * prob.D:
            _bad("dbias must hold H * D values")
    ws, nbytes = prob._workspace(workspace)
    _call(prob, stream, "gdr_gate_bwd", _p(dg), _p(dx), stride, _p(da_log), _p(dbias), ws, nbytes)


class StepProblem(_Base):
    """The recurrence for single tokens and short runs, on a pool of states updated in place.

    q, k: bf16 [T, H_qk, 128]; v: bf16 [T, H_v, 128] (rows at any stride); g, beta: as Problem; state: fp32
    [n_slots, H_v, 128, 128]; cu_seqlens: int32 [N+1] on the device, or None for one token per sequence; slots: int32
    [N] on the device, the sequences' distinct slots (outside [0, n_slots): sequence skipped), or None for slot n."""

    def __init__(self, variant, q, k, v, g, beta, state, cu_seqlens=None, slots=None, scale=None, input_flags=0):
        import torch

        self._device_of(q, "q")
        dev = self.device
        if variant not in (GDR_KDA, GDR_GDN):
            _bad("variant must be GDR_KDA or GDR_GDN")
        if q.dim() != 3 or v.dim() != 3 or state.dim() != 4:
            _bad("q and v must be [T, H, 128] and state [n_slots, H_v, 128, 128]")
        self.variant = variant
        self.T, self.H_qk, self.H_v, self.n_slots = int(q.shape[0]), int(q.shape[1]), int(v.shape[1]), int(state.shape[0])
        K, V = int(q.shape[2]), int(v.shape[2])
        _sizes(self.T, self.H_qk, self.H_v, self.n_slots, K, V)
        bf, f32 = torch.bfloat16, torch.float32
        qs = _rows(q, "q", None, bf, dev)
        ks = _rows(k, "k", tuple(q.shape), bf, dev)
        vs = _rows(v, "v", (self.T, self.H_v, V), bf, dev)
        _need(g, "g", (self.T, self.H_v) + ((K,) if variant == GDR_KDA else ()), f32, dev)
        _need(beta, "beta", (self.T, self.H_v), bf if variant == GDR_KDA else f32, dev)
        _need(state, "state", (self.n_slots, self.H_v, K, V), f32, dev)
        self.N = self.T if cu_seqlens is None else int(cu_seqlens.shape[0]) - 1
        if cu_seqlens is not None:
            _sizes(self.N)
            _need(cu_seqlens, "cu_seqlens", (self.N + 1,), torch.int32, dev)
        if slots is not None:
            _need(slots, "slots", (self.N,), torch.int32, dev)
        self.scale = float(K ** -0.5 if scale is None else scale)
        self.q, self.k, self.v, self.g, self.beta, self.state = q, k, v, g, beta, state
        self.cu_seqlens, self.slots = cu_seqlens, slots
        self._c = _CStep(self.T, self.N, self.H_qk, self.H_v, K, V, self.n_slots, int(input_flags), self.scale, qs, ks, vs,
                         _p(q), _p(k), _p(v), _p(g), _p(beta), _p(cu_seqlens), _p(slots), _p(state))
        self.cstruct = ctypes.byref(self._c)


def _step(name, variant, prob, o, stream):
    import torch

    if prob.variant != variant:
        _bad("the problem is of the other variant")
    _need(o, "o", tuple(prob.v.shape), torch.bfloat16, prob.device)
    _call(prob, stream, name, _p(o))


def kda_step(prob, o, stream=None):
    """o: bf16 [T, H_v, 128].  Updates prob.state."""
    _step("gdr_kda_step", GDR_KDA, prob, o, stream)


def gdn_step(prob, o, stream=None):
    """o: bf16 [T, H_v, 128].  Updates prob.state."""
    _step("gdr_gdn_step", GDR_GDN, prob, o, stream)


class NormProblem(_Base):
    """RMS norm with gate and residual.

    x: bf16 or fp32 [T, D] or [T, H, D], rows at any stride (None for a GDR_RES_BEFORE backward, which reads s);
    weight: [D] (bf16 or fp32) or None; gate: as x, or None; residual: x's shape, contiguous, fp32 or x's dtype;
    s: the stream of GDR_RES_BEFORE, as residual (written by the forward, read by the backward)."""

    def __init__(self, x, weight, gate=None, activation=GDR_ACT_NONE, residual=None, s=None, placement=GDR_RES_NONE, scale=1.0,
                 eps=1e-6, dtype=None):
        like = x if x is not None else s
        if like is None:
            _bad("x is None")
        self._device_of(like, "x")
        dev = self.device
        if like.dim() not in (2, 3):
            _bad("x must be [T, D] or [T, H, D]")
        if x is None and dtype is None:
            _bad("dtype (of y, dy and dx) must be given without x")
        self.shape = tuple(like.shape)
        self.T, self.D = int(like.shape[0]), int(like.shape[-1])
        self.H = int(like.shape[1]) if like.dim() == 3 else 1
        _sizes(self.T, self.H, self.D)
        self.dtype = dtype if x is None else x.dtype
        if x is not None and dtype is not None and dtype != x.dtype:
            _bad("dtype differs from x's")
        xs = _rows(x, "x", None, None, dev) if x is not None else self.H * self.D
        gs = _rows(gate, "gate", self.shape, self.dtype, dev) if gate is not None else 0
        w_dtype = GDR_F32
        if weight is not None:
            _need(weight, "weight", (self.D,), None, dev)
            w_dtype = _dtype_code(weight.dtype, "weight")
        self.res_dtype = self.dtype
        for t, name in ((residual, "residual"), (s, "s")):
            if t is not None:
                if placement == GDR_RES_NONE:
                    _bad("%s without a placement" % name)
                _need(t, name, self.shape, None, dev)
                self.res_dtype = t.dtype
        if residual is not None and s is not None:
            _need(s, "s", None, residual.dtype, dev)
            if s.data_ptr() == residual.data_ptr() and s.numel():
                _bad("s and residual are the same memory")
        self.placement = int(placement)
        self.x, self.weight, self.gate, self.residual, self.s = x, weight, gate, residual, s
        self._c = _CNorm(self.T, self.H, self.D, _dtype_code(self.dtype, "x"), _dtype_code(self.res_dtype, "residual"), w_dtype, int(activation),
                         self.placement, float(scale), float(eps), xs, gs, _p(x), _p(weight), _p(gate), _p(residual), _p(s))
        self.cstruct = ctypes.byref(self._c)

    def workspace_bytes(self) -> int:
        return norm_workspace_bytes(self.T, self.H, self.D)

    @property
    def y_dtype(self):
        return self.res_dtype if self.placement == GDR_RES_AFTER else self.dtype


def norm_workspace_bytes(T, H, D) -> int:
    _sizes(T, H, D)
    return _bytes(lib().gdr_norm_workspace_bytes(T, H, D))


def norm_fwd(prob, y, stream=None):
    """y: x's shape, contiguous, in x's dtype (the residual's with GDR_RES_AFTER).  Writes prob.s with GDR_RES_BEFORE."""
    _need(y, "y", prob.shape, prob.y_dtype, prob.device)
    _call(prob, stream, "gdr_norm_fwd", _p(y))


def norm_bwd(prob, dy, dx, dw, workspace, dgate=None, ds=None, dres=None, stream=None):
    """dy: as y; dx, dgate: as x, rows at any stride; dw: fp32 [D] or None (then workspace may be None);
    ds, dres: as s, GDR_RES_BEFORE only (dx may be None there, ds too)."""
    import torch

    dev = prob.device
    _need(dy, "dy", prob.shape, prob.y_dtype, dev)
    xs = _rows(dx, "dx", prob.shape, prob.dtype, dev) if dx is not None else 0
    gs = _rows(dgate, "dgate", prob.shape, prob.dtype, dev) if dgate is not None else 0
    for t, name in ((ds, "ds"), (dres, "dres")):
        if t is not None:
            _need(t, name, prob.shape, prob.res_dtype, dev)
    if dw is not None:
        _need(dw, "dw", (prob.D,), torch.float32, dev)
    ws, nbytes = prob._workspace(workspace) if workspace is not None else (None, 0)
    _call(prob, stream, "gdr_norm_bwd", _p(dy), _p(ds), _p(dx), xs, _p(dgate), gs, _p(dres), _p(dw), ws, nbytes)
