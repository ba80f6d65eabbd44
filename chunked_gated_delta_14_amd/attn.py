"""Binding of the softmax-attention layers' operators (see include/gdr.h): rotary
positions, attention over packed documents with its backward, and the cache held in
4 bits with the attention of new tokens over it.

As in the binding of the operators around the recurrence, a problem object holds the
input tensors of a call and its C struct, built and checked once and used for any
number of calls on those tensors; a tensor that does not fit raises GdrError with
GDR_ERR_INVALID_ARG before anything is enqueued.  Calls run on the device of the problem's
tensors, on `stream` or that device's current stream.
"""
from __future__ import annotations

import ctypes

import numpy as np

from . import _check, lib
from .layer import _Base, _bad, _bytes, _call, _dtype_code, _f32, _i32, _i64, _need, _p, _rows, _sizes, _vp

GDR_ROPE_HALF, GDR_ROPE_PAIRS = 0, 1
GDR_ROPE_PLAIN, GDR_ROPE_LINEAR, GDR_ROPE_BASE, GDR_ROPE_BLEND = 0, 1, 2, 3

_f64 = ctypes.c_double


class _CRope(ctypes.Structure):
    _fields_ = [("T", _i32), ("N", _i32), ("H_q", _i32), ("H_k", _i32), ("D", _i32), ("rot", _i32), ("dtype", _i32),
                ("layout", _i32), ("n_chunks", _i32), ("magnitude", _f32), ("q_stride", _i64), ("k_stride", _i64), ("q", _vp),
                ("k", _vp), ("positions", _vp), ("chunk_table", _vp), ("freqs", _vp)]


class _CAttnPlan(ctypes.Structure):
    _fields_ = [("n_q_tiles", _i32), ("n_k_tiles", _i32), ("q_longest", _i32), ("k_longest", _i32), ("q_steps", _i64),
                ("k_steps", _i64), ("table_len", _i64), ("q_items", _i32 * 12), ("k_items", _i32 * 12)]


class _CAttn(ctypes.Structure):
    _fields_ = [("T_q", _i32), ("T_k", _i32), ("N", _i32), ("H_q", _i32), ("H_kv", _i32), ("D", _i32), ("causal", _i32),
                ("window", _i32), ("plan", _CAttnPlan), ("scale", _f32), ("q_stride", _i64),
                ("k_stride", _i64), ("v_stride", _i64), ("q", _vp), ("k", _vp), ("v", _vp), ("tile_table", _vp)]


class _CKv(ctypes.Structure):
    _fields_ = [("n_pages", _i32), ("page", _i32), ("H_kv", _i32), ("D", _i32), ("N", _i32), ("max_pages", _i32),
                ("k_codes", _vp), ("v_codes", _vp), ("k_scale", _vp), ("v_scale", _vp), ("page_table", _vp)]


class _CAttnStep(ctypes.Structure):
    _fields_ = [("T", _i32), ("H_q", _i32), ("window", _i32), ("scale", _f32), ("q_stride", _i64), ("q", _vp), ("lens", _vp),
                ("cu_seqlens", _vp)]


def declare(L) -> None:
    """Argument types of these entry points on the loaded library."""
    P = ctypes.POINTER
    ip = P(_i32)
    for name, args in (
        ("gdr_rope_freqs", [_i32, _f64, _i32, _f64, _f64, _f64, _f64, P(_f64)]),
        ("gdr_rope_fwd", [P(_CRope), _vp, _i64, _vp, _i64, _vp]),
        ("gdr_rope_bwd", [P(_CRope), _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp]),
        ("gdr_plan_attn", [ip, ip, _i32, _i32, _i32, ip, _i64, P(_CAttnPlan)]),
        ("gdr_attn_fwd", [P(_CAttn), _vp, _vp, _vp, _i64, _vp]),
        ("gdr_attn_bwd", [P(_CAttn), _vp, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp]),
        ("gdr_kv_store", [P(_CKv), _i32, _vp, _vp, _vp, _i64, _vp, _i64, _vp]),
        ("gdr_kv_load", [P(_CKv), _i32, _vp, _vp, _vp, _i64, _vp, _i64, _vp]),
        ("gdr_attn_step_fwd", [P(_CKv), P(_CAttnStep), _vp, _vp, _i64, _vp]),
    ):
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, _i32
    L.gdr_attn_workspace_bytes.argtypes, L.gdr_attn_workspace_bytes.restype = [P(_CAttn), _i32], _i64
    L.gdr_attn_step_workspace_bytes.argtypes, L.gdr_attn_step_workspace_bytes.restype = [_i32] * 6, _i64


def _heads(t, name, shape, dtype, device):
    """Rows of [T, H, D] at any stride, as _rows checks them; whole tensors and single tokens pass first."""
    if t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous():
        return shape[1] * shape[2] or 1
    return _rows(t, name, shape, dtype, device)


# ---- rotary positions ----


def rope_freqs(rot, base=10000.0, scaling=GDR_ROPE_PLAIN, factor=1.0, original=4096, low=1.0, high=32.0, device="cuda"):
    """Frequencies of a rope of `rot` channels, in turns a token: fp64 [rot / 2] on `device`."""
    import torch

    _sizes(rot)
    f = np.zeros(max(rot // 2, 1), dtype=np.float64)
    _check(lib().gdr_rope_freqs(rot, base, scaling, factor, original, low, high, f.ctypes.data_as(ctypes.POINTER(_f64))))
    return torch.from_numpy(f).to(device)


class RopeProblem(_Base):
    """Rotary positions of q and k.

    q: bf16 or fp32 [T, H_q, D]; k: [T, H_k, D] of q's type, or None (rows at any stride); freqs: fp64 [rot / 2], as
    rope_freqs gives them; positions: int32 [T] on the device, or None: then plan, the batch's Plan or Problem, and every
    token stands at its place in its document."""

    def __init__(self, q, k, freqs, positions=None, plan=None, layout=GDR_ROPE_HALF, magnitude=1.0):
        import torch

        self._device_of(q, "q")
        dev = self.device
        if q.dim() != 3 or (k is not None and k.dim() != 3):
            _bad("q and k must be [T, H, D]")
        self.T, self.H_q, self.D = (int(x) for x in q.shape)
        self.H_k = int(k.shape[1]) if k is not None else 0
        self.dtype = q.dtype
        code = _dtype_code(q.dtype, "q")
        qs = _rows(q, "q", None, None, dev)
        ks = _rows(k, "k", (self.T, self.H_k, self.D), q.dtype, dev) if k is not None else 0
        _need(freqs, "freqs", None, torch.float64, dev)
        if freqs.dim() != 1:
            _bad("freqs must be [rot / 2]")
        self.rot = 2 * int(freqs.shape[0])
        _sizes(self.T, self.H_q, self.H_k, self.D, self.rot)
        if (positions is None) == (plan is None):
            _bad("either positions or a plan")
        if positions is not None:
            _need(positions, "positions", (self.T,), torch.int32, dev)
        else:
            if plan.T != self.T:
                _bad("the plan holds %d tokens, q %d" % (plan.T, self.T))
            _need(plan.table, "the plan's table", None, None, dev)
        self.q, self.k, self.freqs, self.positions, self.plan = q, k, freqs, positions, plan
        self._c = _CRope(self.T, plan.N if plan else 0, self.H_q, self.H_k, self.D, self.rot, code, int(layout),
                         plan.n_chunks if plan else 0, float(magnitude), qs, ks, _p(q), _p(k), _p(positions),
                         _p(plan.table) if plan else None, _p(freqs))
        self.cstruct = ctypes.byref(self._c)


def _rope_side(prob, t, H, name):
    if H == 0 and t is None:
        return None, 0
    if t is None:
        _bad("%s is None" % name)
    return t.data_ptr(), _heads(t, name, (prob.T, H, prob.D), prob.dtype, prob.device)


def rope_fwd(prob, q_out, k_out=None, stream=None):
    """q_out, k_out: as q and k, rows at any stride; may be q and k themselves."""
    q, qs = _rope_side(prob, q_out, prob.H_q, "q_out")
    k, ks = _rope_side(prob, k_out, prob.H_k, "k_out")
    _call(prob, stream, "gdr_rope_fwd", q, qs, k, ks)


def rope_bwd(prob, dq_out, dk_out, dq, dk, stream=None):
    """dq_out, dk_out: the gradients of the outputs; dq, dk: as q and k, rows at any stride; may be dq_out and dk_out."""
    a, x = _rope_side(prob, dq_out, prob.H_q, "dq_out"), _rope_side(prob, dk_out, prob.H_k, "dk_out")
    b, y = _rope_side(prob, dq, prob.H_q, "dq"), _rope_side(prob, dk, prob.H_k, "dk")
    _call(prob, stream, "gdr_rope_bwd", *a, *x, *b, *y)


# ---- attention over packed documents ----


class AttnPlan:
    """A packed batch's attention tiles on the device, shared by the layers of a step.

    cu_q, cu_k: host sequences or tensors of N+1 ints (cu_k None: cu_q's); window 0: none."""

    def __init__(self, cu_q, cu_k=None, causal=True, window=0, device="cuda"):
        import torch

        def host(cu):
            cu = np.asarray(cu.cpu() if hasattr(cu, "cpu") else cu)
            if cu.size and cu.dtype.kind not in "iu":
                _bad("cu_q and cu_k must be ints, not %s" % cu.dtype)
            if cu.size:
                _sizes(int(cu.min()), int(cu.max()))
            return np.ascontiguousarray(cu, dtype=np.int32)

        cu_q = host(cu_q)
        cu_k = cu_q if cu_k is None else host(cu_k)
        if cu_q.ndim != 1 or cu_q.shape != cu_k.shape or not len(cu_q):
            _bad("cu_q and cu_k must be N+1 ints each")
        _sizes(window)
        self.N, self.T_q, self.T_k = len(cu_q) - 1, int(cu_q[-1]), int(cu_k[-1])
        self.causal, self.window = bool(causal), int(window)
        ip, self.cplan = ctypes.POINTER(_i32), _CAttnPlan()
        args = (cu_q.ctypes.data_as(ip), cu_k.ctypes.data_as(ip), self.N, int(self.causal), self.window)
        _check(lib().gdr_plan_attn(*args, None, 0, ctypes.byref(self.cplan)))
        table = np.zeros(max(self.cplan.table_len, 1), dtype=np.int32)
        _check(lib().gdr_plan_attn(*args, table.ctypes.data_as(ip), table.size, ctypes.byref(self.cplan)))
        self.table = torch.from_numpy(table).to(device)


class AttnProblem(_Base):
    """Softmax attention over a packed batch.

    q: bf16 [T_q, H_q, 128]; k, v: bf16 [T_k, H_kv, 128], rows 16-byte aligned at any stride; plan: the batch's AttnPlan.
    The problem holds the forward's workspace: none unless tiles of 128 rows and 64 keys differ so much in number of keys, or are
    so few, that long ones are shared by several blocks; then 65 KB a part and head, 182 MB at most (below 2^11 steps of
    64 keys a part).  What it holds follows from the problem's inputs alone, so calls that overlap without those changing write
    the same there; overlapping calls on changing inputs would race on the inputs already.  Keep the problem until its calls
    are done.  share: another problem, whose forward's workspace this one uses too, as the layers of a model can, whose calls
    follow each other (those of problems that share must not overlap)."""

    def __init__(self, q, k, v, plan, scale=None, share=None):
        import torch

        self._device_of(q, "q")
        dev, bf = self.device, torch.bfloat16
        if q.dim() != 3 or k.dim() != 3:
            _bad("q and k must be [T, H, 128]")
        self.T_q, self.H_q, self.D = (int(x) for x in q.shape)
        self.T_k, self.H_kv = int(k.shape[0]), int(k.shape[1])
        _sizes(self.T_q, self.H_q, self.D, self.T_k, self.H_kv)
        if plan.T_q != self.T_q or plan.T_k != self.T_k:
            _bad("the plan holds %d queries and %d keys, q %d and k %d" % (plan.T_q, plan.T_k, self.T_q, self.T_k))
        qs = _rows(q, "q", None, bf, dev)
        ks = _rows(k, "k", (self.T_k, self.H_kv, self.D), bf, dev)
        vs = _rows(v, "v", (self.T_k, self.H_kv, self.D), bf, dev)
        _need(plan.table, "the plan's table", None, None, dev)
        self.q, self.k, self.v, self.plan = q, k, v, plan
        self.scale = float(self.D ** -0.5 if scale is None else scale)
        self._c = _CAttn(self.T_q, self.T_k, plan.N, self.H_q, self.H_kv, self.D, int(plan.causal), plan.window, plan.cplan,
                         self.scale, qs, ks, vs, _p(q), _p(k), _p(v), _p(plan.table))
        self.cstruct = ctypes.byref(self._c)
        self._fwd_bytes = _bytes(lib().gdr_attn_workspace_bytes(self.cstruct, 0))
        self._fwd_ws = None
        if self._fwd_bytes and share is not None:
            if share.device != dev or share._fwd_bytes < self._fwd_bytes:
                _bad("the shared workspace must be on %s and hold %d bytes, not %d" % (dev, self._fwd_bytes, share._fwd_bytes))
            self._fwd_ws = share._fwd_ws
        elif self._fwd_bytes:
            self._fwd_ws = torch.empty(self._fwd_bytes, dtype=torch.uint8, device=dev)

    def workspace_bytes(self) -> int:
        return _bytes(lib().gdr_attn_workspace_bytes(self.cstruct, 1))


def attn_fwd(prob, o, lse=None, stream=None):
    """o: bf16 [T_q, H_q, 128]; lse: fp32 [H_q, T_q] (which the backward takes), or None."""
    import torch

    _need(o, "o", (prob.T_q, prob.H_q, prob.D), torch.bfloat16, prob.device)
    if lse is not None:
        _need(lse, "lse", (prob.H_q, prob.T_q), torch.float32, prob.device)
    _call(prob, stream, "gdr_attn_fwd", _p(o), _p(lse), _p(prob._fwd_ws), prob._fwd_bytes)


def attn_bwd(prob, o, lse, dout, dq, dk, dv, workspace, stream=None):
    """o, lse: as the forward wrote them; dout: bf16 [T_q, H_q, 128]; dq: as q, dk, dv: as k and v, rows 16-byte aligned
    at any stride."""
    import torch

    dev, bf = prob.device, torch.bfloat16
    q, kv = (prob.T_q, prob.H_q, prob.D), (prob.T_k, prob.H_kv, prob.D)
    _need(o, "o", q, bf, dev)
    _need(dout, "dout", q, bf, dev)
    _need(lse, "lse", (prob.H_q, prob.T_q), torch.float32, dev)
    dqs, dks, dvs = _heads(dq, "dq", q, bf, dev), _heads(dk, "dk", kv, bf, dev), _heads(dv, "dv", kv, bf, dev)
    ws, nbytes = prob._workspace(workspace)
    _call(prob, stream, "gdr_attn_bwd", _p(o), _p(lse), _p(dout), _p(dq), dqs, _p(dk), dks, _p(dv), dvs, ws, nbytes)


# ---- the cache in 4 bits ----


class KvCache:
    """A pool of pages: codes uint8 [n_pages, H_kv, page, 64], scales uint8 [n_pages, H_kv, page, 4], for k and for v."""

    def __init__(self, k_codes, k_scale, v_codes, v_scale):
        import torch

        if k_codes.device.type != "cuda":
            _bad("k_codes must be on a GPU")
        if k_codes.dim() != 4:
            _bad("k_codes must be [n_pages, H_kv, page, 64]")
        self.device = k_codes.device
        self.n_pages, self.H_kv, self.page = (int(x) for x in k_codes.shape[:3])
        self.D = 2 * int(k_codes.shape[3])
        _sizes(self.n_pages, self.H_kv, self.page, self.D)
        codes, scale = tuple(k_codes.shape), (self.n_pages, self.H_kv, self.page, self.D // 32)
        for t, name, shape in ((k_codes, "k_codes", codes), (v_codes, "v_codes", codes), (k_scale, "k_scale", scale),
                               (v_scale, "v_scale", scale)):
            _need(t, name, shape, torch.uint8, self.device)
        self.k_codes, self.k_scale, self.v_codes, self.v_scale = k_codes, k_scale, v_codes, v_scale

    @classmethod
    def empty(cls, n_pages, H_kv, page=64, device="cuda"):
        import torch

        def make(width):
            return torch.zeros(n_pages, H_kv, page, width, dtype=torch.uint8, device=device)

        return cls(make(64), make(4), make(64), make(4))

    def _struct(self, page_table):
        import torch

        if page_table.dim() != 2:
            _bad("page_table must be [N, max_pages]")
        N, width = (int(x) for x in page_table.shape)
        _sizes(N, width)
        _need(page_table, "page_table", None, torch.int32, self.device)
        return _CKv(self.n_pages, self.page, self.H_kv, self.D, N, width, _p(self.k_codes), _p(self.v_codes), _p(self.k_scale),
                    _p(self.v_scale), _p(page_table))


class KvProblem(_Base):
    """Tokens of N sequences and their places in a cache.

    page_table: int32 [N, max_pages]; start: int32 [N], each sequence's place of its first token here, or None for zeros;
    T: tokens (rows of k and v); cu_seqlens: int32 [N+1], or None for one token a sequence (all on the cache's device)."""

    def __init__(self, cache, page_table, start, T, cu_seqlens=None):
        import torch

        self.device, self.cache, self.T = cache.device, cache, int(T)
        _sizes(self.T)
        self._c = cache._struct(page_table)
        self.N = int(page_table.shape[0])
        if start is not None:
            _need(start, "start", (self.N,), torch.int32, self.device)
        if cu_seqlens is not None:
            _need(cu_seqlens, "cu_seqlens", (self.N + 1,), torch.int32, self.device)
        self.page_table, self.start, self.cu_seqlens = page_table, start, cu_seqlens
        self.cstruct = ctypes.byref(self._c)


def _kv(name, prob, k, v, stream):
    import torch

    shape = (prob.T, prob.cache.H_kv, prob.cache.D)
    ks, vs = (_heads(t, n, shape, torch.bfloat16, prob.device) for t, n in ((k, "k"), (v, "v")))
    _call(prob, stream, name, prob.T, _p(prob.cu_seqlens), _p(prob.start), _p(k), ks, _p(v), vs)


def kv_store(prob, k, v, stream=None):
    """k, v: bf16 [T, H_kv, 128], rows at any stride.  Updates the cache."""
    _kv("gdr_kv_store", prob, k, v, stream)


def kv_load(prob, k, v, stream=None):
    """k, v: bf16 [T, H_kv, 128], rows at any stride, written."""
    _kv("gdr_kv_load", prob, k, v, stream)


class AttnStep(_Base):
    """Attention of each sequence's last tokens over its cache.

    q: bf16 [T, H_q, 128], rows at any stride; page_table: int32 [N, max_pages]; lens: int32 [N], the tokens each sequence
    holds, these rows' own among them; cu_seqlens: int32 [N+1], or None for one row a sequence; window 0: none."""

    def __init__(self, q, cache, page_table, lens, cu_seqlens=None, window=0, scale=None):
        import torch

        self._device_of(q, "q")
        dev = self.device
        if q.dim() != 3:
            _bad("q must be [T, H_q, 128]")
        if cache.device != dev:
            _bad("the cache must be on %s, not %s" % (dev, cache.device))
        self.T, self.H_q = int(q.shape[0]), int(q.shape[1])
        _sizes(self.T, self.H_q, window)
        qs = _rows(q, "q", (self.T, self.H_q, cache.D), torch.bfloat16, dev)
        self._cache = cache._struct(page_table)
        self.N, self.max_pages = (int(x) for x in page_table.shape)
        _need(lens, "lens", (self.N,), torch.int32, dev)
        if cu_seqlens is not None:
            _need(cu_seqlens, "cu_seqlens", (self.N + 1,), torch.int32, dev)
        self.scale = float(cache.D ** -0.5 if scale is None else scale)
        self.q, self.cache, self.page_table, self.lens, self.cu_seqlens = q, cache, page_table, lens, cu_seqlens
        self._c = _CAttnStep(self.T, self.H_q, int(window), self.scale, qs, _p(q), _p(lens), _p(cu_seqlens))
        self.cstruct = ctypes.byref(self._cache)
        self._step = ctypes.byref(self._c)

    def workspace_bytes(self) -> int:
        return attn_step_workspace_bytes(self.T, self.N, self.H_q, self.cache.H_kv, self.max_pages, self.cache.page)


def attn_step_workspace_bytes(T, N, H_q, H_kv, max_pages, page) -> int:
    _sizes(T, N, H_q, H_kv, max_pages, page)
    return _bytes(lib().gdr_attn_step_workspace_bytes(T, N, H_q, H_kv, max_pages, page))


def attn_step(prob, o, workspace, stream=None):
    """o: bf16 [T, H_q, 128]."""
    import torch

    _need(o, "o", tuple(prob.q.shape), torch.bfloat16, prob.device)
    ws, nbytes = prob._workspace(workspace)
    _call(prob, stream, "gdr_attn_step_fwd", prob._step, _p(o), ws, nbytes)
