"""GPU tests of the operators around the recurrence (convolution, gate, single-token
recurrence, norm) against fp64 references with derived bounds (layer_ref.py)."""
import numpy as np
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DT = {"bf16": BF, "f32": F32}


def gdr():
    import chunked_gated_delta_14_amd as m

    return m


def rng(seed):
    return np.random.default_rng(seed)


def dev(a, dtype=F32, pad=0):
    """The array on the GPU, rounded to dtype; with pad, as rows of a wider buffer filled with NaN."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()
    if not pad:
        return t
    rows = t.reshape(t.shape[0], -1)
    wide = torch.full((rows.shape[0], rows.shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
    wide[:, :rows.shape[1]] = rows
    v = wide[:, :rows.shape[1]]
    return v if t.dim() == 2 else v.unflatten(1, tuple(t.shape[1:]))


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def nan(shape, dtype, pad=0):
    shape = tuple(shape)
    inner = int(np.prod(shape[1:])) if len(shape) > 1 else 1
    if not pad:
        return torch.full(shape, float("nan"), dtype=dtype, device="cuda")
    wide = torch.full((shape[0], inner + pad), float("nan"), dtype=dtype, device="cuda")
    v = wide[:, :inner]
    return v if len(shape) == 2 else v.unflatten(1, shape[1:])


def padding_untouched(t, width):
    """The pad columns of a strided output still hold NaN."""
    base = t._base if t._base is not None else t
    while base._base is not None:
        base = base._base
    if base.shape[1] > width:
        assert bool(torch.isnan(base[:, width:].float()).all()), "columns beside the rows were written"


# ---- convolution ----

CONV = [
    # docs, C, W, dtype, w dtype, silu, bias, s0, pad
    ((1,), 1, 2, "bf16", "bf16", True, True, True, 0),
    ((1, 0, 2, 3, 1), 8, 4, "bf16", "bf16", True, True, True, 0),
    ((200, 312), 128, 4, "bf16", "bf16", True, False, False, 0),
    ((1, 63, 64, 65, 130, 7, 0), 264, 4, "bf16", "f32", True, True, True, 8),
    ((130, 66, 2), 130, 3, "bf16", "bf16", True, True, True, 3),   # rows off 16-byte alignment, odd tail
    ((3, 129, 1, 64), 7, 5, "bf16", "bf16", False, True, True, 0),  # narrower than a group
    ((70, 5), 2056, 4, "bf16", "bf16", True, False, True, 0),       # two channel blocks
    ((64, 1, 127), 36, 2, "f32", "f32", True, True, True, 0),
    ((300, 0, 5), 131, 8, "f32", "bf16", True, False, True, 5),
    ((2, 2, 2, 191), 3, 8, "f32", "f32", False, False, False, 1),
    ((64, 64), 1028, 6, "f32", "f32", True, True, False, 0),
    ((90, 38), 72, 7, "bf16", "f32", True, True, True, 0),
    ((9000, 3, 3400), 2048, 4, "bf16", "bf16", True, False, False, 0),  # workers of several 64-token runs
    ((1500, 700), 512, 4, "bf16", "bf16", True, False, True, 16),
]


def conv_inputs(docs, C, W, dt, wdt, bias, s0, pad, seed):
    r, T, N = rng(seed), sum(docs), len(docs)
    x = dev(r.standard_normal((T, C)), DT[dt], pad)
    w = dev(0.5 * r.standard_normal((C, W)), DT[wdt])
    b = dev(0.2 * r.standard_normal(C), DT[wdt]) if bias else None
    h = dev(r.standard_normal((N, W - 1, C)), DT[dt]) if s0 else None
    dy = dev(r.standard_normal((T, C)), DT[dt], pad)
    dst = dev(r.standard_normal((N, W - 1, C)), DT[dt]) if s0 else None
    return x, w, b, h, dy, dst


def cu_of(docs):
    return np.concatenate([[0], np.cumsum(docs)]).astype(np.int32)


@pytest.mark.parametrize("case", CONV, ids=lambda c: "%s_C%d_W%d_%s" % ("-".join(map(str, c[0])), c[1], c[2], c[3]))
def test_conv(case):
    docs, C, W, dt, wdt, silu, bias, s0, pad = case
    g = gdr()
    x, w, b, h, dy, dst = conv_inputs(docs, C, W, dt, wdt, bias, s0, pad, sum(docs) + C)
    T, N = sum(docs), len(docs)
    act = g.GDR_ACT_SILU if silu else g.GDR_ACT_NONE
    p = g.ConvProblem(x, w, g.Plan(cu_of(docs)), b, h, act)
    print("[case] conv", case, flush=True)
    y, st = nan((T, C), DT[dt], pad), nan((N, W - 1, C), DT[dt])
    g.conv_fwd(p, y, st)
    ws = p.alloc_workspace().fill_(0xFF)
    dx, dw, db = nan((T, C), DT[dt], pad), nan((C, W), F32), nan((C,), F32)
    ds0 = nan((N, W - 1, C), DT[dt])
    g.conv_bwd(p, dy, dst, dx, dw, db, ds0, ws)
    torch.cuda.synchronize()
    f = ref.conv(f64(x), f64(w), f64(b) if bias else 0.0 * f64(w)[:, 0], f64(h), docs, silu)
    d = ref.conv_grad(f, f64(x), f64(w), docs, f64(dy), f64(dst), silu)
    ref.close(y, f["y"], f["Ey"], DT[dt], "y")
    assert np.array_equal(f64(st), f["st"]), "st"
    for name, t, odt in (("dx", dx, DT[dt]), ("dw", dw, F32), ("db", db, F32), ("ds0", ds0, DT[dt])):
        ref.close(t, d[name], d["E" + name], odt, name)
    padding_untouched(y, C)
    padding_untouched(dx, C)
    # the optional outputs left out change nothing else, and the sums repeat bit for bit
    y2, dx2, dw2 = nan((T, C), DT[dt]), nan((T, C), DT[dt]), nan((C, W), F32)
    g.conv_fwd(p, y2)
    g.conv_bwd(p, dy, dst, dx2, dw2, None, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(y2, y.contiguous()) and torch.equal(dx2, dx.contiguous()) and torch.equal(dw2, dw)


def test_conv_empty_batches():
    """No tokens: final rows are the carried-in ones, parameter gradients zero; no documents: nothing but the zeros."""
    g = gdr()
    for docs in ((), (0, 0)):
        x, w, b, h, dy, dst = conv_inputs(docs, 24, 4, "bf16", "bf16", True, True, 0, 3)
        p = g.ConvProblem(x, w, g.Plan(cu_of(docs)), b, h)
        st, ds0 = nan(h.shape, BF), nan(h.shape, BF)
        y, dx, dw, db = nan((0, 24), BF), nan((0, 24), BF), nan((24, 4), F32), nan((24,), F32)
        g.conv_fwd(p, y, st)
        g.conv_bwd(p, dy, dst, dx, dw, db, ds0, p.alloc_workspace())
        torch.cuda.synchronize()
        assert torch.equal(st, h) and torch.equal(ds0, dst)
        assert not dw.any() and not db.any()


@pytest.mark.parametrize("N,C,W,dt,pad", [(1, 128, 4, "bf16", 0), (5, 10240, 4, "bf16", 16), (9, 37, 3, "bf16", 0),
                                          (4, 260, 2, "f32", 3), (3, 6, 8, "f32", 0), (70, 24, 5, "bf16", 0)])
def test_conv_step(N, C, W, dt, pad):
    """Three tokens in turn equal the convolution of the sequence; idle and padding slots stay as they were."""
    g, r = gdr(), rng(N + C)
    dtype = DT[dt]
    n_slots = N + 3
    w, b = dev(0.5 * r.standard_normal((C, W)), dtype), dev(0.2 * r.standard_normal(C), dtype)
    state = dev(r.standard_normal((n_slots, W - 1, C)), dtype)
    slots = torch.from_numpy(r.permutation(n_slots)[:N].astype(np.int32)).cuda()
    if N > 3:
        slots[1], slots[2] = -1, n_slots  # padding rows
    live = [n for n in range(N) if 0 <= int(slots[n]) < n_slots]
    before = state.clone()
    xs = [dev(r.standard_normal((N, C)), dtype, pad) for _ in range(3)]
    ys = []
    print("[case] conv step", N, C, W, dt, flush=True)
    for x in xs:
        y = nan((N, C), dtype, pad)
        g.conv_step(g.ConvStep(x, w, state, slots, b), y)
        ys.append(y)
    torch.cuda.synchronize()
    sl = slots.cpu().numpy()
    want = f64(before)
    for n in live:
        s0 = f64(before)[sl[n]]
        f = ref.conv(np.stack([f64(x)[n] for x in xs]), f64(w), f64(b), s0[None], (3,), True)
        ref.close(torch.stack([y[n] for y in ys]), f["y"], f["Ey"], dtype, "y of sequence %d" % n)
        want[sl[n]] = f["st"][0]
    assert np.array_equal(f64(state), want), "state"
    for n in set(range(N)) - set(live):
        assert all(bool(torch.isnan(y[n].float()).all()) for y in ys), "a padding row was written"
    # without slots: sequence n in slot n
    state2, y = before.clone(), nan((N, C), dtype)
    g.conv_step(g.ConvStep(xs[0], w, state2, None, b), y)
    torch.cuda.synchronize()
    f = ref.conv(f64(xs[0]), f64(w), f64(b), f64(before)[:N], (1,) * N, True)
    ref.close(y, f["y"], f["Ey"], dtype, "y without slots")
    assert np.array_equal(f64(state2)[:N], f["st"]) and torch.equal(state2[N:], before[N:])


# ---- gate ----

GATE = [
    # T, H, D, kind, dtype, bias, pad
    (1, 1, 1, "softplus", "f32", True, 0),
    (1, 1, 128, "sigmoid", "bf16", True, 0),
    (77, 3, 128, "softplus", "bf16", True, 0),
    (130, 2, 128, "sigmoid", "f32", False, 4),
    (300, 48, 1, "softplus", "bf16", True, 0),
    (65, 5, 1, "softplus", "f32", False, 3),
    (9, 13, 1, "sigmoid", "bf16", True, 1),
    (700, 1, 1, "sigmoid", "bf16", True, 0),
    (40, 17, 128, "softplus", "f32", True, 0),
    (5000, 2, 128, "softplus", "bf16", True, 0),
    (20000, 3, 1, "softplus", "f32", True, 0),
]


@pytest.mark.parametrize("case", GATE, ids=lambda c: "T%d_H%d_D%d_%s_%s" % c[:5])
def test_gate(case):
    T, H, D, kind, dt, bias, pad = case
    g, r = gdr(), rng(T * H + D)
    dtype = DT[dt]
    print("[case] gate", case, flush=True)
    x = dev(2.0 * r.standard_normal((T, H * D)), dtype, pad)
    a = dev(0.7 * r.standard_normal(H))
    b = dev(r.standard_normal(H * D)) if bias else None
    dg = dev(r.standard_normal((T, H * D)))
    p = g.GateProblem(x, a, b, g.GDR_GATE_SOFTPLUS if kind == "softplus" else g.GDR_GATE_SIGMOID, -5.0)
    out, dx = nan((T, H * D), F32), nan((T, H * D), dtype, pad)
    da, db = nan((H,), F32), nan((H * D,), F32)
    g.gate_fwd(p, out)
    g.gate_bwd(p, dg, dx, da, db, p.alloc_workspace().fill_(0xFF))
    torch.cuda.synchronize()
    X, B, DG = f64(x).reshape(T, H, D), (f64(b) if bias else np.zeros(H * D)).reshape(H, D), f64(dg).reshape(T, H, D)
    v, E = ref.gate(X, f64(a), B, kind, -5.0)
    if kind == "softplus":
        # a value within its fp32 error of the floor may land on either side of it, where the slope jumps: none here
        raw = -np.exp(f64(a))[:, None] * np.logaddexp(X + B, 0)
        assert not (np.abs(raw + 5.0) <= E * ref.U).any()
        assert (v == -5.0).any() or T < 60 or not bias, "the floor is not exercised"
    ref.close(out.view(T, H, D), v, E, F32, "g")
    d = ref.gate_grad(X, f64(a), B, kind, -5.0, DG)
    ref.close(dx.reshape(T, H, D), d["dx"], d["Edx"], dtype, "dx")
    ref.close(da, d["da"], d["Eda"], F32, "da")
    ref.close(db.view(H, D), d["db"], d["Edb"], F32, "db")
    padding_untouched(dx, H * D)
    da2, dx2 = nan((H,), F32), nan((T, H * D), dtype)
    g.gate_bwd(p, dg, dx2, da2, None, p.alloc_workspace())
    torch.cuda.synchronize()
    assert torch.equal(da2, da) and torch.equal(dx2, dx.contiguous())


def test_gate_extremes():
    """Infinities, far values and NaN: the limits of the formulas, and zero slopes there."""
    g = gdr()
    x = torch.tensor([[float("inf"), -float("inf"), 300.0, -300.0, float("nan"), 0.0]], device="cuda")
    a = torch.zeros(6, device="cuda")
    for kind, want in ((g.GDR_GATE_SOFTPLUS, [-5, 0, -5, 0, float("nan"), -np.log(2)]),
                       (g.GDR_GATE_SIGMOID, [-5, 0, -5, 0, float("nan"), -2.5])):
        p = g.GateProblem(x, a, None, kind, -5.0)
        out, dx, da, dg = nan((1, 6), F32), nan((1, 6), F32), nan((6,), F32), torch.ones(1, 6, device="cuda")
        g.gate_fwd(p, out)
        g.gate_bwd(p, dg, dx, da, None, p.alloc_workspace())
        torch.cuda.synchronize()
        assert np.allclose(f64(out)[0], want, rtol=1e-6, atol=1e-30, equal_nan=True), out
        slopes = f64(dx)[0]
        assert np.array_equal(np.isnan(slopes), np.isnan(want)) and np.all(np.abs(slopes[:4]) < 1e-30), dx
        assert np.array_equal(np.isnan(f64(da)), np.isnan(want)), da


def test_gate_empty():
    g = gdr()
    p = g.GateProblem(torch.empty(0, 256, dtype=BF, device="cuda"), torch.zeros(2, device="cuda"))
    da, db = nan((2,), F32), nan((256,), F32)
    g.gate_fwd(p, torch.empty(0, 256, device="cuda"))
    g.gate_bwd(p, torch.empty(0, 256, device="cuda"), torch.empty(0, 256, dtype=BF, device="cuda"), da, db, p.alloc_workspace())
    torch.cuda.synchronize()
    assert not da.any() and not db.any()


# ---- single-token recurrence ----

STEP = [
    # variant, docs, H_qk, H_v, spare slots, activations, pad
    ("kda", (1,), 1, 1, 0, False, 0),
    ("gdn", (1,), 1, 1, 0, True, 0),
    ("kda", (1, 1, 1), 3, 3, 2, True, 0),
    ("gdn", (1, 1, 1, 1, 1), 2, 6, 1, False, 8),
    ("kda", (4, 0, 1, 7), 2, 2, 3, False, 3),
    ("gdn", (2, 9, 0, 1), 1, 3, 0, True, 0),
    ("gdn", (33,), 4, 4, 0, False, 0),
]


def step_inputs(variant, docs, hqk, hv, spare, pad, seed, unit=True):
    r, T = rng(seed), sum(docs)

    def heads(H, u):
        x = r.standard_normal((T, H, 128))
        return dev(x / np.linalg.norm(x, axis=-1, keepdims=True) if u else x, BF, pad)

    q, k, v = heads(hqk, unit), heads(hqk, unit), heads(hv, False)
    g = dev(-5 * r.random((T, hv, 128) if variant == "kda" else (T, hv)))
    beta = dev(r.standard_normal((T, hv)) if not unit else 1 / (1 + np.exp(-r.standard_normal((T, hv)))),
               BF if variant == "kda" else F32)
    state = dev(0.1 * r.standard_normal((len(docs) + spare, hv, 128, 128)))
    slots = torch.from_numpy(r.permutation(len(docs) + spare)[:len(docs)].astype(np.int32)).cuda()
    return q, k, v, g, beta, state, slots


@pytest.mark.parametrize("case", STEP, ids=lambda c: "%s_%s_h%d_%d" % (c[0], "-".join(map(str, c[1])), c[2], c[3]))
def test_step(case):
    variant, docs, hqk, hv, spare, act, pad = case
    g = gdr()
    q, k, v, gate, beta, state, slots = step_inputs(variant, docs, hqk, hv, spare, pad, sum(docs) + hv, not act)
    before = state.clone()
    single = all(n == 1 for n in docs)
    cu = None if single else torch.from_numpy(cu_of(docs)).cuda()
    print("[case] step", case, flush=True)
    p = g.StepProblem(g.GDR_KDA if variant == "kda" else g.GDR_GDN, q, k, v, gate, beta, state, cu, slots,
                      input_flags=g.GDR_IN_QK_L2NORM | g.GDR_IN_BETA_SIGMOID if act else 0)
    o = nan(v.shape, BF)
    (g.kda_step if variant == "kda" else g.gdn_step)(p, o)
    torch.cuda.synchronize()
    ro, Eo, rs, Es = ref.step(f64(q), f64(k), f64(v), f64(gate), f64(beta), f64(before), docs, slots.cpu().numpy(), 128 ** -0.5,
                              act, act)
    ref.close(o, ro, Eo, BF, "o")
    ref.close(state, rs, Es, F32, "state")
    idle = sorted(set(range(len(before))) - {int(s) for s, n in zip(slots, docs) if n})
    assert torch.equal(state[idle], before[idle]), "an idle slot was written"


def test_step_skips_padding():
    """Slots outside the pool, empty sequences and rows behind the last sequence are left as they were; a cu_seqlens that
    runs past T is clipped."""
    g = gdr()
    docs = (1, 2, 1, 1)
    q, k, v, gate, beta, state, slots = step_inputs("gdn", docs, 1, 2, 1, 0, 5)
    slots[1], slots[2] = -3, 5
    before = state.clone()
    cu = torch.tensor([0, 1, 3, 4, 4], dtype=torch.int32, device="cuda")  # the last row belongs to no sequence
    o = nan(v.shape, BF)
    g.gdn_step(g.StepProblem(g.GDR_GDN, q, k, v, gate, beta, state, cu, slots), o)
    torch.cuda.synchronize()
    ro, Eo, rs, Es = ref.step(f64(q), f64(k), f64(v), f64(gate), f64(beta), f64(before), (1,), [int(slots[0])], 128 ** -0.5, False, False)
    ref.close(o[:1], ro[:1], Eo[:1], BF, "o")
    assert bool(torch.isnan(o[1:].float()).all())
    ref.close(state, rs, Es, F32, "state")
    state2, o2 = before.clone(), nan(v.shape, BF)
    past = torch.tensor([0, 1, 3, 4, 9], dtype=torch.int32, device="cuda")
    g.gdn_step(g.StepProblem(g.GDR_GDN, q, k, v, gate, beta, state2, past, None), o2)
    torch.cuda.synchronize()
    ro, Eo, rs, Es = ref.step(f64(q), f64(k), f64(v), f64(gate), f64(beta), f64(before), docs, [0, 1, 2, 3], 128 ** -0.5, False, False)
    ref.close(o2, ro, Eo, BF, "o")
    ref.close(state2, rs, Es, F32, "state")


# ---- norm ----

NORM = [
    # T, H, D, placement, dtype, residual dtype, activation, weight dtype, pad
    (1, 1, 1, "none", "f32", "f32", "none", "f32", 0),
    (5, 3, 128, "none", "bf16", "bf16", "silu", "f32", 0),
    (37, 16, 128, "none", "bf16", "bf16", "sigmoid", "bf16", 8),
    (9, 2, 128, "none", "f32", "f32", "silu", "f32", 3),
    (7, 5, 64, "none", "bf16", "bf16", "silu", None, 0),
    (11, 1, 7, "before", "bf16", "f32", "none", "f32", 1),
    (19, 1, 257, "before", "bf16", "bf16", "none", "bf16", 0),
    (6, 1, 2048, "before", "bf16", "f32", "none", "f32", 0),
    (6, 1, 2048, "after", "bf16", "bf16", "silu", "f32", 16),
    (3, 1, 2049, "after", "f32", "f32", "sigmoid", "f32", 0),
    (4, 1, 5001, "before", "bf16", "f32", "silu", "bf16", 0),
    (2, 1, 10240, "after", "bf16", "f32", "none", "f32", 0),
    (2, 1, 16384, "none", "f32", "f32", "none", "f32", 0),
    (300, 1, 384, "before", "f32", "f32", "none", None, 4),
    (1030, 5, 40, "none", "bf16", "bf16", "silu", "f32", 0),
    (3, 2, 700, "none", "bf16", "bf16", "sigmoid", "f32", 5),
    (1500, 1, 1200, "before", "bf16", "bf16", "silu", "f32", 0),
    (20000, 1, 40, "after", "bf16", "f32", "sigmoid", "f32", 0),
    (5, 1, 3000, "none", "bf16", "bf16", "silu", "f32", 0),
    (3, 1, 8000, "after", "bf16", "f32", "silu", "f32", 8),
    (700, 1, 5120, "before", "f32", "f32", "none", "f32", 0),
    (2, 1, 12000, "before", "bf16", "f32", "sigmoid", "f32", 0),
    (3, 1, 16001, "before", "bf16", "bf16", "silu", "f32", 1),
    (2, 1, 8192, "after", "f32", "f32", "silu", "f32", 0),
    (2, 1, 16383, "before", "f32", "f32", "silu", "bf16", 0),
]


@pytest.mark.parametrize("case", NORM, ids=lambda c: "T%d_H%d_D%d_%s_%s_%s_%s" % c[:7])
def test_norm(case):
    T, H, D, place, dt, rdt, act, wdt, pad = case
    g, r = gdr(), rng(T + D)
    dtype, rtype = DT[dt], DT[rdt]
    shape = (T, H, D)
    print("[case] norm", case, flush=True)
    x = dev(r.standard_normal(shape), dtype, pad)
    w = dev(1 + 0.2 * r.standard_normal(D), DT[wdt]) if wdt else None
    z = dev(2 * r.standard_normal(shape), dtype, pad) if act != "none" else None
    res = dev(r.standard_normal(shape), rtype) if place != "none" else None
    s = nan(shape, rtype) if place == "before" else None
    ydt = rtype if place == "after" else dtype
    dy = dev(r.standard_normal(shape), ydt)
    ds = dev(r.standard_normal(shape), rtype) if place == "before" else None
    alpha = 0.5 if place != "none" else 1.0
    kinds = {"none": (g.GDR_ACT_NONE, g.GDR_RES_NONE), "silu": (g.GDR_ACT_SILU,), "sigmoid": (g.GDR_ACT_SIGMOID,),
             "before": g.GDR_RES_BEFORE, "after": g.GDR_RES_AFTER}
    code = g.GDR_RES_NONE if place == "none" else kinds[place]
    p = g.NormProblem(x, w, z, kinds[act][0], res, s, code, alpha, 1e-6)
    y, dx, dw = nan(shape, ydt), nan(shape, dtype, pad), nan((D,), F32)
    dz = nan(shape, dtype, pad) if z is not None else None
    dres = nan(shape, rtype) if place == "before" else None
    g.norm_fwd(p, y)
    g.norm_bwd(p, dy, dx, dw, p.alloc_workspace().fill_(0xFF), dz, ds, dres)
    torch.cuda.synchronize()
    W = f64(w) if w is not None else np.ones(D)
    f = ref.norm(f64(x), W, f64(z), f64(res), place, act, alpha, 1e-6)
    ref.close(y, f["y"], f["Ey"], ydt, "y")
    if s is not None:
        ref.close(s, f["s"], f["Es"], rtype, "s")
    d = ref.norm_grad(f64(s) if s is not None else f64(x), W, f64(z), f64(dy), f64(ds), place, act, alpha, 1e-6)
    ref.close(dx, d["dx"], d["Edx"], dtype, "dx")
    ref.close(dw, d["dw"], d["Edw"], F32, "dw")
    padding_untouched(dx, H * D)
    if dz is not None:
        ref.close(dz, d["dz"], d["Edz"], dtype, "dz")
        padding_untouched(dz, H * D)
    if dres is not None:
        ref.close(dres, d["dres"], d["Edres"], rtype, "dres")
        # the backward needs only the stream: without x, without dx, ds and dw
        q = g.NormProblem(None, w, z, kinds[act][0], None, s, code, alpha, 1e-6, dtype=dtype)
        dres2 = nan(shape, rtype)
        g.norm_bwd(q, dy, None, None, None, dz, None, dres2)
        torch.cuda.synchronize()
        d2 = ref.norm_grad(f64(s), W, f64(z), f64(dy), None, place, act, alpha, 1e-6)
        ref.close(dres2, d2["dres"], d2["Edres"], rtype, "dres without ds")


@pytest.mark.parametrize("place,act,eps", [("none", "none", 1e-6), ("after", "silu", 1e-6), ("before", "none", 1e-3),
                                            ("none", "sigmoid", 0.0)])
def test_norm_rows_of_one_value(place, act, eps):
    """D = 1: du = eps rs^3 v, to a few roundings of itself although v and u rs^2 mean(v u) nearly cancel."""
    g, r = gdr(), rng(int(1e4 * eps) + len(act))
    acts = {"none": g.GDR_ACT_NONE, "silu": g.GDR_ACT_SILU, "sigmoid": g.GDR_ACT_SIGMOID}
    codes = {"none": g.GDR_RES_NONE, "before": g.GDR_RES_BEFORE, "after": g.GDR_RES_AFTER}
    shape, alpha = (333, 2, 1), 0.5 if place != "none" else 1.0
    print("[case] norm of one value", place, act, eps, flush=True)
    x, dy, res = (dev(r.standard_normal(shape), F32) for _ in range(3))
    w = dev(1 + 0.2 * r.standard_normal(1), F32)
    z = dev(2 * r.standard_normal(shape), F32) if act != "none" else None
    s = x if place == "before" else None  # the stored stream
    p = g.NormProblem(None if s is not None else x, w, z, acts[act], None if place != "after" else res, s, codes[place], alpha,
                      eps, **(dict(dtype=F32) if s is not None else {}))
    dx, dw = nan(shape, F32), nan((1,), F32)
    dz = nan(shape, F32) if z is not None else None
    dres = nan(shape, F32) if place == "before" else None
    g.norm_bwd(p, dy, None if place == "before" else dx, dw, p.alloc_workspace(), dz, None, dres)
    torch.cuda.synchronize()
    e = float(np.float32(eps))
    a, Ea, _, _ = ref._act(f64(z), act)
    t = f64(dy) * f64(w) * (alpha if place == "after" else 1.0)
    scale = e / np.sqrt(f64(x) ** 2 + e) ** 3
    # rs: the square, the sum and rsq (two) at half the relative error of its argument, 3; cubed 9; its products 3;
    # v's 3 and the last 1, over the activation's own error
    want = scale * t * a
    ref.close(dx if place != "before" else dres, want, 16 * np.abs(want) + scale * np.abs(t) * Ea, F32, "du")


def test_norm_zero_rows_and_empty():
    """A row of zeros stays finite; no rows give zero parameter gradients."""
    g = gdr()
    x = torch.zeros(3, 2, 128, dtype=BF, device="cuda")
    w = torch.ones(128, device="cuda")
    p = g.NormProblem(x, w)
    y, dx, dw = nan(x.shape, BF), nan(x.shape, BF), nan((128,), F32)
    g.norm_fwd(p, y)
    g.norm_bwd(p, torch.ones_like(x), dx, dw, p.alloc_workspace())
    e = torch.empty(0, 128, dtype=BF, device="cuda")
    q = g.NormProblem(e, w)
    dw0 = nan((128,), F32)
    g.norm_fwd(q, torch.empty_like(e))
    g.norm_bwd(q, torch.empty_like(e), torch.empty_like(e), dw0, q.alloc_workspace())
    torch.cuda.synchronize()
    assert not y.any() and not dw.any() and not dw0.any()
    assert bool((dx.float() - 1000.0).abs().max() <= 1000 * (2.0 ** -8 + 64 * ref.U))


# ---- streams, graphs and the whole layer ----


def test_other_stream():
    """A call on another stream runs in that stream's order."""
    g = gdr()
    x, w, b, h, dy, dst = conv_inputs((500, 300), 512, 4, "bf16", "bf16", True, True, 0, 1)
    p = g.ConvProblem(x, w, g.Plan(cu_of((500, 300))), b, h)
    want = nan((800, 512), BF)
    g.conv_fwd(p, want)
    torch.cuda.synchronize()
    side, got, keep = torch.cuda.Stream(), nan((800, 512), BF), x.clone()
    x.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x.copy_(keep)
    g.conv_fwd(p, got, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def layer_pass(g, docs, H, W, seed, T_total=None):
    """Inputs of one KDA layer's core: raw projections of every token."""
    r, T = rng(seed), sum(docs)
    C = H * 128
    return dict(qkv=dev(r.standard_normal((T, 3 * C)), BF), w=dev(0.5 * r.standard_normal((3 * C, W)), BF),
                graw=dev(0.5 * r.standard_normal((T, C)), BF), a=dev(0.3 * r.standard_normal(H)), gb=dev(r.standard_normal(C)),
                beta=dev(r.standard_normal((T, H)), BF), z=dev(r.standard_normal((T, C)), BF), nw=dev(1 + 0.1 * r.standard_normal(128)))


def run_prompt(g, m, docs, H, W):
    """Convolution, gate, recurrence and head norm over a packed batch; returns y, the recurrence's and the convolution's states."""
    T, N, C = sum(docs), len(docs), H * 128
    cu = cu_of(docs)
    plan = g.Plan(cu)
    act, st = nan((T, 3 * C), BF), nan((N, W - 1, 3 * C), BF)
    g.conv_fwd(g.ConvProblem(m["qkv"], m["w"], plan), act, st)
    q, k, v = (act[:, i * C:(i + 1) * C].contiguous().view(T, H, 128) for i in range(3))
    gate = nan((T, H, 128), F32)
    g.gate_fwd(g.GateProblem(m["graw"], m["a"], m["gb"], g.GDR_GATE_SIGMOID), gate)
    prob = g.Problem(g.GDR_KDA, q, k, v, gate, m["beta"], cu, input_flags=g.GDR_IN_QK_L2NORM | g.GDR_IN_BETA_SIGMOID)
    o, ht = nan((T, H, 128), BF), nan((N, H, 128, 128), F32)
    g.kda_fwd(prob, o, ht, prob.alloc_workspace(0))
    y = nan((T, H, 128), BF)
    g.norm_fwd(g.NormProblem(o, m["nw"], m["z"].view(T, H, 128), g.GDR_ACT_SIGMOID), y)
    return y, ht, st


def test_prompt_then_tokens():
    """A layer's core over prompts and then token by token through the single-token calls equals the core over the whole
    sequences: the states handed over are the ones the prompt left.

    Both sides round q, k, v and o to bf16 at the same places; the whole-sequence side also rounds the recurrence's chunk
    products to bf16 (its stated accuracy is 1e-2 relative RMS), so the two agree to that."""
    g = gdr()
    H, W, prompts, more = 2, 4, (70, 1, 129), 5
    C, N = H * 128, len(prompts)
    whole = tuple(p + more for p in prompts)
    m = layer_pass(g, whole, H, W, 9)
    y_all, ht_all, st_all = run_prompt(g, m, whole, H, W)
    starts = cu_of(whole)[:-1]
    rows = np.concatenate([np.arange(s, s + p) for s, p in zip(starts, prompts)])
    part = {k: (t[torch.from_numpy(rows).cuda()].contiguous() if k in ("qkv", "graw", "beta", "z") else t) for k, t in m.items()}
    y0, state, conv_state = run_prompt(g, part, prompts, H, W)
    # static buffers of a serving loop, the slots of a larger pool
    pool, cpool = nan((N + 2, H, 128, 128), F32), nan((N + 2, W - 1, 3 * C), BF)
    slots = torch.tensor([3, 0, 4], dtype=torch.int32, device="cuda")
    pool[slots.long()], cpool[slots.long()] = state, conv_state
    x, act = nan((N, 3 * C), BF), nan((N, 3 * C), BF)
    graw, gate, beta = nan((N, C), BF), nan((N, H, 128), F32), nan((N, H), BF)
    z, o, y = nan((N, H, 128), BF), nan((N, H, 128), BF), nan((N, H, 128), BF)
    heads = [act[:, i * C:(i + 1) * C].unflatten(1, (H, 128)) for i in range(3)]
    cs = g.ConvStep(x, m["w"], cpool, slots)
    gp = g.GateProblem(graw, m["a"], m["gb"], g.GDR_GATE_SIGMOID)
    sp = g.StepProblem(g.GDR_KDA, *heads, gate, beta, pool, None, slots, input_flags=g.GDR_IN_QK_L2NORM | g.GDR_IN_BETA_SIGMOID)
    npb = g.NormProblem(o, m["nw"], z, g.GDR_ACT_SIGMOID)

    def token():
        g.conv_step(cs, act)
        g.gate_fwd(gp, gate)
        g.kda_step(sp, o)
        g.norm_fwd(npb, y)

    def feed(i):
        at = torch.from_numpy(starts + np.array(prompts) + i).long().cuda()
        x.copy_(m["qkv"][at])
        graw.copy_(m["graw"][at])
        beta.copy_(m["beta"][at])
        z.copy_(m["z"].view(-1, H, 128)[at])
        return at

    # the loop captured into a graph, replayed for each token with eager work between; the capture runs nothing
    saved = pool.clone(), cpool.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        feed(0)
        token()  # loads the kernels before the capture
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    pool.copy_(saved[0])
    cpool.copy_(saved[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token()
    epool, ecpool = saved[0].clone(), saved[1].clone()
    for i in range(more):
        at = feed(i)
        graph.replay()
        torch.cuda.synchronize()
        want, got = f64(y_all[at]), f64(y)
        rel = np.linalg.norm(got - want) / np.linalg.norm(want)
        assert rel <= 1.5e-2, "token %d: %.3g" % (i, rel)  # 1e-2 on either side, independent: sqrt(2) 1e-2
        # and the replay equals the eager calls on a state of their own, bit for bit
        ey = y.clone()
        keep = pool.clone(), cpool.clone()
        pool.copy_(epool)
        cpool.copy_(ecpool)
        token()
        torch.cuda.synchronize()
        assert torch.equal(ey, y) and torch.equal(keep[0][slots.long()], pool[slots.long()])
        epool, ecpool = pool.clone(), cpool.clone()
    rel = np.linalg.norm(f64(pool[slots.long()]) - f64(ht_all)) / np.linalg.norm(f64(ht_all))
    assert rel <= 1.5e-2, rel
    assert torch.equal(cpool[slots.long()], st_all)
    for free in (1, 2):
        assert bool(torch.isnan(pool[free]).all()) and bool(torch.isnan(cpool[free].float()).all())


def test_training_graph_replays():
    """Forward and backward of convolution, gate and norm captured once and replayed on changed inputs, with eager work
    between, equal the eager calls."""
    g = gdr()
    docs = (130, 1, 77)
    T, H, C, W = sum(docs), 3, 384, 4
    x, w, b, h, dy, dst = conv_inputs(docs, C, W, "bf16", "bf16", True, True, 0, 2)
    p = g.ConvProblem(x, w, g.Plan(cu_of(docs)), b, h)
    graw, a, gb = dev(rng(1).standard_normal((T, C)), BF), dev(rng(2).standard_normal(H)), dev(rng(3).standard_normal(C))
    gp = g.GateProblem(graw, a, gb)
    dg = dev(rng(4).standard_normal((T, C)))
    nw = dev(1 + 0.1 * rng(5).standard_normal(128))
    s, res = nan((T, H, 128), F32), dev(rng(6).standard_normal((T, H, 128)))
    y = nan((T, C), BF)
    npb = g.NormProblem(y.view(T, H, 128), nw, residual=res, s=s, placement=g.GDR_RES_BEFORE)
    outs = dict(st=nan((3, W - 1, C), BF), gate=nan((T, C), F32), n=nan((T, H, 128), BF), dx=nan((T, C), BF), dw=nan((C, W), F32),
                db=nan((C,), F32), ds0=nan((3, W - 1, C), BF), dgx=nan((T, C), BF), da=nan((H,), F32), dgb=nan((C,), F32),
                dres=nan((T, H, 128), F32), dn=nan((T, H, 128), BF), dnw=nan((128,), F32))
    ws = [q.alloc_workspace() for q in (p, gp, npb)]

    def step():
        g.conv_fwd(p, y, outs["st"])
        g.gate_fwd(gp, outs["gate"])
        g.norm_fwd(npb, outs["n"])
        g.norm_bwd(npb, outs["n"], outs["dn"], outs["dnw"], ws[2], dres=outs["dres"])
        g.gate_bwd(gp, dg, outs["dgx"], outs["da"], outs["dgb"], ws[1])
        g.conv_bwd(p, outs["dn"].view(T, C), dst, outs["dx"], outs["dw"], outs["db"], outs["ds0"], ws[0])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x.copy_(dev(rng(20 + i).standard_normal((T, C)), BF))
        graw.copy_(dev(rng(30 + i).standard_normal((T, C)), BF))
        for t in list(outs.values()) + [s, y]:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = {k: t.clone() for k, t in outs.items()}
        for t in list(outs.values()) + [s, y]:
            t.fill_(float("nan"))
        step()
        torch.cuda.synchronize()
        for k in outs:
            assert torch.equal(got[k], outs[k]), (i, k)


# ---- far offsets, values that must not spread, other ways to call ----


def test_offsets_past_32_bits():
    """Rows, states and outputs whose element offsets pass 2^32: the same bits as from compact buffers."""
    g = gdr()
    T, stride = 440000, 10000  # 4.4e9 elements
    wide = torch.zeros(T, stride, dtype=BF, device="cuda")
    compact = dev(rng(1).standard_normal((T, 136)), BF)
    x = wide[:, 5:141]
    x.copy_(compact)
    docs = (T - 300, 300)
    w, plan = dev(0.5 * rng(2).standard_normal((136, 4)), BF), g.Plan(cu_of(docs))
    y, want = nan((T, 136), BF), nan((T, 136), BF)
    g.conv_fwd(g.ConvProblem(x, w, plan), y)
    g.conv_fwd(g.ConvProblem(compact, w, plan), want)
    assert torch.equal(y, want)
    dx, dwant = wide[:, 200:336], nan((T, 136), BF)
    dw, dw2 = nan((136, 4), F32), nan((136, 4), F32)
    p, q = g.ConvProblem(x, w, plan), g.ConvProblem(compact, w, plan)
    g.conv_bwd(p, y, None, dx, dw, None, None, p.alloc_workspace())
    g.conv_bwd(q, want, None, dwant, dw2, None, None, q.alloc_workspace())
    assert torch.equal(dx, dwant) and torch.equal(dw, dw2)
    a = torch.zeros(1, device="cuda")
    gates, gwant = nan((T, 128), F32), nan((T, 128), F32)
    g.gate_fwd(g.GateProblem(x[:, :128], a), gates)
    g.gate_fwd(g.GateProblem(compact[:, :128].contiguous(), a), gwant)
    assert torch.equal(gates, gwant)
    nw = torch.ones(136, device="cuda")
    g.norm_fwd(g.NormProblem(x, nw), y)
    g.norm_fwd(g.NormProblem(compact, nw), want)
    assert torch.equal(y, want)
    del wide, x, dx, compact, gates, gwant, y, want, dwant, p, q
    torch.cuda.empty_cache()
    slots, hv = 5600, 48  # 4.4e9 state elements
    pool = torch.zeros(slots, hv, 128, 128, device="cuda")
    qq, k, v, gate, beta, state, _ = step_inputs("gdn", (1, 1), 16, hv, 0, 0, 3)
    pool[slots - 1], pool[7] = state[0], state[1]
    at = torch.tensor([slots - 1, 7], dtype=torch.int32, device="cuda")
    o, want = nan(v.shape, BF), nan(v.shape, BF)
    g.gdn_step(g.StepProblem(g.GDR_GDN, qq, k, v, gate, beta, pool, None, at), o)
    g.gdn_step(g.StepProblem(g.GDR_GDN, qq, k, v, gate, beta, state), want)
    assert torch.equal(o, want) and torch.equal(pool[slots - 1], state[0]) and torch.equal(pool[7], state[1])


@pytest.mark.parametrize("C,W", [(130, 4), (40, 8), (5, 2)])
def test_conv_documents_are_separate(C, W):
    """NaN and infinities in one document leave its neighbours' outputs and gradients as they were."""
    g = gdr()
    docs = (3, 70, 1, 65, 2)
    x, w, b, h, dy, dst = conv_inputs(docs, C, W, "bf16", "bf16", True, True, 0, 8)
    plan = g.Plan(cu_of(docs))

    def both():
        p = g.ConvProblem(x, w, plan, b, h)
        y, st, dx, ds0 = nan(x.shape, BF), nan(h.shape, BF), nan(x.shape, BF), nan(h.shape, BF)
        g.conv_fwd(p, y, st)
        g.conv_bwd(p, dy, dst, dx, nan((C, W), F32), nan((C,), F32), ds0, p.alloc_workspace())
        return [t.clone() for t in (y, dx, st, ds0)]

    clean = both()
    x[3:73], dy[3:73], h[1], dst[1] = float("nan"), float("inf"), float("nan"), float("nan")
    dirty = both()
    rows = torch.cat([torch.arange(3), torch.arange(73, 141)]).cuda()
    for a, b2 in zip(clean[:2], dirty[:2]):
        assert torch.equal(a[rows], b2[rows])
    for a, b2 in zip(clean[2:], dirty[2:]):
        assert torch.equal(a[[0, 2, 3, 4]], b2[[0, 2, 3, 4]])


def test_norm_infinity_stays_in_its_row():
    """An infinite value: its row follows the formula (zeros beside a NaN), the other rows and every width are untouched by
    lanes that read a neighbour's value."""
    g = gdr()
    for D in (129, 40, 2050):
        x = dev(rng(D).standard_normal((9, D)))
        clean, y = nan((9, D), F32), nan((9, D), F32)
        g.norm_fwd(g.NormProblem(x, None), clean)
        x[4, D - 2] = float("inf")
        g.norm_fwd(g.NormProblem(x, None), y)
        torch.cuda.synchronize()
        others = [r for r in range(9) if r != 4]
        assert torch.equal(y[others], clean[others])
        row = y[4].tolist()
        assert row[D - 2] != row[D - 2] and all(v == 0 for i, v in enumerate(row) if i != D - 2)


def test_step_extreme_gates_and_nan_padding():
    """g = -inf clears the state before the write, g = 0 keeps it; NaN operands of a skipped sequence reach nothing."""
    g = gdr()
    q, k, v, gate, beta, state, _ = step_inputs("kda", (1, 1, 1), 1, 1, 0, 0, 4)
    gate[0], gate[1] = -float("inf"), 0.0
    for t in (q, k, v, gate):
        t[2] = float("nan")
    slots = torch.tensor([0, 1, -1], dtype=torch.int32, device="cuda")
    before = state.clone()
    o = nan(v.shape, BF)
    g.kda_step(g.StepProblem(g.GDR_KDA, q, k, v, gate, beta, state, None, slots), o)
    torch.cuda.synchronize()
    ro, Eo, rs, Es = ref.step(f64(q[:2]), f64(k[:2]), f64(v[:2]), f64(gate[:2]), f64(beta[:2]), f64(before), (1, 1), [0, 1],
                              128 ** -0.5, False, False)
    ref.close(o[:2], ro, Eo, BF, "o")
    ref.close(state, rs, Es, F32, "state")
    assert bool(torch.isnan(o[2].float()).all())


def test_recurrence_state_feeds_the_step():
    """ht of the chunked forward, taken as a state pool as it is, continues a sequence; a Problem serves as a convolution's
    plan; both variants."""
    g = gdr()
    for variant, hqk, hv in (("kda", 2, 2), ("gdn", 1, 3)):
        from chunked_gated_delta_14_amd import workloads
        from gpu_runner import to_dev

        docs = (65, 3)
        d = to_dev(workloads.make_inputs(workloads.custom(variant, (66, 4), hqk, hv, True, seed=6)))
        rows = torch.cat([torch.arange(65), torch.arange(66, 69)]).cuda()
        last = torch.tensor([65, 69]).cuda()
        code = g.GDR_KDA if variant == "kda" else g.GDR_GDN
        names = ("q", "k", "v", "g", "beta")
        prob = g.Problem(code, *(d[n][rows].contiguous() for n in names), cu_of(docs), d["h0"])
        o, ht = nan((68, hv, 128), BF), nan((2, hv, 128, 128), F32)
        (g.kda_fwd if variant == "kda" else g.gdn_fwd)(prob, o, ht, prob.alloc_workspace(0))
        o1 = nan((2, hv, 128), BF)
        (g.kda_step if variant == "kda" else g.gdn_step)(
            g.StepProblem(code, *(d[n][last].contiguous() for n in names), ht), o1)
        full = g.Problem(code, *(d[n] for n in names), d["cu_seqlens"], d["h0"])
        ofull, htfull = nan((70, hv, 128), BF), nan((2, hv, 128, 128), F32)
        (g.kda_fwd if variant == "kda" else g.gdn_fwd)(full, ofull, htfull, full.alloc_workspace(0))
        torch.cuda.synchronize()
        for a, b in ((o1, ofull[last]), (ht, htfull)):  # each side within the recurrence's 1e-2
            rel = np.linalg.norm(f64(a) - f64(b)) / np.linalg.norm(f64(b))
            assert rel <= 1.5e-2, (variant, rel)
        x = d["v"].view(70, -1)
        y, want = nan(x.shape, BF), nan(x.shape, BF)
        w = dev(rng(1).standard_normal((x.shape[1], 4)), BF)
        g.conv_fwd(g.ConvProblem(x, w, full), y)
        g.conv_fwd(g.ConvProblem(x, w, g.Plan(cu_of((66, 4)))), want)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_gpu_refusals_write_nothing():
    """Calls that the binding or the library refuses leave their outputs as they were."""
    g = gdr()
    x = torch.ones(8, 32, dtype=BF, device="cuda")
    w = torch.ones(32, 4, dtype=BF, device="cuda")
    p = g.ConvProblem(x, w, g.Plan([0, 8]))
    y = nan((8, 32), BF)
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    for call in (lambda: g.conv_fwd(p, y.float()), lambda: g.conv_fwd(p, y[:4]), lambda: g.conv_fwd(p, y.cpu()),
                 lambda: g.conv_fwd(p, nan((32, 8), BF).t()), lambda: g.conv_bwd(p, x, None, y, nan((32, 4), F32), None, None, small[1:]),
                 lambda: g.ConvProblem(x, w, g.Plan([0, 7])), lambda: g.ConvProblem(x, w.t(), g.Plan([0, 8])),
                 lambda: g.ConvProblem(x, w[:, :1], g.Plan([0, 8])) and g.conv_fwd(g.ConvProblem(x, w[:, :1].contiguous(), g.Plan([0, 8])), y),
                 lambda: g.ConvStep(x, w, torch.ones(4, 3, 32, dtype=BF, device="cuda"), torch.zeros(8, dtype=torch.int64, device="cuda")),
                 lambda: g.GateProblem(x.half(), torch.ones(32, device="cuda")),
                 lambda: g.NormProblem(x, None, residual=x), lambda: g.NormProblem(x, None, residual=x, s=x, placement=g.GDR_RES_BEFORE),
                 lambda: g.gate_fwd(g.GateProblem(x, torch.ones(32, device="cuda"), floor=-9.0), nan((8, 32), F32))):
        with pytest.raises(g.GdrError):
            call()
    torch.cuda.synchronize()
    assert bool(torch.isnan(y.float()).all())


@pytest.mark.parametrize("variant", ["kda", "gdn"])
def test_training_step_of_a_layer(variant):
    """A layer's core forwards and backwards through the library (convolution, gate, recurrence with its activations, head
    norm with gate) against the fp64 references and oracle, chained.

    The reference rounds q, k, v, o and their gradients to bf16 where the library stores them.  What is left is the
    recurrence's own stated accuracy (1e-2 relative RMS for dq, dk and dv, 2e-2 for dg and dbeta), which reaches the
    projections' and parameters' gradients through linear maps: twice it is allowed, since an error may align with a
    map's larger directions better than the gradient does, and half a bf16 step (2^-8) for the last rounding.  dz
    depends on o alone (1e-2)."""
    import oracle

    g = gdr()
    docs, hqk, hv, W = (70, 1, 129), 1, 2, 4
    if variant == "kda":
        hqk = hv
    T, cu = sum(docs), cu_of(docs)
    cq, cv, D = hqk * 128, hv * 128, 128 if variant == "kda" else 1
    C = 2 * cq + cv
    r = rng(12)
    qkv, w = dev(r.standard_normal((T, C)), BF), dev(0.5 * r.standard_normal((C, W)), BF)
    graw, a, gb = dev(0.5 * r.standard_normal((T, hv * D)), BF), dev(0.3 * r.standard_normal(hv)), dev(r.standard_normal(hv * D))
    beta = dev(r.standard_normal((T, hv)), BF if variant == "kda" else F32)
    z, nw = dev(r.standard_normal((T, hv, 128)), BF), dev(1 + 0.1 * r.standard_normal(128))
    dy = dev(r.standard_normal((T, hv, 128)), BF)
    plan = g.Plan(cu)
    act = nan((T, C), BF)
    cp = g.ConvProblem(qkv, w, plan)
    g.conv_fwd(cp, act)
    cuts = (0, cq, 2 * cq, C)
    q, k, v = (act[:, i:j].contiguous().view(T, -1, 128) for i, j in zip(cuts, cuts[1:]))
    gate = nan((T, hv, 128) if D > 1 else (T, hv), F32)
    gp = g.GateProblem(graw, a, gb, g.GDR_GATE_SIGMOID)
    g.gate_fwd(gp, gate)
    prob = g.Problem(g.GDR_KDA if variant == "kda" else g.GDR_GDN, q, k, v, gate, beta, cu,
                     input_flags=g.GDR_IN_QK_L2NORM | g.GDR_IN_BETA_SIGMOID)
    ws, o = prob.alloc_workspace(), nan((T, hv, 128), BF)
    (g.kda_fwd if variant == "kda" else g.gdn_fwd)(prob, o, None, ws, g.GDR_FWD_SAVE)
    y, npb = nan(o.shape, BF), g.NormProblem(o, nw, z, g.GDR_ACT_SILU)
    g.norm_fwd(npb, y)
    do, dz, dnw = nan(o.shape, BF), nan(o.shape, BF), nan((128,), F32)
    g.norm_bwd(npb, dy, do, dnw, npb.alloc_workspace(), dgate=dz)
    dq, dk, dv = nan(q.shape, BF), nan(k.shape, BF), nan(v.shape, BF)
    dg, dbeta = nan(gate.shape, F32), torch.empty_like(beta)
    (g.kda_bwd if variant == "kda" else g.gdn_bwd)(prob, do, None, dq, dk, dv, dg, dbeta, None, ws)
    dgraw, da, dgb = nan((T, hv * D), BF), nan((hv,), F32), nan((hv * D,), F32)
    g.gate_bwd(gp, dg, dgraw, da, dgb, gp.alloc_workspace())
    dact = torch.cat([dq.view(T, -1), dk.view(T, -1), dv.view(T, -1)], 1)
    dqkv, dw = nan((T, C), BF), nan((C, W), F32)
    g.conv_bwd(cp, dact, None, dqkv, dw, None, None, cp.alloc_workspace())
    torch.cuda.synchronize()

    def bf(x):
        return torch.from_numpy(np.ascontiguousarray(x)).to(BF).double().numpy()

    f = ref.conv(f64(qkv), f64(w), 0.0 * f64(w)[:, 0], None, docs, True)
    rq, rk, rv = (bf(f["y"][:, i:j].reshape(T, -1, 128)) for i, j in zip(cuts, cuts[1:]))
    rg = ref.gate(f64(graw).reshape(T, hv, D), f64(a), f64(gb).reshape(hv, D), "sigmoid", -5.0)[0]
    rg = rg if D > 1 else rg[..., 0]
    flags = dict(qk_l2norm=True, beta_sigmoid=True)
    ro = bf(oracle.forward_act(rq, rk, rv, rg, f64(beta), cu, None, **flags)[0])
    n = ref.norm_grad(ro, f64(nw), f64(z), f64(dy), None, "none", "silu", 1.0, 1e-6)
    b = oracle.backward_act(rq, rk, rv, rg, f64(beta), cu, bf(n["dx"]), None, None, **flags)
    gg = ref.gate_grad(f64(graw).reshape(T, hv, D), f64(a), f64(gb).reshape(hv, D), "sigmoid", -5.0, b["dg"].reshape(T, hv, D))
    rdact = np.concatenate([bf(b[x]).reshape(T, -1) for x in ("dq", "dk", "dv")], 1)
    c = ref.conv_grad(f, f64(qkv), f64(w), docs, rdact, None, True)
    half = 2.0 ** -8
    for name, got, want, lim in (("y", y, ref.norm(ro, f64(nw), f64(z), None, "none", "silu", 1.0, 1e-6)["y"], 2e-2 + half),
                                 ("dz", dz, n["dz"], 2e-2 + half), ("dnw", dnw, n["dw"], 2e-2), ("dqkv", dqkv, c["dx"], 2e-2 + half),
                                 ("dw", dw, c["dw"], 2e-2), ("dgraw", dgraw, gg["dx"].reshape(T, -1), 4e-2 + half), ("da", da, gg["da"], 4e-2),
                                 ("dgb", dgb, gg["db"].reshape(-1), 4e-2), ("dbeta", dbeta, b["dbeta"], 4e-2 + half)):
        got = f64(got)
        rel = np.linalg.norm(got - want) / np.linalg.norm(want)
        print("[layer] %s %s %.2e" % (variant, name, rel), flush=True)
        assert rel <= lim, "%s: %.3g" % (name, rel)
