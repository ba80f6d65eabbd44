"""GPU tests of the layer operators where a value is easily lost: gates far from zero, decay rates past fp32's range, sums
over many passes of a worker.  References in fp64, bounds counted in u = 2^-24 as in layer_ref.py."""
import numpy as np
import pytest
import torch

import layer_ref as ref
from test_gpu_layer import BF, DT, F32, cu_of, dev, f64, gdr, nan, rng

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("place", ["none", "before", "after"])
@pytest.mark.parametrize("D,dt", [(5, "f32"), (64, "f32"), (64, "bf16"), (3000, "f32"), (7000, "bf16"), (16000, "bf16")])
def test_norm_gate_far_from_zero(D, dt, place):
    """dgate of a sigmoid gate follows s (1 - s) to a few roundings of itself however far z lies: 1 - s, taken from a
    rounded s, would be off by u / (1 - s), all of it from z = 17 on.

    e^-z: 2 (exp2), 2 more roundings, and with bf16 rows the argument's, 1.5 |z|; s: e's and 3; 1 - s: e's, s's and 1;
    their product 1; the row's rs at most 16 (the lanes' and wavefronts' additions halved, and rsq); four more products."""
    g, r = gdr(), rng(D + len(place))
    shape, alpha = (9, 1, D), 0.5 if place != "none" else 1.0
    dtype = DT[dt]
    print("[case] far gates", D, dt, place, flush=True)
    x, dy = dev(r.standard_normal(shape), dtype), dev(r.standard_normal(shape), dtype)
    z = dev(r.uniform(-40, 40, shape), dtype)
    w = dev(1 + 0.2 * r.standard_normal(D))
    code = {"none": g.GDR_RES_NONE, "before": g.GDR_RES_BEFORE, "after": g.GDR_RES_AFTER}[place]
    if place == "before":
        p = g.NormProblem(None, w, z, g.GDR_ACT_SIGMOID, s=x, placement=code, scale=alpha, dtype=dtype)
    else:
        p = g.NormProblem(x, w, z, g.GDR_ACT_SIGMOID, residual=x if place == "after" else None, placement=code, scale=alpha)
    dx, dz, dw = nan(shape, dtype), nan(shape, dtype), nan((D,), F32)
    dres = nan(shape, dtype) if place == "before" else None
    g.norm_bwd(p, dy, dx, dw, p.alloc_workspace(), dgate=dz, dres=dres)
    torch.cuda.synchronize()
    u, zz = f64(x), f64(z)
    n = u / np.sqrt((u * u).mean(-1, keepdims=True) + float(np.float32(1e-6)))
    want = f64(dy) * (alpha if place == "after" else 1.0) * f64(w) * n * ref.sig(zz) * ref.sig(-zz)
    e = 4 + (1.5 * np.abs(zz) if dt == "bf16" else 0)
    ref.close(dz, want, np.abs(want) * ((e + 3) + (2 * e + 4) + 1 + 16 + 4), dtype, "dz")


@pytest.mark.parametrize("D", [1, 128])
@pytest.mark.parametrize("kind", ["softplus", "sigmoid"])
def test_gate_rates_past_the_range(kind, D):
    """e^a near and past fp32's largest value: the floor (softplus), or a step at u = 0 (sigmoid), and no slope beside it."""
    g = gdr()
    a = torch.tensor([88.0, 88.5, 89.0, 300.0, float("inf")], device="cuda")
    u = torch.tensor([-50.0, -1.0, -1e-6, 0.0, 1e-6, 3.0, 40.0], device="cuda")
    H, T = len(a), len(u)
    x = u[:, None].expand(T, H * D).contiguous()
    print("[case] gate rates", kind, D, flush=True)
    p = g.GateProblem(x, a, None, g.GDR_GATE_SOFTPLUS if kind == "softplus" else g.GDR_GATE_SIGMOID, -5.0)
    out, dx, da, db = nan((T, H * D), F32), nan((T, H * D), F32), nan((H,), F32), nan((H * D,), F32)
    g.gate_fwd(p, out)
    dg = torch.ones(T, H * D, device="cuda")
    dg[3] = 0.0 if kind == "sigmoid" else 1.0  # the step itself: a slope of -5 A / 4, past the range
    g.gate_bwd(p, dg, dx, da, db, p.alloc_workspace())
    torch.cuda.synchronize()
    want = torch.full((T,), -5.0) if kind == "softplus" else torch.tensor([0.0, 0.0, 0.0, -2.5, -5.0, -5.0, -5.0])
    assert torch.equal(out.cpu(), want[:, None].expand(T, H * D)), out
    for t in (dx, da, db):
        assert not t.any(), t


# ---- workers that make several passes ----
#
# Small whole numbers, for which every product and every partial sum is exact in fp32 (|sum| < 2^24), so the outputs equal
# the definition's bit for bit: a row dropped, repeated or given to a neighbour shows as a difference of whole units.  The
# activations stand at 0, where the sigmoid is 1/2 and its slope 1/4.


def ints(r, shape, most, dtype=F32, step=1):
    gen = torch.Generator("cuda").manual_seed(int(r.integers(1 << 31)))
    return (step * torch.randint(-most, most + 1, tuple(shape), generator=gen, device="cuda", dtype=torch.int32)).to(dtype)


def lanes(groups):
    """(threads of a row, rows side by side, blocks of a row) of a row of `groups` thread groups."""
    waves = (groups + 63) // 64
    if groups * 5 >= waves * 64 * 4:
        k = next(k for k in (4, 3, 2, 1) if waves % k == 0)
        lx, nchb = 64 * k, waves // k
    else:
        nchb = (groups + 255) // 256
        lx = (groups + nchb - 1) // nchb
    return lx, max(1, 256 // lx), nchb


def workers(rows, groups, target):
    lx, ly, nchb = lanes(groups)
    n = min(rows, max(1, target // (nchb * lx)))
    return (n + ly - 1) // ly * ly, ly


def conv_workers(n_chunks, C, W):
    """Workers of the convolution's backward over runs of 64 tokens; the workspace's size says the same."""
    n, ly = workers(n_chunks, (C + 3) // 4 if C >= 4 else C, 131072)
    assert gdr().conv_workspace_bytes(n_chunks, C, W, 0) == (n // ly * (W + 1) * C * 4 + 255) // 256 * 256
    return n, ly


LONG = [
    # docs, C, W, dtype, pad
    ((20011, 7, 0, 31250), 2048, 4, "bf16", 0),
    ((5000, 65, 4000), 12288, 3, "bf16", 0),
    ((700001, 3, 310000), 100, 4, "bf16", 5),
    ((40001, 39300), 1028, 2, "f32", 3),
    ((5000011, 3500000), 3, 8, "bf16", 0),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "C%d_W%d_%s" % c[1:4])
def test_conv_of_many_runs_is_exact(case):
    docs, C, W, dt, pad = case
    g, r, dtype = gdr(), rng(C), DT[dt]
    T, N = sum(docs), len(docs)
    plan = g.Plan(cu_of(docs))
    assert plan.n_chunks >= 3 * conv_workers(plan.n_chunks, C, W)[0], "a worker takes fewer than three runs"
    print("[case] long conv", case, flush=True)

    def rows(most):
        wide = ints(r, (T, C + pad), most, dtype)
        return wide[:, :C]

    x, dy = rows(3), rows(3)
    w, b = ints(r, (C, W), 2, dtype), ints(r, (C,), 3, dtype)
    s0, dst = ints(r, (N, W - 1, C), 3, dtype), ints(r, (N, W - 1, C), 3, dtype)
    p = g.ConvProblem(x, w, plan, b, s0, g.GDR_ACT_NONE)
    y, st = nan((T, C), dtype, pad), nan((N, W - 1, C), dtype)
    dx, ds0, dw, db = nan((T, C), dtype, pad), nan((N, W - 1, C), dtype), nan((C, W), F32), nan((C,), F32)
    g.conv_fwd(p, y, st)
    g.conv_bwd(p, dy, dst, dx, dw, db, ds0, p.alloc_workspace().fill_(0xFF))
    torch.cuda.synchronize()
    want_dw, want_db = torch.zeros(C, W, dtype=torch.float64, device="cuda"), torch.zeros(C, dtype=torch.float64, device="cuda")
    t0, wf = 0, w.float()
    for n, L in enumerate(docs):
        X, d = torch.cat([s0[n].float(), x[t0:t0 + L].float()]), dy[t0:t0 + L].float()
        z, dX = b.float().expand(L, C).clone(), torch.zeros_like(X)
        for i in range(W):
            z += wf[:, i] * X[i:i + L]
            dX[i:i + L] += d * wf[:, i]
            want_dw[:, i] += (d * X[i:i + L]).sum(0, dtype=torch.float64)
        want_db += d.sum(0, dtype=torch.float64)
        dX[L:] += dst[n].float()
        assert torch.equal(y[t0:t0 + L].float(), z) and torch.equal(st[n].float(), X[L:]), "forward, document %d" % n
        assert torch.equal(dx[t0:t0 + L].float(), dX[W - 1:]) and torch.equal(ds0[n].float(), dX[:W - 1]), "backward, document %d" % n
        t0 += L
    assert torch.equal(dw.double(), want_dw) and torch.equal(db.double(), want_db)


def test_conv_of_many_runs_with_silu():
    """The same loop with the activation, a few channels against the fp64 reference.  The parameter sums are allowed the
    roundings of their real depth (a worker's rows, the block's sets, the blocks' partial rows), less than one average
    term in all, so a lost or repeated row does not hide in them."""
    docs, C, W = (20011, 7, 0, 31250), 2048, 4
    g, r = gdr(), rng(77)
    T, plan = sum(docs), g.Plan(cu_of(docs))
    n, ly = conv_workers(plan.n_chunks, C, W)
    per = -(-plan.n_chunks // n)  # runs of a worker
    assert per >= 3
    depth = 64 * per + int(np.ceil(np.log2(ly))) + -(-(n // ly) // 32) + 16 + 4
    x, dy = (torch.randn(T, C, generator=torch.Generator("cuda").manual_seed(i), device="cuda").to(BF) for i in (1, 2))
    w, b = dev(0.5 * r.standard_normal((C, W)), BF), dev(0.2 * r.standard_normal(C), BF)
    p = g.ConvProblem(x, w, plan, b)
    print("[case] long conv with SiLU", flush=True)
    y, dx, dw, db = nan((T, C), BF), nan((T, C), BF), nan((C, W), F32), nan((C,), F32)
    g.conv_fwd(p, y)
    g.conv_bwd(p, dy, None, dx, dw, db, None, p.alloc_workspace().fill_(0xFF))
    torch.cuda.synchronize()
    ch = [0, 3, 1021, 1024, 2047]
    X, D = f64(x[:, ch]), f64(dy[:, ch])
    f = ref.conv(X, f64(w[ch]), f64(b[ch]), None, docs, True)
    d = ref.conv_grad(f, X, f64(w[ch]), docs, D, None, True)
    ref.close(y[:, ch], f["y"], f["Ey"], BF, "y")
    ref.close(dx[:, ch], d["dx"], d["Edx"], BF, "dx")
    s = ref.sig(f["z"])
    dz = np.abs(D * s * (1 + f["z"] * (1 - s)))
    Sw = np.zeros((len(ch), W))  # the sums of the terms' magnitudes, for which layer_ref allows T + 4 roundings
    t0 = 0
    for k, L in enumerate(docs):
        for i in range(W):
            Sw[:, i] += (dz[t0:t0 + L] * np.abs(f["ext"][k][i:i + L])).sum(0)
        t0 += L
    Sb = dz.sum(0)
    for got, want, E, S in ((dw[ch], d["dw"], d["Edw"], Sw), (db[ch], d["db"], d["Edb"], Sb)):
        assert (depth * ref.U * S < S / T).all()
        ref.close(got, want, E - (T + 4) * S + depth * S, F32, "parameter gradient")


@pytest.mark.parametrize("T,H,D,dt", [(30011, 16, 128, "bf16"), (98321, 4, 128, "bf16"), (1100011, 3, 1, "f32"), (524669, 48, 1, "bf16")])
def test_gate_gradient_of_many_passes_is_exact(T, H, D, dt):
    """At u = 0, where the sigmoid gate's slope is -5 / 4."""
    g, r, dtype = gdr(), rng(T), DT[dt]
    C = H * D
    groups = (C + 7) // 8 if C >= 8 else C
    n, ly = workers((T + 7) // 8, groups, 262144 if lanes(groups)[0] < 64 else 131072)
    assert T >= 3 * 4 * n, "fewer than three passes"
    print("[case] long gate", T, H, D, dt, flush=True)
    row = dev(r.standard_normal(C), dtype)
    p = g.GateProblem(row.expand(T, C).contiguous(), torch.zeros(H, device="cuda"), -row.float(), g.GDR_GATE_SIGMOID, -5.0)
    dg = ints(r, (T, C), 3, step=4)
    out, dx, da, db = nan((T, C), F32), nan((T, C), dtype), nan((H,), F32), nan((C,), F32)
    g.gate_fwd(p, out)
    g.gate_bwd(p, dg, dx, da, db, p.alloc_workspace().fill_(0xFF))
    torch.cuda.synchronize()
    assert bool((out == -2.5).all())
    assert torch.equal(dx.float(), -1.25 * dg)
    assert torch.equal(db.double(), -1.25 * dg.sum(0, dtype=torch.float64)) and not da.any()


def test_gate_gradient_takes_every_row_once():
    """da and dbias where one row alone counts for each head, another for each: the row's own slopes, not zero or twice them."""
    g, r, T = gdr(), rng(8), 3000
    n, _ = workers((T + 7) // 8, T // 8, 131072)
    assert T > 2 * 4 * n
    x, a = r.standard_normal((T, T)), 0.3 * r.standard_normal(T)
    xs, at, row = dev(x), dev(a), torch.from_numpy(r.permutation(T)).cuda()
    head = torch.arange(T, device="cuda")
    dg = torch.zeros(T, T, device="cuda")
    dg[row, head] = 1.0
    p = g.GateProblem(xs, at, None, g.GDR_GATE_SOFTPLUS, -8.0)
    print("[case] one row for each head", flush=True)
    dx, da, db = nan((T, T), F32), nan((T,), F32), nan((T,), F32)
    g.gate_bwd(p, dg, dx, da, db, p.alloc_workspace().fill_(0xFF))
    torch.cuda.synchronize()
    u, A = f64(xs[row, head]), np.exp(f64(at))
    raw, slope = -A * np.logaddexp(u, 0), -A * ref.sig(u)
    live = raw >= -8.0
    assert live.sum() > T * 0.9 and not (np.abs(raw + 8.0) < 1e-4).any()
    la = 1.5 * np.abs(f64(at))  # layer_ref's counts for A, softplus and sigma; u = x is exact
    ref.close(da, np.where(live, raw, 0), np.abs(raw) * (la + 20), F32, "da")
    ref.close(db, np.where(live, slope, 0), np.abs(slope) * (la + 20), F32, "dbias")
    assert torch.equal(dx[row, head], db) and int((dx != 0).sum()) == int((db != 0).sum())


@pytest.mark.parametrize("T,H,D,dt,kind", [(98321, 16, 128, "bf16", "softplus"), (17000003, 3, 1, "f32", "sigmoid")])
def test_gate_forward_of_many_passes(T, H, D, dt, kind):
    """Every row, in torch's fp64 on the GPU, within layer_ref's bound."""
    g, dtype, C = gdr(), DT[dt], H * D
    n, _ = workers((T + 3) // 4, (C + 3) // 4 if C > 3 else C, 1 << 22)
    assert T >= 3 * 4 * n, "fewer than three passes"
    x = torch.randn(T, C, generator=torch.Generator("cuda").manual_seed(3), device="cuda").to(dtype)
    a, b = dev(0.3 * rng(1).standard_normal(H)), dev(rng(2).standard_normal(C))
    print("[case] gate forward of many passes", T, H, D, dt, flush=True)
    out = nan((T, C), F32)
    g.gate_fwd(g.GateProblem(x, a, b, g.GDR_GATE_SOFTPLUS if kind == "softplus" else g.GDR_GATE_SIGMOID, -5.0), out)
    A = a.double().exp().repeat_interleave(D)
    la = 1.5 * A.log().abs()
    for lo in range(0, T, 1 << 22 if D == 1 else 1 << 14):
        rows = slice(lo, lo + (1 << 22 if D == 1 else 1 << 14))
        u = x[rows].double() + b.double()
        s = torch.sigmoid(u if kind == "softplus" else A * u)
        if kind == "softplus":
            raw = -A * torch.logaddexp(u, torch.zeros_like(u))
            want, E = raw.clamp_min(-5.0), A * s * u.abs() + raw.abs() * (la + 20)
        else:
            want, E = -5.0 * s, 5.0 * (s * (1 - s) * (A * u).abs() * (la + 8) + s * 8)
        tol = E * ref.U + ref.U * (want.abs() + E * ref.U)
        bad = ~((out[rows].double() - want).abs() <= tol)
        assert not bad.any(), (lo, bad.nonzero()[:3])


@pytest.mark.parametrize("T,H,D,dt,rdt,place,gated", [
    (40001, 3, 128, "bf16", "bf16", "none", True),
    (100003, 1, 8, "f32", "f32", "none", False),
    (33337, 3, 64, "bf16", "f32", "after", True),
    (3001, 1, 2048, "bf16", "f32", "before", False),
    (2001, 1, 4096, "f32", "f32", "after", True),
    (800, 1, 16384, "bf16", "bf16", "before", True),
])
def test_norm_of_many_passes_is_exact(T, H, D, dt, rdt, place, gated):
    """Rows of ones of either sign and eps = 0: the norm is the row itself; z = 0, where a sigmoid gate is 1/2, its slope 1/4."""
    g, r, dtype, rtype = gdr(), rng(T), DT[dt], DT[rdt]
    shape, alpha = (T, H, D), 0.5 if place != "none" else 1.0
    vec = 8 if dt == "bf16" else 4
    lpr = next(t for t in (16, 32, 64, 128, 192, 256, 512, 768, 1024, 2048) if D <= t * vec)
    assert T * H >= 3 * (2048 * (256 // lpr) if lpr <= 64 else 256), "fewer than three passes"
    print("[case] long norm", T, H, D, dt, place, flush=True)
    u = torch.where(torch.rand(shape, generator=torch.Generator("cuda").manual_seed(5), device="cuda") < 0.5, -1.0, 1.0)
    w = torch.from_numpy(r.integers(1, 4, D)).float().cuda()
    x, z = u.to(dtype), torch.zeros(shape, dtype=dtype, device="cuda") if gated else None
    ydt = rtype if place == "after" else dtype
    dy = ints(r, shape, 3, ydt, step=4)
    res = (0.5 * u).to(rtype) if place == "before" else ints(r, shape, 3, rtype) if place == "after" else None
    s = nan(shape, rtype) if place == "before" else None
    ds = ints(r, shape, 3, rtype) if place == "before" else None
    code = {"none": g.GDR_RES_NONE, "before": g.GDR_RES_BEFORE, "after": g.GDR_RES_AFTER}[place]
    p = g.NormProblem(x, w, z, g.GDR_ACT_SIGMOID if gated else g.GDR_ACT_NONE, res, s, code, alpha, 0.0)
    y, dx, dw = nan(shape, ydt), nan(shape, dtype), nan((D,), F32)
    dz = nan(shape, dtype) if gated else None
    dres = nan(shape, rtype) if place == "before" else None
    g.norm_fwd(p, y)
    g.norm_bwd(p, dy, dx, dw, p.alloc_workspace().fill_(0xFF), dgate=dz, ds=ds, dres=dres)
    torch.cuda.synchronize()
    act = 0.5 if gated else 1.0
    n = u * w * act
    if place == "before":
        assert torch.equal(s.float(), u)
    assert torch.equal(y, (res.float() + alpha * n if place == "after" else n).to(ydt))
    t = dy.float() * (alpha if place == "after" else 1.0)
    assert torch.equal(dw.double(), (t * act * u).sum((0, 1), dtype=torch.float64))
    if gated:
        assert torch.equal(dz, (0.25 * t * w * u).to(dtype))
    v = t * act * w
    d = v - u * (v * u).sum(-1, keepdim=True, dtype=torch.float64).float() / D  # all of it exact: multiples of act / D
    if place == "before":
        d = d + ds.float()
        assert torch.equal(dres, d.to(rtype))
        d = alpha * d
    assert torch.equal(dx, d.to(dtype))


def test_partial_rows_are_added_without_loss():
    """The workers' partial sums may differ by more than fp32 holds: one of 2^24 beside 198 of 1, each exact in its run of
    64 tokens, add up to what fp32 holds, 2^24 + 198."""
    g, C, runs = gdr(), 2048, 200
    assert conv_workers(runs, C, 2) == (runs, 1)  # a run for each worker, a partial row for each run
    T = 64 * runs
    dy = torch.zeros(T, C, device="cuda")
    dy[37::64] = 1.0
    dy[64 * 77 + 37], dy[64 * 5 + 37] = 2.0 ** 24, 0.0
    p = g.ConvProblem(torch.ones(T, C, device="cuda"), torch.zeros(C, 2, device="cuda"), g.Plan([0, T]), None, None, g.GDR_ACT_NONE)
    print("[case] partial rows", flush=True)
    dx, dw, db = nan((T, C), F32), nan((C, 2), F32), nan((C,), F32)
    g.conv_bwd(p, dy, None, dx, dw, db, None, p.alloc_workspace())
    torch.cuda.synchronize()
    assert bool((db == 2.0 ** 24 + 198).all()) and bool((dw == 2.0 ** 24 + 198).all())


@pytest.mark.parametrize("C,W,dt", [(24, 4, "bf16"), (5, 8, "f32"), (260, 2, "bf16")])
def test_conv_of_tiny_documents_is_exact(C, W, dt):
    """Twenty thousand documents of 0 to 5 tokens, most of them shorter than the history: whole numbers again."""
    g, r, dtype, N, H = gdr(), rng(C), DT[dt], 20011, W - 1
    lens = r.integers(0, 6, N)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    x, dy, w, b = ints(r, (T, C), 3, dtype), ints(r, (T, C), 3, dtype), ints(r, (C, W), 2, dtype), ints(r, (C,), 3, dtype)
    s0, dst = ints(r, (N, H, C), 3, dtype), ints(r, (N, H, C), 3, dtype)
    print("[case] tiny documents", C, W, dt, flush=True)
    p = g.ConvProblem(x, w, g.Plan(cu), b, s0, g.GDR_ACT_NONE)
    y, st, dx, ds0 = nan((T, C), dtype), nan((N, H, C), dtype), nan((T, C), dtype), nan((N, H, C), dtype)
    dw, db = nan((C, W), F32), nan((C,), F32)
    g.conv_fwd(p, y, st)
    g.conv_bwd(p, dy, dst, dx, dw, db, ds0, p.alloc_workspace().fill_(0xFF))
    torch.cuda.synchronize()
    # all documents laid out one after the other, each with its history before it
    L = torch.from_numpy(lens).cuda()
    start = torch.from_numpy(cu[:-1]).cuda().long() + torch.arange(N, device="cuda") * H  # of a document's history
    at = torch.arange(T, device="cuda") + torch.repeat_interleave(torch.arange(N, device="cuda"), L) * H + H  # of a token
    hist = start[:, None] + torch.arange(H, device="cuda")
    X = torch.zeros(T + N * H, C, device="cuda")
    X[at], X[hist] = x.float(), s0.float()
    dX, wf, d = torch.zeros_like(X), w.float(), dy.float()
    z = b.float().expand(T, C).clone()
    for i in range(W):
        z += wf[:, i] * X[at - H + i]
        dX[at - H + i] += d * wf[:, i]  # the rows of one tap are distinct
        assert torch.equal(dw[:, i].double(), (d * X[at - H + i]).sum(0, dtype=torch.float64)), i
    tail = hist + L[:, None]
    dX[tail] += dst.float()
    assert torch.equal(y.float(), z) and torch.equal(st.float(), X[tail])
    assert torch.equal(dx.float(), dX[at]) and torch.equal(ds0.float(), dX[hist])
    assert torch.equal(db.double(), d.sum(0, dtype=torch.float64))


def test_widest_rows():
    """Channels, heads and states at the largest counts that the checks take."""
    g, r = gdr(), rng(4)
    C, W, docs = 1 << 24, 6, (2, 0, 1)  # 32 (W + 1) C just below 2^32
    T = sum(docs)
    x, dy, w = ints(r, (T, C), 3), ints(r, (T, C), 3), ints(r, (C, W), 2)
    print("[case] widest convolution", flush=True)
    p = g.ConvProblem(x, w, g.Plan(cu_of(docs)), None, None, g.GDR_ACT_NONE)
    y, dx, dw, db = nan((T, C), F32), nan((T, C), F32), nan((C, W), F32), nan((C,), F32)
    g.conv_fwd(p, y)
    g.conv_bwd(p, dy, None, dx, dw, db, None, p.alloc_workspace())
    torch.cuda.synchronize()
    assert torch.equal(y[0], w[:, 5] * x[0]) and torch.equal(y[2], w[:, 5] * x[2])
    assert torch.equal(y[1], w[:, 5] * x[1] + w[:, 4] * x[0])
    assert torch.equal(dx[0], w[:, 5] * dy[0] + w[:, 4] * dy[1]) and torch.equal(dx[1:], w[:, 5] * dy[1:])
    assert torch.equal(dw[:, 5], (x * dy).sum(0)) and torch.equal(dw[:, 4], x[0] * dy[1]) and not dw[:, :4].any()
    assert torch.equal(db, dy.sum(0))
    del x, dy, w, p, y, dx, dw, db
    H, T = 65536, 5
    print("[case] most gate heads", flush=True)
    row = torch.randn(H * 128, device="cuda").to(BF)
    dg = ints(r, (T, H * 128), 3, step=4)
    q = g.GateProblem(row.expand(T, -1).contiguous(), torch.zeros(H, device="cuda"), -row.float(), g.GDR_GATE_SIGMOID, -5.0)
    out, dx, da, db = nan((T, H * 128), F32), nan((T, H * 128), BF), nan((H,), F32), nan((H * 128,), F32)
    g.gate_fwd(q, out)
    g.gate_bwd(q, dg, dx, da, db, q.alloc_workspace())
    torch.cuda.synchronize()
    assert bool((out == -2.5).all()) and torch.equal(dx.float(), -1.25 * dg) and torch.equal(db, -1.25 * dg.sum(0)) and not da.any()
    del row, dg, q, out, dx, da, db
    print("[case] most state heads", flush=True)
    k, v = torch.randn(1, 1, 128, device="cuda").to(BF), torch.randn(1, H, 128, device="cuda").to(BF)
    beta, decay = torch.rand(1, H, device="cuda"), -torch.rand(1, H, device="cuda")
    state, some = torch.randn(1, H, 128, 128, device="cuda"), [0, 1, 32767, 65535]
    few = state[:, some].contiguous()
    o, want = nan(v.shape, BF), nan((1, 4, 128), BF)
    g.gdn_step(g.StepProblem(g.GDR_GDN, k, k, v, decay, beta, state), o)
    g.gdn_step(g.StepProblem(g.GDR_GDN, k, k, v[:, some].contiguous(), decay[:, some].contiguous(), beta[:, some].contiguous(), few), want)
    torch.cuda.synchronize()
    assert torch.equal(o[:, some], want) and torch.equal(state[:, some], few) and bool(torch.isfinite(o.float()).all())


@pytest.mark.parametrize("place", ["none", "before", "after"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_at_the_borders_of_its_shapes(dt, place):
    """Widths on either side of every row shape's last value, with a gate, both ways."""
    g, dtype = gdr(), DT[dt]
    vec, alpha = 8 if dt == "bf16" else 4, 0.5 if place != "none" else 1.0
    ends = [vec] + [t * vec for t in (16, 32, 64, 128, 192, 256, 512, 768, 1024, 1280, 1536, 2048)] + [16384]
    widths = sorted({D for e in ends for D in (e - 1, e, e + 1) if 2 <= D <= 16384})
    code = {"none": g.GDR_RES_NONE, "before": g.GDR_RES_BEFORE, "after": g.GDR_RES_AFTER}[place]
    for D in widths:
        r, shape, act = rng(D), (5, 1, D), ("silu", "sigmoid")[D & 1]
        print("[case] norm border", dt, place, D, flush=True)
        x, z, dy = (dev(r.standard_normal(shape), dtype) for _ in range(3))
        w = dev(1 + 0.2 * r.standard_normal(D))
        res = dev(r.standard_normal(shape)) if place != "none" else None
        s, ydt = nan(shape, F32) if place == "before" else None, F32 if place == "after" else dtype
        dy = dy.to(ydt)
        p = g.NormProblem(x, w, z, g.GDR_ACT_SILU if act == "silu" else g.GDR_ACT_SIGMOID, res, s, code, alpha)
        y, dx, dz, dw = nan(shape, ydt), nan(shape, dtype), nan(shape, dtype), nan((D,), F32)
        dres = nan(shape, F32) if place == "before" else None
        g.norm_fwd(p, y)
        g.norm_bwd(p, dy, dx, dw, p.alloc_workspace().fill_(0xFF), dgate=dz, dres=dres)
        torch.cuda.synchronize()
        f = ref.norm(f64(x), f64(w), f64(z), f64(res), place, act, alpha, 1e-6)
        d = ref.norm_grad(f64(s) if s is not None else f64(x), f64(w), f64(z), f64(dy), None, place, act, alpha, 1e-6)
        ref.close(y, f["y"], f["Ey"], ydt, "y %d" % D)
        for name, t, odt in (("dx", dx, dtype), ("dz", dz, dtype), ("dw", dw, F32)) + ((("dres", dres, F32),) if dres is not None else ()):
            ref.close(t, d[name], d["E" + name], odt, "%s %d" % (name, D))
