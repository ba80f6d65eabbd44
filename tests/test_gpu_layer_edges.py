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
