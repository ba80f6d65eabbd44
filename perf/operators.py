"""Measured cases of the operators around the gated delta rule: the short causal
convolution, the decay gate, the single-token recurrence, and the norm with gate
and residual.

A case is one pass through one operator.  `run` computes it in elementary torch
operations (fp32, long sums in fp64, one rounding at the end), or, with `own`,
through libgdr's binding; `exact` computes the same in fp64 from the definition.

Operators (rows of a packed batch are tokens; documents restart every history):
  conv   z[t,c] = b[c] + sum_i w[c,i] X[t-(W-1)+i, c], y = z or SiLU(z); X is the
         document's rows preceded by W-1 rows s0 (zeros without one)
  gate   u = x + b; g = max(floor, -e^a softplus(u)) or g = floor sigmoid(e^a u)
  step   S <- diag(e^g) S; r = S^T k; S <- S + beta k (v - r)^T; o = scale S^T q
  norm   n(x) = x / sqrt(mean x^2 + eps) * w * act(z);  none: y = n(x);
         before: s = res + alpha x, y = n(s);  after: y = res + alpha n(x)
"""
import math

import torch

own = False

PACK4 = "42024,57573,73122,88673"
PACK6 = "18000,27500,36000,44317,52000,64000"
SHARD = "32674"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
FLOOR = -5.0
DEV = "cuda"


def listed():
    return [
        # decode: one token of 64 sequences through the q|k|v convolution of a grouped-head layer (16 + 16 + 48 heads)
        dict(name="conv step 64 seqs C10240", op="conv", mode="step", seqs=64, slots=96, C=10240, W=4, dtype="bf16", act="silu", bias=False),
        # training forward: one projection of a 16-head layer over the four-document pack
        dict(name="conv fwd pack4 C2048", op="conv", mode="fwd", docs=PACK4, C=2048, W=4, dtype="bf16", act="silu", bias=False, s0=False, pad=0),
        # training backward: the value projection of 48 heads over the six-document pack
        dict(name="conv bwd pack6 C6144", op="conv", mode="bwd", docs=PACK6, C=6144, W=4, dtype="bf16", act="silu", bias=False, s0=False, pad=0),
        # a ragged small batch in fp32 with bias and carried-in rows, read out of a wider projection
        dict(name="conv train ragged f32 C385", op="conv", mode="train", docs="1,63,0,64,65,130,7,2000,2,511", C=385, W=3, dtype="f32", act="silu", bias=True, s0=True, pad=15),
        # training forward of the per-channel decay at 16 heads
        dict(name="gate fwd pack4 H16", op="gate", mode="fwd", T=261392, H=16, D=128, kind="softplus", dtype="bf16", bias=True, pad=0),
        # training backward of the bounded per-channel decay on one document's shard
        dict(name="gate bwd shard H16", op="gate", mode="bwd", T=32674, H=16, D=128, kind="sigmoid", dtype="bf16", bias=True, pad=0),
        # the scalar decay of 48 value heads, both directions
        dict(name="gate train pack6 Hv48 D1", op="gate", mode="train", T=241817, H=48, D=1, kind="softplus", dtype="f32", bias=True, pad=0),
        # decode of one sequence, 16 heads: latency
        dict(name="step kda 1 seq H16", op="step", variant="kda", docs="1", slots=1, Hqk=16, Hv=16, act=False, pad=0),
        # decode of a large batch, grouped heads, slots in any order of a larger pool
        dict(name="step gdn 256 seqs Hv48", op="step", variant="gdn", docs="1," * 255 + "1", slots=288, Hqk=16, Hv=48, act=True, pad=0),
        # short runs of tokens per sequence (several proposed tokens at once), an idle sequence among them
        dict(name="step kda runs H64", op="step", variant="kda", docs="4,1,0,8,3,5,1,2,4,4,1,7,6,4,1,1", slots=16, Hqk=64, Hv=64, act=False, pad=128),
        # the head norm of the layer's output with its SiLU gate, training forward over the pack
        dict(name="norm fwd heads pack4 H16", op="norm", mode="fwd", T=261392, H=16, D=128, place="none", dtype="bf16", res="bf16", act="silu", pad=0),
        # the next block's norm with the residual stream in fp32, both directions, on one document's shard
        dict(name="norm train resid shard D2048", op="norm", mode="train", T=32674, H=1, D=2048, place="before", dtype="bf16", res="f32", act="none", pad=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _docs(rng, T):
    """T tokens in a few documents of uneven length, an empty one among them now and then."""
    n = min(T, _log(rng, 1, 40))
    cuts = sorted(rng.randint(0, T) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [T]))


def draw(rng):
    op = rng.choice(["conv", "gate", "step", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "conv":
        C, W, act = _log(rng, 1, 6144), rng.randint(2, 5), rng.choice(["none", "silu", "silu"])
        if rng.random() < 0.5:
            C = (C + 7) // 8 * 8
        if rng.random() < 0.3:
            seqs = _log(rng, 1, 512)
            return dict(op=op, mode="step", seqs=seqs, slots=seqs + rng.randint(0, 40), C=C, W=W, dtype=dtype, act=act, bias=rng.random() < 0.5)
        T = _log(rng, 1, 40000)
        return dict(op=op, mode=rng.choice(["fwd", "bwd", "train"]), docs=_docs(rng, T), C=C, W=W, dtype=dtype, act=act,
                    bias=rng.random() < 0.5, s0=rng.random() < 0.5, pad=rng.choice([0, 0, 8, 13]))
    if op == "gate":
        D = rng.choice([1, 128])
        return dict(op=op, mode=rng.choice(["fwd", "bwd", "train"]), T=_log(rng, 1, 40000), H=rng.randint(1, 64), D=D,
                    kind=rng.choice(["softplus", "sigmoid"]), dtype=dtype, bias=rng.random() < 0.7, pad=rng.choice([0, 8, 5]))
    if op == "step":
        variant = rng.choice(["kda", "gdn"])
        Hqk = rng.choice([1, 2, 3, 4, 8, 16])
        Hv = Hqk * (1 if variant == "kda" else rng.choice([1, 2, 3, 4]))
        seqs, most = _log(rng, 1, 200), rng.choice([1, 1, 1, 2, 5, 8])
        docs = ",".join(str(1 if most == 1 else rng.randint(0, most)) for _ in range(seqs - 1)) + ("," if seqs > 1 else "") + str(most)
        return dict(op=op, variant=variant, docs=docs, slots=seqs + rng.randint(0, 20), Hqk=Hqk, Hv=Hv, act=rng.random() < 0.5, pad=rng.choice([0, 64, 8]))
    res = "f32" if dtype == "f32" else rng.choice(["bf16", "f32"])
    if rng.random() < 0.5:
        H, D, T = rng.randint(1, 48), rng.choice([64, 96, 128, 128, 256]), _log(rng, 1, 20000)
    else:
        H, D, T = 1, _log(rng, 1, 12000), _log(rng, 1, 20000)
    return dict(op=op, mode=rng.choice(["fwd", "bwd", "train"]), T=T, H=H, D=D, place=rng.choice(["none", "before", "after"]), dtype=dtype,
                res=res, act=rng.choice(["none", "silu", "sigmoid"]), pad=rng.choice([0, 0, 8, 3]))


def _lens(case):
    return [int(d) for d in case["docs"].split(",")]


class _Rand:
    """Seeded tensors on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)

    def normal(self, *shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=self.g, device=DEV) * std).to(dtype)

    def uniform(self, lo, hi, *shape):
        return torch.rand(*shape, generator=self.g, device=DEV) * (hi - lo) + lo

    def rows(self, T, C, pad, dtype):
        """[T, C] rows of a buffer `pad` values wider."""
        return self.normal(T, C + pad, dtype=dtype)[:, :C]

    def slots(self, n, of):
        return torch.randperm(of, generator=self.g, device=DEV)[:n].to(torch.int32)


def prepare(case, seed):
    """The inputs of one pass, as tensors on the GPU; cu_seqlens is a host list, as a data loader gives it."""
    r, op = _Rand(seed), case["op"]
    s = {"case": case}
    if op == "conv":
        dt, C, W = DTYPES[case["dtype"]], case["C"], case["W"]
        s["weight"] = r.normal(C, W, std=0.5, dtype=dt)
        s["bias"] = r.normal(C, std=0.2, dtype=dt) if case["bias"] else None
        if case["mode"] == "step":
            s["x"] = r.rows(case["seqs"], C, 0, dt)
            s["state"] = r.normal(case["slots"], W - 1, C, dtype=dt)
            s["slots"] = r.slots(case["seqs"], case["slots"])
            return s
        lens = _lens(case)
        T, N = sum(lens), len(lens)
        s["cu"] = [sum(lens[:i]) for i in range(N + 1)]
        s["x"] = r.rows(T, C, case["pad"], dt)
        s["s0"] = r.normal(N, W - 1, C, dtype=dt) if case["s0"] else None
        s["dy"] = r.normal(T, C, dtype=dt)
        s["dst"] = r.normal(N, W - 1, C, dtype=dt) if case["s0"] else None
    elif op == "gate":
        dt, T, H, D = DTYPES[case["dtype"]], case["T"], case["H"], case["D"]
        s["x"] = r.rows(T, H * D, case["pad"], dt).mul_(0.5)  # the decay projection's output
        s["a_log"] = torch.log(r.uniform(0.25, 4.0, H))
        # a time step of 0.001 to 0.1 at x = 0, through the inverse of softplus
        dt0 = torch.exp(r.uniform(math.log(1e-3), math.log(0.1), H * D))
        s["bias"] = torch.log(torch.expm1(dt0)) if case["bias"] else None
        s["dg"] = r.normal(T, H * D)
    elif op == "step":
        lens, Hqk, Hv, pad = _lens(case), case["Hqk"], case["Hv"], case["pad"]
        T, kda = sum(lens), case["variant"] == "kda"
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
        s["single"] = all(n == 1 for n in lens)

        def heads(H, unit):
            x = r.normal(T, H * 128 + pad)
            if unit:
                x[:, : H * 128] = torch.nn.functional.normalize(x[:, : H * 128].view(T, H, 128), dim=-1).view(T, -1)
            return x.to(torch.bfloat16)[:, : H * 128].unflatten(1, (H, 128))

        s["q"], s["k"], s["v"] = heads(Hqk, not case["act"]), heads(Hqk, not case["act"]), heads(Hv, False)
        s["g"] = r.uniform(-5.0, 0.0, *((T, Hv, 128) if kda else (T, Hv)))
        b = r.normal(T, Hv)
        s["beta"] = (b if case["act"] else torch.sigmoid(b)).to(torch.bfloat16 if kda else torch.float32)
        s["state"] = r.normal(case["slots"], Hv, 128, 128, std=0.1)
        s["slots"] = r.slots(len(lens), case["slots"])
    else:
        dt, rt, T, H, D = DTYPES[case["dtype"]], DTYPES[case["res"]], case["T"], case["H"], case["D"]
        place = case["place"]
        s["x"] = r.rows(T, H * D, case["pad"], dt).unflatten(1, (H, D))
        s["weight"] = r.normal(D, std=0.2) + 1.0
        s["z"] = r.rows(T, H * D, case["pad"], dt).unflatten(1, (H, D)) if case["act"] != "none" else None
        s["residual"] = r.normal(T, H, D, dtype=rt) if place != "none" else None
        s["dy"] = r.normal(T, H, D, dtype=rt if place == "after" else dt)
        s["ds"] = r.normal(T, H, D, dtype=rt) if place == "before" else None
        s["scale"] = 0.5 if place != "none" else 1.0
        if case["mode"] == "bwd" and place == "before":  # the stream that the forward left
            s["s"] = (s["residual"].float() + s["scale"] * s["x"].float()).to(rt)
    return s


def run(s):
    op, mode = s["case"]["op"], s["case"].get("mode")
    if own:
        return {"conv": _own_conv, "gate": _own_gate, "step": _own_step, "norm": _own_norm}[op](s, mode)
    return {"conv": _plain_conv, "gate": _plain_gate, "step": _plain_step, "norm": _plain_norm}[op](s, mode)


# ---- the library's calls -------------------------------------------------------------------------------------


def _own_conv(s, mode):
    import chunked_gated_delta_14_amd as gdr

    c, x = s["case"], s["x"]
    act = gdr.GDR_ACT_SILU if c["act"] == "silu" else gdr.GDR_ACT_NONE
    if mode == "step":
        if "p" not in s:  # the handle of a serving loop's static buffers
            s["p"] = gdr.ConvStep(x, s["weight"], s["state"], s["slots"], s["bias"], act)
        y = torch.empty(x.shape, dtype=x.dtype, device=DEV)
        gdr.conv_step(s["p"], y)
        return {"y": y, "state": s["state"]}
    if "p" not in s:  # the batch's plan and workspace
        s["p"] = gdr.ConvProblem(x, s["weight"], gdr.Plan(s["cu"], DEV), s["bias"], s["s0"], act)
        s["ws"] = s["p"].alloc_workspace()
    p, out = s["p"], {}
    if mode != "bwd":
        out["y"] = torch.empty(x.shape, dtype=x.dtype, device=DEV)
        out["st"] = torch.empty(p.N, c["W"] - 1, c["C"], dtype=x.dtype, device=DEV)
        gdr.conv_fwd(p, out["y"], out["st"])
    if mode != "fwd":
        out["dx"] = torch.empty(x.shape, dtype=x.dtype, device=DEV)
        out["dw"] = torch.empty(c["C"], c["W"], device=DEV)
        out["db"] = torch.empty(c["C"], device=DEV) if c["bias"] else None
        out["ds0"] = torch.empty_like(s["s0"]) if c["s0"] else None
        gdr.conv_bwd(p, s["dy"], s["dst"], out["dx"], out["dw"], out["db"], out["ds0"], s["ws"])
    return out


def _own_gate(s, mode):
    import chunked_gated_delta_14_amd as gdr

    c, x = s["case"], s["x"]
    if "p" not in s:
        kind = gdr.GDR_GATE_SOFTPLUS if c["kind"] == "softplus" else gdr.GDR_GATE_SIGMOID
        s["p"] = gdr.GateProblem(x, s["a_log"], s["bias"], kind, FLOOR)
        s["ws"] = s["p"].alloc_workspace()
    out = {}
    if mode != "bwd":
        out["g"] = torch.empty(x.shape, device=DEV)
        gdr.gate_fwd(s["p"], out["g"])
    if mode != "fwd":
        out["dx"] = torch.empty(x.shape, dtype=x.dtype, device=DEV)
        out["da"] = torch.empty_like(s["a_log"])
        out["db"] = torch.empty_like(s["bias"]) if c["bias"] else None
        gdr.gate_bwd(s["p"], s["dg"], out["dx"], out["da"], out["db"], s["ws"])
    return out


def _own_step(s, mode):
    import chunked_gated_delta_14_amd as gdr

    c = s["case"]
    kda = c["variant"] == "kda"
    if "p" not in s:  # the handle of a serving loop's static buffers
        s["p"] = gdr.StepProblem(gdr.GDR_KDA if kda else gdr.GDR_GDN, s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"],
                                 None if s["single"] else s["cu"], s["slots"],
                                 input_flags=gdr.GDR_IN_QK_L2NORM | gdr.GDR_IN_BETA_SIGMOID if c["act"] else 0)
    o = torch.empty(s["v"].shape, dtype=torch.bfloat16, device=DEV)
    (gdr.kda_step if kda else gdr.gdn_step)(s["p"], o)
    return {"o": o, "state": s["state"]}


def _own_norm(s, mode):
    import chunked_gated_delta_14_amd as gdr

    c, x = s["case"], s["x"]
    act = {"none": gdr.GDR_ACT_NONE, "silu": gdr.GDR_ACT_SILU, "sigmoid": gdr.GDR_ACT_SIGMOID}[c["act"]]
    place = {"none": gdr.GDR_RES_NONE, "before": gdr.GDR_RES_BEFORE, "after": gdr.GDR_RES_AFTER}[c["place"]]
    if "p" not in s:
        stream = s.get("s") if c["mode"] == "bwd" else torch.empty_like(s["residual"]) if c["place"] == "before" else None
        s["p"] = gdr.NormProblem(x, s["weight"], gate=s["z"], activation=act, residual=s["residual"], s=stream, placement=place,
                                 scale=s["scale"], eps=EPS)
        s["ws"] = s["p"].alloc_workspace()
    p, out = s["p"], {}
    if mode != "bwd":
        out["y"] = torch.empty(x.shape, dtype=s["dy"].dtype, device=DEV)
        gdr.norm_fwd(p, out["y"])
        out["s"] = p.s
    if mode != "fwd":
        out["dx"] = torch.empty(x.shape, dtype=x.dtype, device=DEV)
        out["dw"] = torch.empty(c["D"], device=DEV)
        out["dz"] = torch.empty(x.shape, dtype=x.dtype, device=DEV) if s["z"] is not None else None
        out["dres"] = torch.empty_like(s["residual"]) if c["place"] == "before" else None
        gdr.norm_bwd(p, s["dy"], out["dx"], out["dw"], s["ws"], dgate=out["dz"], ds=s["ds"], dres=out["dres"])
    return out


# ---- the plain forms -----------------------------------------------------------------------------------------


def _rows_of(cu, hist):
    """For documents laid out with `hist` rows before each: the row of every token's first tap, the rows of the carried-in
    part and those of the last `hist` rows, [N, hist]."""
    N = len(cu) - 1
    c = torch.tensor(cu, device=DEV)
    lens = c[1:] - c[:-1]
    doc = torch.repeat_interleave(torch.arange(N, device=DEV), lens)
    first = torch.arange(cu[-1], device=DEV) + doc * hist
    j = torch.arange(hist, device=DEV)
    start = c[:-1] + torch.arange(N, device=DEV) * hist
    return first, start[:, None] + j, (start + lens)[:, None] + j


def _plain_conv(s, mode):
    c, x = s["case"], s["x"]
    dt, C, W, silu = x.dtype, c["C"], c["W"], c["act"] == "silu"
    w = s["weight"].float()
    b = s["bias"].float() if c["bias"] else torch.zeros(C, device=DEV)
    if mode == "step":
        at = s["slots"].long()
        rows = torch.cat([s["state"][at], x[:, None]], 1)
        z = (rows.float() * w.t()).sum(1) + b
        s["state"][at] = rows[:, 1:]
        return {"y": (z * torch.sigmoid(z) if silu else z).to(dt), "state": s["state"]}
    hist, T, N = W - 1, s["cu"][-1], len(s["cu"]) - 1
    first, head, tail = _rows_of(s["cu"], hist)
    X = torch.zeros(T + N * hist, C, device=DEV)
    X[first + hist] = x.float()
    if c["s0"]:
        X[head] = s["s0"].float()
    z = sum((X[first + i] * w[:, i] for i in range(W)), b)
    sig = torch.sigmoid(z)
    out = {}
    if mode != "bwd":
        out["y"] = (z * sig if silu else z).to(dt)
        out["st"] = X[tail].to(dt)
    if mode != "fwd":
        dz = s["dy"].float() * (sig * (1 + z * (1 - sig)) if silu else 1.0)
        del z, sig
        out["dw"] = torch.stack([(dz * X[first + i]).sum(0, dtype=torch.float64) for i in range(W)], 1).float()
        out["db"] = dz.sum(0, dtype=torch.float64).float() if c["bias"] else None
        dX = torch.zeros_like(X)
        dX = sum((torch.zeros_like(X).index_copy_(0, first + i, dz * w[:, i]) for i in range(W)), dX)
        if s["dst"] is not None:
            dX[tail] += s["dst"].float()
        out["dx"] = dX[first + hist].to(dt)
        out["ds0"] = dX[head].to(dt) if c["s0"] else None
    return out


def _plain_gate(s, mode):
    c, x = s["case"], s["x"]
    T, H, D = c["T"], c["H"], c["D"]
    u = x.float().reshape(T, H, D)
    if c["bias"]:
        u = u + s["bias"].view(H, D)
    ea = torch.exp(s["a_log"])[:, None]
    if c["kind"] == "softplus":
        raw = -ea * (u.clamp_min(0) + torch.log1p(torch.exp(-u.abs())))
        g = raw.clamp_min(FLOOR)
        live = (raw >= FLOOR).float()
    else:
        sig = torch.sigmoid(ea * u)
        g = FLOOR * sig
    out = {}
    if mode != "bwd":
        out["g"] = g.reshape(T, H * D)
    if mode != "fwd":
        dg = s["dg"].view(T, H, D)
        if c["kind"] == "softplus":
            du, da = -dg * live * ea * torch.sigmoid(u), dg * live * raw
        else:
            t = dg * FLOOR * ea * (sig * (1 - sig))
            du, da = t, t * u
        out["dx"] = du.reshape(T, H * D).to(x.dtype)
        out["da"] = da.sum((0, 2), dtype=torch.float64).float()
        out["db"] = du.sum(0, dtype=torch.float64).float().reshape(H * D) if c["bias"] else None
    return out


def _plain_step(s, mode):
    c = s["case"]
    Hv, group, kda = c["Hv"], c["Hv"] // c["Hqk"], c["variant"] == "kda"
    q, k = (s[n].float().repeat_interleave(group, 1) for n in ("q", "k"))
    v, beta, decay = s["v"].float(), s["beta"].float(), torch.exp(s["g"])
    if c["act"]:
        q, k = (t * torch.rsqrt(t.square().sum(-1, keepdim=True) + 1e-6) for t in (q, k))
        beta = torch.sigmoid(beta)
    decay = decay[..., None] if kda else decay[..., None, None]
    at, lens = s["slots"].long(), torch.tensor(_lens(c))
    start = torch.cumsum(lens, 0) - lens
    o = torch.zeros(v.shape, dtype=torch.bfloat16, device=DEV)
    for i in range(int(lens.max())):  # token i of every sequence that has one: each needs the state of the one before
        live = (lens > i).nonzero().flatten()
        t, slot = (start[live] + i).to(DEV), at[live.to(DEV)]
        S = s["state"][slot] * decay[t]
        r = (S * k[t][..., None]).sum(-2)
        S = S + k[t][..., None] * (beta[t][..., None] * (v[t] - r))[..., None, :]
        o[t] = ((S * q[t][..., None]).sum(-2) * 128 ** -0.5).to(torch.bfloat16)
        s["state"][slot] = S
    return {"o": o, "state": s["state"]}


def _plain_norm(s, mode):
    c, x = s["case"], s["x"]
    w, alpha, D, place = s["weight"], s["scale"], c["D"], c["place"]
    if place == "before" and mode != "bwd":
        base = s["residual"].float() + alpha * x.float()
    else:
        base = s["s"].float() if place == "before" else x.float()
    z = s["z"].float() if s["z"] is not None else None
    sig = torch.sigmoid(z) if z is not None else None
    a = 1.0 if z is None else z * sig if c["act"] == "silu" else sig
    rs = torch.rsqrt(base.square().mean(-1, keepdim=True) + EPS)
    out = {}
    if mode != "bwd":
        y = base * rs * w * a
        out["y"] = (s["residual"].float() + alpha * y if place == "after" else y).to(s["dy"].dtype)
        out["s"] = base.to(s["residual"].dtype) if place == "before" else None
    if mode != "fwd":
        if place == "before" and mode == "train":  # the backward reads the stream as it was stored
            base = out["s"].float()
            rs = torch.rsqrt(base.square().mean(-1, keepdim=True) + EPS)
        dy = s["dy"].float() * (alpha if place == "after" else 1.0)
        n = base * rs
        if z is not None:
            da = sig * (1 + z * (1 - sig)) if c["act"] == "silu" else sig * (1 - sig)
            out["dz"] = (dy * n * w * da).to(x.dtype)
        t = dy * a
        out["dw"] = (t * n).sum((0, 1), dtype=torch.float64).float()
        t = t * w
        d = rs * (t - n * (t * n).mean(-1, keepdim=True))
        if place == "before":
            d = d + s["ds"].float()
            out["dres"] = d.to(s["residual"].dtype)
            d = alpha * d
        out["dx"] = d.to(x.dtype)
    return out


# ---- what a pass cannot do without ---------------------------------------------------------------------------


def work(case):
    op, mode = case["op"], case.get("mode")
    e = 2 if case.get("dtype") == "bf16" else 4
    if op == "conv":
        C, W = case["C"], case["W"]
        if mode == "step":
            n = case["seqs"] * C
            return {"bytes": e * n * (2 + 2 * (W - 1)), "flops": n * (2 * W + 6)}
        n = sum(_lens(case)) * C
        rows = len(_lens(case)) * (W - 1) * C * e
        moved = {"fwd": 2, "bwd": 3, "train": 5}[mode] * n * e + rows * (2 if case["s0"] else 1)
        return {"bytes": moved + 5 * C * W, "flops": n * {"fwd": 2 * W + 6, "bwd": 6 * W + 16, "train": 8 * W + 22}[mode]}
    if op == "gate":
        n = case["T"] * case["H"] * case["D"]
        return {"bytes": n * {"fwd": e + 4, "bwd": 2 * e + 4, "train": 3 * e + 8}[mode], "flops": n * {"fwd": 12, "bwd": 20, "train": 32}[mode]}
    if op == "step":
        lens, Hqk, Hv = _lens(case), case["Hqk"], case["Hv"]
        T, live = sum(lens), sum(1 for n in lens if n)
        g = T * Hv * (128 * 4 if case["variant"] == "kda" else 4)
        return {"bytes": live * Hv * 2 * 65536 + T * (2 * Hqk + 2 * Hv) * 256 + g, "flops": T * Hv * 128 * 128 * 7}
    n = case["T"] * case["H"] * case["D"]
    r = 2 if case["res"] == "bf16" else 4
    z = e if case["act"] != "none" else 0
    place = case["place"]
    fwd = {"none": 2 * e, "before": 2 * e + 2 * r, "after": e + 2 * r}[place] + z
    bwd = {"none": 3 * e, "before": 2 * e + 3 * r, "after": 2 * e + r}[place] + 2 * z
    return {"bytes": n * {"fwd": fwd, "bwd": bwd, "train": fwd + bwd}[mode], "flops": n * {"fwd": 8, "bwd": 16, "train": 24}[mode]}


# ---- the definitions in fp64 ---------------------------------------------------------------------------------


def exact(case, seed):
    s, op, mode = prepare(case, seed), case["op"], case.get("mode")
    with torch.enable_grad():
        return {"conv": _exact_conv, "gate": _exact_gate, "step": _exact_step, "norm": _exact_norm}[op](s, mode)


def _f64(t, grad=True):
    t = t.detach().double()
    return t.clone().requires_grad_(True) if grad else t


def _exact_conv(s, mode):
    """Document by document and 256 channels at a time; gradients by reverse mode over the definition."""
    c, W, C = s["case"], s["case"]["W"], s["case"]["C"]
    act = torch.nn.functional.silu if c["act"] == "silu" else lambda u: u
    if mode == "step":
        at = s["slots"].tolist()
        rows = torch.stack([torch.cat([s["state"][m].double(), s["x"][n : n + 1].double()]) for n, m in enumerate(at)])
        z = torch.einsum("nwc,cw->nc", rows, s["weight"].double())
        z = z + s["bias"].double() if c["bias"] else z
        state = s["state"].double().clone()
        for n, m in enumerate(at):
            state[m] = rows[n, 1:]
        return {"y": act(z), "state": state}
    N, block = len(s["cu"]) - 1, 256
    out = {}

    def put(key, shape, index, val):
        if key not in out:
            out[key] = torch.zeros(shape, dtype=torch.float64, device=DEV)
        out[key][index] += val

    T = s["cu"][-1]
    for lo in range(0, C, block):
        ch = slice(lo, min(C, lo + block))
        w = _f64(s["weight"][ch])
        b = _f64(s["bias"][ch]) if c["bias"] else torch.zeros(w.shape[0], dtype=torch.float64, device=DEV, requires_grad=True)
        for n in range(N):
            span = slice(s["cu"][n], s["cu"][n + 1])
            x = _f64(s["x"][span, ch])
            s0 = _f64(s["s0"][n][:, ch]) if c["s0"] else torch.zeros(W - 1, w.shape[0], dtype=torch.float64, device=DEV, requires_grad=True)
            seen = torch.cat([s0, x])
            y = act(b + (seen.unfold(0, W, 1) * w).sum(-1)) if len(x) else x
            st = seen[len(x) :]
            if mode != "bwd":
                put("y", (T, C), (span, ch), y.detach())
                put("st", (N, W - 1, C), (n, slice(None), ch), st.detach())
            if mode == "fwd":
                continue
            loss = (y * s["dy"][span, ch].double()).sum()
            if s["dst"] is not None:
                loss = loss + (st * s["dst"][n][:, ch].double()).sum()
            gx, gs, gw, gb = torch.autograd.grad(loss, [x, s0, w, b], allow_unused=True)
            put("dx", (T, C), (span, ch), 0 if gx is None else gx)
            put("dw", (C, W), ch, 0 if gw is None else gw)
            if c["bias"]:
                put("db", (C,), ch, 0 if gb is None else gb)
            if c["s0"]:
                put("ds0", (N, W - 1, C), (n, slice(None), ch), 0 if gs is None else gs)
    return out


def _exact_gate(s, mode):
    """A few heads at a time."""
    c = s["case"]
    T, H, D, parts = c["T"], c["H"], c["D"], []
    step = max(1, min(H, (1 << 27) // max(1, T * D)))
    for lo in range(0, H, step):
        hs, cs = slice(lo, min(H, lo + step)), slice(lo * D, min(H, lo + step) * D)
        x, a = _f64(s["x"][:, cs]), _f64(s["a_log"][hs])
        b = _f64(s["bias"][cs]) if c["bias"] else torch.zeros(x.shape[1], dtype=torch.float64, device=DEV, requires_grad=True)
        u = (x + b).view(T, -1, D)
        A = a.exp()[:, None]
        if c["kind"] == "softplus":
            g = torch.maximum(-A * torch.logaddexp(u, torch.zeros_like(u)), torch.full_like(u, FLOOR))
        else:
            g = FLOOR / (1 + torch.exp(-A * u))
        g = g.reshape(T, -1)
        got = {} if mode == "bwd" else {"g": g.detach()}
        if mode != "fwd":
            got["dx"], got["da"], db = torch.autograd.grad(g, [x, a, b], s["dg"][:, cs].double())
            if c["bias"]:
                got["db"] = db
        parts.append(got)
    return {key: torch.cat([p[key] for p in parts], dim=-1) for key in parts[0]}


def _exact_step(s, mode):
    """The recurrence with the erase matrix written out, 16 sequences at a time."""
    c, lens = s["case"], _lens(s["case"])
    Hqk, Hv, kda = c["Hqk"], c["Hv"], c["variant"] == "kda"
    of = [h // (Hv // Hqk) for h in range(Hv)]
    state = s["state"].double()
    o = torch.zeros(s["v"].shape, dtype=torch.float64, device=DEV)
    eye = torch.eye(128, dtype=torch.float64, device=DEV)
    start, at = [sum(lens[:n]) for n in range(len(lens))], s["slots"].tolist()
    for i in range(max(lens)):
        rows = [n for n in range(len(lens)) if lens[n] > i]
        for lo in range(0, len(rows), 16):
            some = rows[lo : lo + 16]
            t, m = [start[n] + i for n in some], [at[n] for n in some]
            q, k, v, b = s["q"][t].double()[:, of], s["k"][t].double()[:, of], s["v"][t].double(), s["beta"][t].double()
            if c["act"]:
                q, k = q / (q.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt(), k / (k.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt()
                b = 1 / (1 + torch.exp(-b))
            g = s["g"][t].double().exp()
            g = g if kda else g[..., None].expand(-1, -1, 128)
            erase = eye - b[..., None, None] * k[..., :, None] * k[..., None, :]
            S = erase @ (g[..., :, None] * state[m]).contiguous() + b[..., None, None] * k[..., :, None] * v[..., None, :]
            state[m] = S
            o[t] = (S * q[..., :, None]).sum(-2) / math.sqrt(128)
    return {"o": o, "state": state}


def _exact_norm(s, mode):
    """A few thousand rows at a time; gradients by reverse mode over the definition."""
    c, place, alpha = s["case"], s["case"]["place"], s["scale"]
    T, D, rt = c["T"], c["D"], DTYPES[c["res"]]
    step = max(1, (1 << 26) // (c["H"] * D))
    act = {"none": None, "silu": torch.nn.functional.silu, "sigmoid": torch.sigmoid}[c["act"]]
    parts, dw = [], torch.zeros(D, dtype=torch.float64, device=DEV)

    def norm(base, w, z):
        n = base / (base.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w
        return n if z is None else n * act(z)

    for lo in range(0, T, step):
        rows, got = slice(lo, min(T, lo + step)), {}
        x, w = _f64(s["x"][rows]), _f64(s["weight"])
        z = _f64(s["z"][rows]) if s["z"] is not None else None
        res = s["residual"][rows].double() if s["residual"] is not None else None
        if place == "before":
            stream = s["s"][rows].double() if mode == "bwd" else (res + alpha * x).detach()
            y = norm(stream, w, z)
        else:
            y = norm(x, w, z) if place == "none" else res + alpha * norm(x, w, z)
        if mode != "bwd":
            got["y"] = y.detach()
            if place == "before":
                got["s"] = stream
        if mode != "fwd":
            base = x
            if place == "before":  # the backward's input is the stored stream
                base = (stream if mode == "bwd" else (s["residual"][rows].float() + alpha * s["x"][rows].float()).to(rt).double()).requires_grad_(True)
                y = norm(base, w, z)
            leaves = [base, w] + ([z] if z is not None else [])
            grads = torch.autograd.grad(y, leaves, s["dy"][rows].double())
            dw += grads[1]
            d = grads[0]
            if place == "before":
                d = d + s["ds"][rows].double()
                got["dres"], d = d, alpha * d
            got["dx"] = d
            if z is not None:
                got["dz"] = grads[2]
        parts.append(got)
    out = {key: torch.cat([p[key] for p in parts]) for key in parts[0]}
    if mode != "fwd":
        out["dw"] = dw
    return out
