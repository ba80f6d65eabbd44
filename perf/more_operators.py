"""Measured cases of the operators of the softmax-attention layers that stand between
gated delta-rule layers: rotary positions, attention over packed documents with its
backward, and a cache held in 4 bits with the attention that reads it.

A case is one pass through one operator.  `run` computes it in elementary torch
operations (fp32, angles and long sums in fp64, one rounding at the end), or, with
`own`, through libgdr's binding; `exact` computes the same in fp64 from the definition.

Operators (D = 128 channels a head; rows of a packed batch are tokens):
  rope    (a, b) -> m (a cos - b sin, b cos + a sin) by the angle p f_i, for pair i of the
          first R channels: (i, i + R/2) or (2i, 2i + 1); backward: by -p f_i
  attn    o_i = sum_j softmax_j(scale q_i k_j) v_j over the keys that row i sees: with p =
          i + Lk - Lq in its document, j <= p if causal, and j > p - w with a window w; a
          row that sees none gives 0 and a log-sum-exp of -inf
  kv      a token's 128 channels in blocks of 32: e2m1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and
          a sign, ties to even) times 2^e, e the smallest with max|x| <= 6 2^e
  attend  attn of the last tokens of each sequence over keys and values held so
"""
import math

import torch

own = False

PACK4 = "42024,57573,73122,88673"
SHARD = "32674"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
D = 128
DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK_SCORES = 1 << 29  # scores that the plain form holds at once


def listed():
    return [
        # decode: one token of one sequence, far into a long context, half of each head rotated
        dict(name="rope 1 token H16+2", op="rope", mode="fwd", docs="", T=1, Hq=16, Hk=2, rot=64, layout="half", scaling="none", base=1e6, far=200000, dtype="bf16", pad=0),
        # training forward: queries and keys of the four-document pack, positions by document
        dict(name="rope fwd pack4 H16+4", op="rope", mode="fwd", docs=PACK4, T=0, Hq=16, Hk=4, rot=128, layout="half", scaling="none", base=1e4, far=0, dtype="bf16", pad=0),
        # both directions on one document's shard in fp32, neighbouring pairs, frequencies blended for a longer context
        dict(name="rope train shard f32 H8+8", op="rope", mode="train", docs=SHARD, T=0, Hq=8, Hk=8, rot=96, layout="pairs", scaling="blend", base=5e5, far=0, dtype="f32", pad=32),
        # training forward on one document's shard, four query heads to a key head
        dict(name="attn fwd shard H16/4", op="attn", mode="fwd", docs=SHARD, docs_k="", Hq=16, Hkv=4, causal=True, window=0, pad=0),
        # its backward
        dict(name="attn bwd shard H16/4", op="attn", mode="bwd", docs=SHARD, docs_k="", Hq=16, Hkv=4, causal=True, window=0, pad=0),
        # a pack of short documents, one of them empty, out of a wider projection
        dict(name="attn train ragged H4/1", op="attn", mode="train", docs="1,63,0,64,65,130,7,2000,2,511", docs_k="", Hq=4, Hkv=1, causal=True, window=0, pad=64),
        # a step over documents of ordinary length with a window
        dict(name="attn train window H8/8", op="attn", mode="train", docs="4100,2047,1025,3000,2500,1900,1812", docs_k="", Hq=8, Hkv=8, causal=True, window=1024, pad=0),
        # a prompt's next chunk: queries that follow keys already held, one sequence with fewer keys than queries
        dict(name="attn fwd chunk H32/8", op="attn", mode="fwd", docs="512,300,1,700", docs_k="8192,5000,3000,650", Hq=32, Hkv=8, causal=True, window=0, pad=0),
        # a long prompt stored in 4 bits and read back
        dict(name="kv prompt shard H4", op="kv", past="0", new=SHARD, Hkv=4, page=64, pad=0),
        # the next chunk of several requests: stored, and the whole of each read back
        dict(name="kv chunks 6 seqs H8", op="kv", past="4001,0,130,15,2048,777", new="512,511,1,1,300,0", Hkv=8, page=16, pad=64),
        # decode of one sequence: latency
        dict(name="attend 1 seq 4096 H16/2", op="attend", lens="4096", runs="1", Hq=16, Hkv=2, page=16, window=0, pad=0),
        # decode of a large ragged batch
        dict(name="attend 64 seqs to 32k H32/8", op="attend", lens=",".join(str(1 + 517 * i - (i * i) % 97) for i in range(64)), runs="1", Hq=32, Hkv=8, page=64, window=0, pad=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _docs(rng, T):
    """T tokens in a few documents of uneven length, an empty one among them now and then."""
    n = min(T, _log(rng, 1, 30))
    cuts = sorted(rng.randint(0, T) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [T]))


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "kv", "attend", "attend"])
    pad = rng.choice([0, 0, 64, 8])
    if op == "rope":
        T, docs = _log(rng, 1, 40000), rng.random() < 0.5
        return dict(op=op, mode=rng.choice(["fwd", "bwd", "train"]), docs=_docs(rng, T) if docs else "", T=0 if docs else T, Hq=rng.randint(1, 32),
                    Hk=rng.randint(0, 8), rot=2 * rng.randint(1, 64), layout=rng.choice(["half", "pairs"]), scaling=rng.choice(["none", "linear", "base", "blend"]),
                    base=rng.choice([1e4, 5e5, 1e6]), far=_log(rng, 1, 1000000), dtype=rng.choice(["bf16", "bf16", "f32"]), pad=rng.choice([0, 0, 8, 13]))
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 1, 2, 3, 4, 6, 8])
    if op == "attn":
        T = _log(rng, 1, max(64, min(20000, int(240000 / math.sqrt(Hq * 16)))))
        mode, docs = rng.choice(["fwd", "bwd", "train"]), _docs(rng, T)
        causal = rng.random() < 0.8
        docs_k = ""
        if rng.random() < 0.3:  # keys of another length than the queries
            docs_k = ",".join(str(max(0, int(n) + rng.randint(-20, 600))) for n in docs.split(","))
        window = _log(rng, 1, 4000) if causal and rng.random() < 0.4 else 0
        return dict(op=op, mode=mode, docs=docs, docs_k=docs_k, Hq=Hq, Hkv=Hkv, causal=causal, window=window, pad=pad)
    n, page = _log(rng, 1, 64), rng.choice([16, 32, 64, 128])
    if op == "kv":
        most = 60000 // n
        past = ",".join(str(rng.randint(0, _log(rng, 1, most))) for _ in range(n))
        new = ",".join(str(rng.randint(0 if n > 1 else 1, _log(rng, 1, most))) for _ in range(n)) if rng.random() < 0.5 else ",".join(["1"] * n)
        return dict(op=op, past=past, new=new, Hkv=Hkv, page=page, pad=pad)
    lens = ",".join(str(rng.randint(1, _log(rng, 1, 300000 // n))) for _ in range(n))
    runs = "1" if rng.random() < 0.6 else ",".join(str(min(int(m), rng.randint(0, 8))) for m in lens.split(","))
    if not any(int(r) for r in runs.split(",")):
        runs = "1"
    return dict(op=op, lens=lens, runs=runs, Hq=Hq, Hkv=Hkv, page=page, window=_log(rng, 1, 4000) if rng.random() < 0.2 else 0, pad=pad)


def _ints(text):
    return [int(x) for x in text.split(",")] if text else []


def _starts(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


def _runs(case):
    n = len(_ints(case["lens"]))
    return [1] * n if case["runs"] == "1" else _ints(case["runs"])


def _tokens(case):
    return case["T"] or sum(_ints(case["docs"]))


class _Rand:
    """Seeded tensors on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32):
        return torch.randn(*shape, generator=self.g, device=DEV).to(dtype)

    def heads(self, T, H, pad, dtype=torch.bfloat16):
        """[T, H, 128] rows of a buffer `pad` values wider."""
        return self.normal(T, H * D + pad, dtype=dtype)[:, : H * D].unflatten(1, (H, D))

    def ints(self, hi, n):
        return torch.randint(0, hi, (n,), generator=self.g, device=DEV, dtype=torch.int32)

    def order(self, n):
        return torch.randperm(n, generator=self.g, device=DEV)


SCALE = {"linear": 4.0, "base": 8.0, "blend": 8.0}


def _freqs(case):
    """Radians a token for every pair, fp64 on the host, and the magnitude."""
    R, base, kind = case["rot"], case["base"], case["scaling"]
    s = SCALE.get(kind, 1.0)
    if kind == "base" and R > 2:
        base *= s ** (R / (R - 2))
    f = [base ** (-2.0 * i / R) for i in range(R // 2)]
    if kind == "linear":
        f = [x / s for x in f]
    if kind != "blend":
        return f, 1.0
    ramp = [min(max((4096 * x / (2 * math.pi) - 1.0) / 31.0, 0.0), 1.0) for x in f]
    return [x * ((1 - c) / s + c) for x, c in zip(f, ramp)], 0.1 * math.log(s) + 1.0


def _pool(s, r, lens, Hkv, page):
    """Pages for sequences of these lengths, handed out in no order, a few pages more in the pool."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + 3
    order = r.order(total).to(torch.int32)
    s["table"] = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32, device=DEV)
    at = _starts(need)
    for n in range(len(lens)):
        s["table"][n, : need[n]] = order[at[n] : at[n + 1]]
    for side in ("k", "v"):
        s[side + "_codes"] = torch.empty(total, Hkv, page, D // 2, dtype=torch.uint8, device=DEV)
        s[side + "_scale"] = torch.empty(total, Hkv, page, D // 32, dtype=torch.uint8, device=DEV)
        for p in range(0, total, 512):  # what earlier tokens left
            x = r.normal(min(512, total - p), Hkv, page, D, dtype=torch.bfloat16)
            s[side + "_codes"][p : p + 512], s[side + "_scale"][p : p + 512] = _to_4bit(x)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    """The inputs of one pass, as tensors on the GPU; cu_seqlens of a packed batch is a host list, as a data loader gives it."""
    r, op = _Rand(seed), case["op"]
    s = {"case": case}
    if op == "rope":
        T, dt, pad = _tokens(case), DTYPES[case["dtype"]], case["pad"]
        s["cu"] = _starts(_ints(case["docs"])) if case["docs"] else None
        s["pos"] = None if case["docs"] else r.ints(case["far"], T)
        for n in ("", "d"):  # the projections' rows, and the gradients of the rotated ones
            s[n + "q"] = r.heads(T, case["Hq"], pad, dt)
            s[n + "k"] = r.heads(T, case["Hk"], pad, dt) if case["Hk"] else None
    elif op == "attn":
        Lq = _ints(case["docs"])
        Lk = _ints(case["docs_k"]) or Lq
        s["cu_q"], s["cu_k"] = _starts(Lq), _starts(Lk)
        s["q"] = r.heads(sum(Lq), case["Hq"], case["pad"])
        s["k"], s["v"] = (r.heads(sum(Lk), case["Hkv"], case["pad"]) for _ in range(2))
        if case["mode"] != "fwd":
            s["do"] = r.normal(sum(Lq), case["Hq"], D, dtype=torch.bfloat16)
        if case["mode"] == "bwd":  # what the forward left
            s["o"], s["lse"] = _plain_attn_fwd(s)
    elif op == "kv":
        past, new = _ints(case["past"]), _ints(case["new"])
        s["k"], s["v"] = (r.heads(sum(new), case["Hkv"], case["pad"]) for _ in range(2))
        _pool(s, r, [a + b for a, b in zip(past, new)], case["Hkv"], case["page"])
        s["past"] = torch.tensor(past, dtype=torch.int32, device=DEV)
        s["zero"] = torch.zeros_like(s["past"])
        s["cu_new"] = torch.tensor(_starts(new), dtype=torch.int32, device=DEV)
        s["cu_all"] = torch.tensor(_starts([a + b for a, b in zip(past, new)]), dtype=torch.int32, device=DEV)
        s["single"], s["T_all"] = all(n == 1 for n in new), sum(past) + sum(new)
    else:
        runs = _runs(case)
        s["q"] = r.heads(sum(runs), case["Hq"], case["pad"])
        _pool(s, r, _ints(case["lens"]), case["Hkv"], case["page"])
        s["cu"] = torch.tensor(_starts(runs), dtype=torch.int32, device=DEV)
        s["single"] = all(n == 1 for n in runs)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _own_rope, "attn": _own_attn, "kv": _own_kv, "attend": _own_attend}[op](s)
    return {"rope": _plain_rope, "attn": _plain_attn, "kv": _plain_kv, "attend": _plain_attend}[op](s)


# ---- the library's calls -------------------------------------------------------------------------------------


def _own_rope(s):
    import chunked_gated_delta_14_amd as gdr

    c = s["case"]
    if "p" not in s:
        kind = {"none": gdr.GDR_ROPE_PLAIN, "linear": gdr.GDR_ROPE_LINEAR, "base": gdr.GDR_ROPE_BASE, "blend": gdr.GDR_ROPE_BLEND}[c["scaling"]]
        freqs = gdr.rope_freqs(c["rot"], c["base"], kind, factor=SCALE.get(c["scaling"], 1.0), original=4096, low=1.0, high=32.0, device=DEV)
        s["p"] = gdr.RopeProblem(s["q"], s["k"], freqs, positions=s["pos"], plan=gdr.Plan(s["cu"], DEV) if s["cu"] else None,
                                 layout=gdr.GDR_ROPE_HALF if c["layout"] == "half" else gdr.GDR_ROPE_PAIRS, magnitude=_freqs(c)[1])
    out = {}
    new = lambda t: torch.empty(t.shape, dtype=t.dtype, device=DEV) if t is not None else None  # noqa: E731
    if c["mode"] != "bwd":
        out["q"], out["k"] = new(s["q"]), new(s["k"])
        gdr.rope_fwd(s["p"], out["q"], out["k"])
    if c["mode"] != "fwd":
        out["dq"], out["dk"] = new(s["q"]), new(s["k"])
        gdr.rope_bwd(s["p"], s["dq"], s["dk"], out["dq"], out["dk"])
    return out


def _own_attn(s):
    import chunked_gated_delta_14_amd as gdr

    c, q = s["case"], s["q"]
    if "p" not in s:  # the batch's plan and workspace
        plan = gdr.AttnPlan(s["cu_q"], s["cu_k"] if c["docs_k"] else None, causal=c["causal"], window=c["window"], device=DEV)
        s["p"] = gdr.AttnProblem(q, s["k"], s["v"], plan)
        s["ws"] = s["p"].alloc_workspace() if c["mode"] != "fwd" else None
    out, o, lse = {}, s.get("o"), s.get("lse")
    if c["mode"] != "bwd":
        o, lse = torch.empty(q.shape, dtype=q.dtype, device=DEV), torch.empty(c["Hq"], q.shape[0], device=DEV)
        gdr.attn_fwd(s["p"], o, lse)
        out.update(o=o, lse=lse)
    if c["mode"] != "fwd":
        for n in ("q", "k", "v"):
            out["d" + n] = torch.empty(s[n].shape, dtype=q.dtype, device=DEV)
        gdr.attn_bwd(s["p"], o, lse, s["do"], out["dq"], out["dk"], out["dv"], s["ws"])
    return out


def _cache(s):
    import chunked_gated_delta_14_amd as gdr

    return gdr.KvCache(s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"])


def _own_kv(s):
    import chunked_gated_delta_14_amd as gdr

    if "p" not in s:  # a serving loop's static buffers
        cache = _cache(s)
        s["p"] = gdr.KvProblem(cache, s["table"], s["past"], s["k"].shape[0], None if s["single"] else s["cu_new"])
        s["all"] = gdr.KvProblem(cache, s["table"], s["zero"], s["T_all"], s["cu_all"])
    gdr.kv_store(s["p"], s["k"], s["v"])
    k, v = (torch.empty(s["T_all"], s["case"]["Hkv"], D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    gdr.kv_load(s["all"], k, v)
    return {"k": k, "v": v}


def _own_attend(s):
    import chunked_gated_delta_14_amd as gdr

    if "p" not in s:  # a serving loop's static buffers
        s["p"] = gdr.AttnStep(s["q"], _cache(s), s["table"], s["lens"], None if s["single"] else s["cu"], window=s["case"]["window"])
        s["ws"] = s["p"].alloc_workspace()
    o = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=DEV)
    gdr.attn_step(s["p"], o, s["ws"])
    return {"o": o}


# ---- the plain forms -----------------------------------------------------------------------------------------


def _positions(s):
    if s["pos"] is not None:
        return s["pos"].double()
    c = torch.tensor(s["cu"], device=DEV)
    return (torch.arange(s["cu"][-1], device=DEV) - torch.repeat_interleave(c[:-1], c[1:] - c[:-1])).double()


def _plain_rope(s):
    c = s["case"]
    R, half = c["rot"], c["layout"] == "half"
    freqs, m = _freqs(c)
    angle = _positions(s)[:, None, None] * torch.tensor(freqs, dtype=torch.float64, device=DEV)
    cos, sin = (torch.cos(angle) * m).float(), (torch.sin(angle) * m).float()

    def turn(x, sign):
        if x is None:
            return None
        y = x.float()
        a, b = (y[..., : R // 2], y[..., R // 2 : R]) if half else (y[..., 0:R:2], y[..., 1:R:2])
        a, b = a * cos - b * (sign * sin), b * cos + a * (sign * sin)
        y = torch.cat([torch.cat([a, b], -1) if half else torch.stack([a, b], -1).flatten(-2), y[..., R:]], -1)
        return y.to(x.dtype)

    out = {}
    if c["mode"] != "bwd":
        out["q"], out["k"] = turn(s["q"], 1.0), turn(s["k"], 1.0)
    if c["mode"] != "fwd":
        out["dq"], out["dk"] = turn(s["dq"], -1.0), turn(s["dk"], -1.0)
    return out


def _blocks(s):
    """(rows, keys, mask) for blocks of query rows: slices of the packed rows, and which scores are hidden."""
    c = s["case"]
    for n in range(len(s["cu_q"]) - 1):
        q0, q1, k0, k1 = s["cu_q"][n], s["cu_q"][n + 1], s["cu_k"][n], s["cu_k"][n + 1]
        Lq, Lk = q1 - q0, k1 - k0
        step = max(64, BLOCK_SCORES // max(1, c["Hq"] * Lk))
        for r in range(0, Lq, step):
            e = min(Lq, r + step)
            hi = min(Lk, max(0, e + Lk - Lq)) if c["causal"] else Lk
            lo = min(hi, max(0, r + Lk - Lq - c["window"] + 1)) if c["window"] else 0
            p = (torch.arange(r, e, device=DEV) + Lk - Lq)[:, None]
            j = torch.arange(lo, hi, device=DEV)[None]
            hidden = (j > p) if c["causal"] else torch.zeros(e - r, hi - lo, dtype=torch.bool, device=DEV)
            if c["window"]:
                hidden = hidden | (j <= p - c["window"])
            yield slice(q0 + r, q0 + e), slice(k0 + lo, k0 + hi), hidden


def _by_kv_head(x, Hkv):
    """[rows, H, 128] as fp32 [Hkv, (H / Hkv) rows, 128]."""
    T, H = x.shape[:2]
    return x.float().view(T, Hkv, H // Hkv, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D)


def _by_row(x, T):
    """Its inverse."""
    Hkv = x.shape[0]
    return x.view(Hkv, -1, T, D).permute(2, 0, 1, 3).reshape(T, -1, D)


def _plain_attn_fwd(s):
    q, k, v = s["q"], s["k"], s["v"]
    T, Hq, Hkv = q.shape[0], q.shape[1], k.shape[1]
    o = torch.zeros(T, Hq, D, dtype=q.dtype, device=DEV)
    lse = torch.full((Hq, T), -math.inf, device=DEV)
    for rows, keys, hidden in _blocks(s):
        n, m = hidden.shape
        if not m:
            continue
        S = torch.bmm(_by_kv_head(q[rows], Hkv), _by_kv_head(k[keys], Hkv).transpose(1, 2)).mul_(D ** -0.5).view(Hkv, -1, n, m)
        S.masked_fill_(hidden, -math.inf)
        top = S.amax(-1, keepdim=True).clamp_min(-1e30)
        P = S.sub_(top).exp_()
        total = P.sum(-1, keepdim=True)
        lse[:, rows] = (top + total.log()).view(Hq, n)
        P.div_(total.clamp_min(1e-30))
        o[rows] = _by_row(torch.bmm(P.view(Hkv, -1, m), _by_kv_head(v[keys], Hkv)), n).to(q.dtype)
    return o, lse


def _plain_attn_bwd(s, o, lse):
    q, k, v = s["q"], s["k"], s["v"]
    Hq, Hkv, scale = q.shape[1], k.shape[1], D ** -0.5
    dq = torch.zeros(q.shape, dtype=q.dtype, device=DEV)
    dk, dv = (torch.zeros(Hkv, k.shape[0], D, device=DEV) for _ in range(2))
    for rows, keys, hidden in _blocks(s):
        n, m = hidden.shape
        if not m:
            continue
        Q, K, V, G = _by_kv_head(q[rows], Hkv), _by_kv_head(k[keys], Hkv), _by_kv_head(v[keys], Hkv), _by_kv_head(s["do"][rows], Hkv)
        delta = (G * _by_kv_head(o[rows], Hkv)).sum(-1, keepdim=True)
        L = lse[:, rows].reshape(Hkv, -1, 1)
        P = torch.bmm(Q, K.transpose(1, 2)).mul_(scale).view(Hkv, -1, n, m).masked_fill_(hidden, -math.inf).view(Hkv, -1, m)
        P = P.sub_(L.clamp_min(-1e30)).exp_()
        dv[:, keys] += torch.bmm(P.transpose(1, 2), G)
        dS = torch.bmm(G, V.transpose(1, 2)).sub_(delta).mul_(P)
        del P
        dq[rows] = _by_row(torch.bmm(dS, K) * scale, n).to(q.dtype)
        dk[:, keys] += torch.bmm(dS.transpose(1, 2), Q) * scale
    return dq, dk.transpose(0, 1).to(q.dtype), dv.transpose(0, 1).to(q.dtype)


def _plain_attn(s):
    mode, out, o, lse = s["case"]["mode"], {}, s.get("o"), s.get("lse")
    if mode != "bwd":
        o, lse = _plain_attn_fwd(s)
        out.update(o=o, lse=lse)
    if mode != "fwd":
        out["dq"], out["dk"], out["dv"] = _plain_attn_bwd(s, o, lse)
    return out


def _to_4bit(x):
    """Rows of 128 values as 64 bytes of code pairs (the even channel in the low half) and 4 exponents, biased by 127."""
    b = x.float().unflatten(-1, (D // 32, 32))
    frac, e = torch.frexp(b.abs().amax(-1, keepdim=True))  # max = frac 2^e, frac in [0.5, 1)
    e = torch.where(frac > 0.75, e - 2, e - 3).clamp(-126, 127)
    a = torch.ldexp(b.abs(), -e)
    # ties go to the even code: a value on a border below an even code rounds up to it
    code = (a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte()
    code = (code + 8 * (b < 0).byte()).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).byte().squeeze(-1)


def _from_4bit(codes, scale):
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    value = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=DEV)[code]
    return torch.ldexp(value.unflatten(-1, (D // 32, 32)), scale.int()[..., None] - 127).flatten(-2)


def _places(s, cu, start):
    """Page and row in it of every token of a packed batch whose sequences begin at `start`."""
    cu, T = cu.long(), int(s["T_all"]) if cu is s["cu_all"] else s["k"].shape[0]
    seq = torch.repeat_interleave(torch.arange(len(start), device=DEV), cu[1:] - cu[:-1], output_size=T)
    at = torch.arange(T, device=DEV) - cu[seq] + start[seq]
    page = s["case"]["page"]
    return s["table"][seq, at // page].long(), at % page


def _plain_kv(s):
    out = {}
    new, every = _places(s, s["cu_new"], s["past"]), _places(s, s["cu_all"], s["zero"])
    for side in ("k", "v"):
        codes, scale = s[side + "_codes"], s[side + "_scale"]
        codes[new[0], :, new[1]], scale[new[0], :, new[1]] = _to_4bit(s[side])
        out[side] = _from_4bit(codes[every[0], :, every[1]], scale[every[0], :, every[1]]).to(torch.bfloat16)
    return out


def _held(s, n, L, side):
    """The first L tokens of sequence n as [Hkv, L, 128]."""
    page, Hkv = s["case"]["page"], s["case"]["Hkv"]
    pages = s["table"][n, : -(-L // page)].long()
    x = _from_4bit(s[side + "_codes"][pages], s[side + "_scale"][pages])
    return x.transpose(0, 1).reshape(Hkv, -1, D)[:, :L]


def _plain_attend(s):
    c = s["case"]
    Hkv, o = c["Hkv"], torch.zeros(s["q"].shape, dtype=torch.bfloat16, device=DEV)
    row = 0
    for n, (L, run_) in enumerate(zip(_ints(c["lens"]), _runs(c))):
        if run_:
            rows = slice(row, row + run_)
            K, V = _held(s, n, L, "k"), _held(s, n, L, "v")
            S = torch.bmm(_by_kv_head(s["q"][rows], Hkv), K.transpose(1, 2)).mul_(D ** -0.5).view(Hkv, -1, run_, L)
            p, j = torch.arange(L - run_, L, device=DEV)[:, None], torch.arange(L, device=DEV)
            S.masked_fill_((j > p) | (j <= p - c["window"]) if c["window"] else j > p, -math.inf)
            P = S.sub_(S.amax(-1, keepdim=True)).exp_()
            P.div_(P.sum(-1, keepdim=True))
            o[rows] = _by_row(torch.bmm(P.view(Hkv, -1, L), V), run_).to(torch.bfloat16)
            row += run_
    return {"o": o}


# ---- the same in 64 bits -------------------------------------------------------------------------------------


def _exact_rope(s):
    c = s["case"]
    f, m = _freqs(c)
    angle = _positions(s)[:, None] * torch.tensor(f, dtype=torch.float64, device=DEV)
    turn = torch.polar(torch.full_like(angle, m), angle)[:, None]  # a rotation is a product with m e^(i angle)
    i = torch.arange(c["rot"] // 2, device=DEV)
    first, second = (i, i + c["rot"] // 2) if c["layout"] == "half" else (2 * i, 2 * i + 1)

    def product(x, by):
        if x is None:
            return None
        y = x.double()
        z = torch.complex(y[..., first], y[..., second]) * by
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {}
    if c["mode"] != "bwd":
        out["q"], out["k"] = product(s["q"], turn), product(s["k"], turn)
    if c["mode"] != "fwd":
        out["dq"], out["dk"] = product(s["dq"], turn.conj()), product(s["dk"], turn.conj())
    return out


def _exact_attn(s):
    c = s["case"]
    group, train = c["Hq"] // c["Hkv"], c["mode"] != "fwd"
    shape = {n: torch.zeros(s[n].shape, dtype=torch.float64, device=DEV) for n in ("q", "k", "v")}
    o, lse = torch.zeros_like(shape["q"]), torch.full((c["Hq"], s["q"].shape[0]), -math.inf, dtype=torch.float64, device=DEV)
    for n in range(len(s["cu_q"]) - 1):
        rows, keys = slice(s["cu_q"][n], s["cu_q"][n + 1]), slice(s["cu_k"][n], s["cu_k"][n + 1])
        Lq, Lk = rows.stop - rows.start, keys.stop - keys.start
        if not Lq or not Lk:
            continue
        seen = torch.ones(Lq, Lk, dtype=torch.bool, device=DEV)
        if c["causal"]:
            seen = seen.tril(Lk - Lq)
        if c["window"]:
            seen = seen.triu(Lk - Lq - c["window"] + 1)
        some = seen.any(1)
        for h in range(c["Hq"]):
            q, k, v = s["q"][rows, h].double(), s["k"][keys, h // group].double(), s["v"][keys, h // group].double()
            S = (q @ k.t() / math.sqrt(D)).masked_fill_(~seen, -math.inf)
            lse[h, rows] = torch.logsumexp(S, 1)
            P = S.sub_(lse[h, rows].masked_fill(~some, 0.0)[:, None]).exp_()
            o[rows, h] = P @ v
            if train:
                g = s["do"][rows, h].double()
                shape["v"][keys, h // group] += P.t() @ g
                dP = g @ v.t()
                dS = dP.sub_((P * dP).sum(1, keepdim=True)).mul_(P).div_(math.sqrt(D))
                shape["q"][rows, h] = dS @ k
                shape["k"][keys, h // group] += dS.t() @ q
                del dP, dS
            del S, P
    out = {}
    if c["mode"] != "bwd":
        out.update(o=o, lse=lse)
    if train:
        out.update({"d" + n: x for n, x in shape.items()})
    return out


def _exact_kv(s):
    """From the definition: the nearest of the format's values, by comparing with each."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    c, out = s["case"], {}
    past, new = _ints(c["past"]), _ints(c["new"])
    for side in ("k", "v"):
        x = s[side].double().reshape(-1, 32)
        top = x.abs().amax(1, keepdim=True)
        e = torch.ceil(torch.log2(top / 6.0)).clamp(min=-126.0)
        e = torch.where(top <= 6.0 * torch.exp2(e - 1), e - 1, e).clamp(min=-126.0)
        y = x.abs() / torch.exp2(e)
        near, best = torch.zeros_like(y), torch.full_like(y, math.inf)
        for i in (0, 2, 4, 6, 1, 3, 5, 7):  # even codes first: they keep the ties
            d = (y - grid[i]).abs()
            near, best = torch.where(d < best, grid[i], near), torch.minimum(d, best)
        stored = (near * torch.exp2(e) * torch.sign(x)).view(-1, c["Hkv"], D)
        held, at = [], 0
        for n, (a, b) in enumerate(zip(past, new)):
            if a:  # what was there before keeps its values
                held.append(_held(s, n, a, side).transpose(0, 1).double())
            held.append(stored[at : at + b])
            at += b
        out[side] = torch.cat(held)
    return out


def _exact_attend(s):
    c = s["case"]
    group, o, row = c["Hq"] // c["Hkv"], torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV), 0
    for n, (L, run_) in enumerate(zip(_ints(c["lens"]), _runs(c))):
        if not run_:
            continue
        K, V = (_held(s, n, L, side).double() for side in ("k", "v"))
        for i in range(run_):
            hi = L - run_ + i + 1
            lo = max(0, hi - c["window"]) if c["window"] else 0
            q = s["q"][row + i].double().view(c["Hkv"], group, 1, D)
            w = torch.softmax((q * K[:, None, lo:hi]).sum(-1) / math.sqrt(D), -1)
            o[row + i] = (w[..., None] * V[:, None, lo:hi]).sum(-2).view(c["Hq"], D)
        row += run_
    return {"o": o}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attn": _exact_attn, "kv": _exact_kv, "attend": _exact_attend}[case["op"]](s)


# ---- what a pass cannot do without -----------------------------------------------------------------------------


def _seen(case):
    """Pairs of a row and a key that it sees."""
    Lq = _ints(case["docs"])
    total = 0
    for n, m in zip(Lq, _ints(case["docs_k"]) or Lq):
        if not case["causal"]:
            total += n * m
            continue
        w = case["window"] or n + m
        most = lambda p: sum_to(p + 1) - sum_to(p + 1 - w)  # noqa: E731
        sum_to = lambda x: x * (x + 1) // 2 if x > 0 else 0  # noqa: E731
        total += most(m - 1) - most(m - n - 1)
    return total


def work(case):
    op = case["op"]
    if op == "rope":
        T, passes = _tokens(case), 2 if case["mode"] == "train" else 1
        size = 2 if case["dtype"] == "bf16" else 4
        heads = T * (case["Hq"] + case["Hk"])
        return {"bytes": passes * (2 * heads * D * size + 4 * T), "flops": passes * 3 * heads * case["rot"]}
    if op == "attn":
        Tq = sum(_ints(case["docs"]))
        Tk = sum(_ints(case["docs_k"]) or _ints(case["docs"]))
        q, kv = 2 * D * Tq * case["Hq"], 2 * D * Tk * case["Hkv"]
        each = {"fwd": (2 * q + 2 * kv + 4 * Tq * case["Hq"], 4), "bwd": (4 * q + 4 * kv + 4 * Tq * case["Hq"], 10)}
        parts = [each[m] for m in (("fwd", "bwd") if case["mode"] == "train" else (case["mode"],))]
        return {"bytes": sum(p[0] for p in parts), "flops": sum(p[1] for p in parts) * D * _seen(case) * case["Hq"]}
    if op == "kv":
        new = sum(_ints(case["new"])) * case["Hkv"]
        every = new + sum(_ints(case["past"])) * case["Hkv"]
        return {"bytes": 2 * (new + every) * (2 * D + D // 2 + D // 32), "flops": 0}
    rows = held = pairs = 0
    for L, r in zip(_ints(case["lens"]), _runs(case)):
        keys = min(L, case["window"] + r - 1) if case["window"] else L
        rows, held = rows + r, held + (keys if r else 0)
        pairs += sum(min(case["window"] or L, L - i) for i in range(r))
    return {"bytes": 2 * held * case["Hkv"] * (D // 2 + D // 32) + 4 * rows * case["Hq"] * D, "flops": 4 * D * pairs * case["Hq"]}
