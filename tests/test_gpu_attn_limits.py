"""The attention layers' operators where a formula's terms cancel or leave the ordinary
range: rows that see one key, values in the cache that are not finite, long
documents among many short ones, scores far from zero, positions
whose angles come back to nearly nothing."""
import math
from fractions import Fraction

import pytest
import torch

import attn_ref as ref
import chunked_gated_delta_14_amd as gdr
from test_gpu_attn import BF, cu_of, gen, heads, ints, pool

pytestmark = pytest.mark.gpu


def both_ways(q, k, v, do, cu, ck, window=0):
    p = gdr.AttnProblem(q, k, v, gdr.AttnPlan(cu, ck, window=window))
    o, lse = torch.empty(q.shape, dtype=BF, device="cuda"), torch.empty(q.shape[1], q.shape[0], device="cuda")
    gdr.attn_fwd(p, o, lse)
    grads = [torch.empty(x.shape, dtype=BF, device="cuda") for x in (q, k, v)]
    gdr.attn_bwd(p, o, lse, do, *grads, p.alloc_workspace())
    return o, lse, grads


@pytest.mark.parametrize("docs,docs_k,Hq,Hkv,window", [
    ([1], None, 1, 1, 0), ([1] * 300, None, 4, 2, 0), ([300, 65], None, 6, 2, 1), ([257, 1, 3, 128, 1], None, 8, 8, 0),
    ([40, 1], [39 + 1, 900], 2, 1, 1), ([130, 5], [1, 5], 3, 1, 0), ([2000], None, 2, 1, 1),
])
def test_rows_that_see_one_key(docs, docs_k, Hq, Hkv, window):
    """Their probability is 1 and o is v, so dS = dO v - dO o is nothing: dq is zero, and dk where no other row sees the key."""
    cu, ck = cu_of(docs), cu_of(docs_k or docs)
    g = gen(sum(docs) + Hq)
    q, k, v, do = heads(g, cu[-1], Hq), heads(g, ck[-1], Hkv), heads(g, ck[-1], Hkv), heads(g, cu[-1], Hq).contiguous()
    o, lse, (dq, dk, dv) = both_ways(q, k, v, do, cu, ck, window)
    one, only, at = torch.zeros(cu[-1], dtype=torch.bool), torch.zeros(ck[-1], dtype=torch.bool), 0
    for n in range(len(docs)):
        Lk = ck[n + 1] - ck[n]
        seen = ref.seen_mask(docs[n], Lk, True, window, "cpu")
        rows = seen.sum(1) == 1
        one[cu[n]: cu[n + 1]] = rows
        only[ck[n]: ck[n + 1]] = ~(seen & ~rows[:, None]).any(0)
        for i in torch.nonzero(rows)[:, 0].tolist():
            j = ck[n] + int(seen[i].int().argmax())
            assert o[cu[n] + i].equal(v[j].repeat_interleave(Hq // Hkv, 0))
    assert one.any()
    assert (dq[one.cuda()] == 0).all()
    assert (dk[only.cuda()] == 0).all()
    want = ref.attention(q, k, v, cu, ck, True, window, dout=do)
    for name, x in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        ref.check(name, x, *want[name])


@pytest.mark.parametrize("lens,runs,Hq,Hkv,page,window,poison", [
    ([20], None, 2, 1, 16, 0, [7]),                                  # a token that every row sees
    ([12], [3], 2, 1, 16, 3, [7]),                                   # in the first row's window only
    ([12], [3], 2, 1, 16, 0, [11]),                                  # the last row's own
    ([300, 45], [8, 5], 4, 2, 16, 40, [254, 293, 299, 300 + 2, 300 + 41]),
    ([1000, 70], [6, 1], 16, 1, 64, 100, [0, 895, 897, 899, 996, 1000 + 69]),
    ([3000, 500], [1, 9], 6, 3, 128, 0, [5, 2999, 3000 + 495, 3000 + 33]),
    ([700], [30], 2, 2, 32, 25, list(range(640, 700, 7))),
])
@pytest.mark.parametrize("side", ["k", "v"])
def test_held_values_that_are_not_finite(lens, runs, Hq, Hkv, page, window, poison, side):
    """32 channels with a NaN or infinity among them read as NaN, in attention as in a load, and reach the rows that see their
    token and no others: a key all of a row's channels, a value its own 32."""
    g, rows = gen(sum(lens) + Hq), runs or [1] * len(lens)
    cache, table = pool(g, lens, Hkv, page)
    cu, held = cu_of(rows), cu_of(lens)
    x = {n: heads(g, held[-1], Hkv) for n in ("k", "v")}
    for i, t in enumerate(poison):
        x[side][t, i % Hkv, (37 * i + 5) % 128] = [float("nan"), float("inf"), -float("inf")][i % 3]
    every = gdr.KvProblem(cache, table, None, held[-1], ints(held))
    gdr.kv_store(every, x["k"], x["v"])
    K, V = torch.empty_like(x["k"]), torch.empty_like(x["v"])
    gdr.kv_load(every, K, V)
    q = heads(g, cu[-1], Hq)
    p = gdr.AttnStep(q, cache, table, ints(lens), ints(cu) if runs else None, window=window)
    o = torch.empty(cu[-1], Hq, 128, dtype=BF, device="cuda")
    gdr.attn_step(p, o, p.alloc_workspace().fill_(0xFF))
    nan = torch.zeros(cu[-1], Hkv, 128, dtype=torch.bool, device="cuda")
    for n in range(len(lens)):
        seen = ref.seen_mask(rows[n], lens[n], True, window, "cuda").float()
        bad = torch.isnan((K if side == "k" else V)[held[n]: held[n + 1]]).float()
        assert bad.sum() % 32 == 0
        if side == "k":
            bad = bad.amax(2, keepdim=True).expand(-1, -1, 128)
        nan[cu[n]: cu[n + 1]] = torch.mm(seen, bad.flatten(1)).unflatten(1, (Hkv, 128)) > 0
    nan = nan.repeat_interleave(Hq // Hkv, 1)
    assert nan.any() and torch.isnan(o).equal(nan)
    want, bound = ref.attention(q, K.nan_to_num(0.0), V.nan_to_num(0.0), cu, held, True, window)["o"]
    ref.check("o", o[~nan], want[~nan], bound[~nan])


@pytest.mark.parametrize("docs,docs_k,Hq,Hkv,window", [
    ([16] + [100, 7] * 20, [9000] + [100, 7] * 20, 4, 2, 0), ([1500, 1, 129], None, 3, 1, 0), ([70] + [1] * 50, [20000] + [1] * 50, 2, 1, 0),
    ([4000, 300], None, 2, 2, 700), ([5, 2500], [4000, 2600], 8, 1, 0),
])
def test_parts_stay_in_their_workspaces(docs, docs_k, Hq, Hkv, window):
    """Shared tiles, both ways, in workspaces of just the bytes asked for: right, and nothing behind them is touched."""
    cu, ck = cu_of(docs), cu_of(docs_k or docs)
    g = gen(cu[-1] + Hq)
    q, k, v, do = heads(g, cu[-1], Hq), heads(g, ck[-1], Hkv), heads(g, ck[-1], Hkv), heads(g, cu[-1], Hq).contiguous()
    plan = gdr.AttnPlan(cu, ck, window=window)
    first = gdr.AttnProblem(q, k, v, plan)
    assert first._fwd_bytes > 0

    def around(n):
        return torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device="cuda")

    fwd, bwd = around(first._fwd_bytes), around(first.workspace_bytes())
    first._fwd_ws = fwd
    p = gdr.AttnProblem(q, k, v, plan, share=first)
    assert p._fwd_ws is fwd
    o, lse = torch.empty(q.shape, dtype=BF, device="cuda"), torch.empty(Hq, cu[-1], device="cuda")
    gdr.attn_fwd(p, o, lse)
    grads = [torch.empty(x.shape, dtype=BF, device="cuda") for x in (q, k, v)]
    gdr.attn_bwd(p, o, lse, do, *grads, bwd[: p.workspace_bytes()])
    assert (fwd[p._fwd_bytes:] == 0xFF).all() and (bwd[p.workspace_bytes():] == 0xFF).all()
    want = ref.attention(q, k, v, cu, ck, True, window, dout=do)
    for name, x in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
        ref.check(name, x, *want[name])


def test_shared_workspaces():
    g, cu = gen(31), [0, 2000]
    q, k, v = heads(g, 2000, 4), heads(g, 2000, 2), heads(g, 2000, 2)
    plan, small = gdr.AttnPlan(cu), gdr.AttnPlan([0, 40])
    one = gdr.AttnProblem(q, k, v, plan)
    two = gdr.AttnProblem(k, q[:, :2].contiguous(), v, plan, share=gdr.AttnProblem(k, v, v, plan))
    for p in (one, two, gdr.AttnProblem(v, k, k, plan, share=one)):
        o, lse = torch.empty(p.q.shape, dtype=BF, device="cuda"), torch.empty(p.H_q, 2000, device="cuda")
        gdr.attn_fwd(p, o, lse)
        ref.check("o", o, *ref.attention(p.q, p.k, p.v, cu, cu)["o"])
    tiny = gdr.AttnProblem(q[:40], k[:40], v[:40], small)
    assert gdr.AttnProblem(q[:40], k[:40], v[:40], small, share=one)._fwd_ws is None
    with pytest.raises(gdr.GdrError, match="shared workspace"):
        gdr.AttnProblem(q, k, v, plan, share=tiny)


FAR = [(2.0 ** 63, -(2.0 ** 64)), (1.171875 * 2.0 ** 15, -1.5 * 2.0 ** 14), (1.171875 * 2.0 ** 15, 1.5 * 2.0 ** 14),
       (1.171875 * 2.0 ** 14, -1.5 * 2.0 ** 10), (1.171875 * 2.0 ** 14, 1.5 * 2.0 ** 10), (1.171875 * 2.0 ** 8, 1.5 * 2.0 ** 7)]


@pytest.mark.parametrize("a,b", FAR)
@pytest.mark.parametrize("T", [3, 300, 2600])
def test_scores_far_from_zero(T, a, b):
    """Scores of a b, up to 2^30, and one whose product with log2 e rounds nothing off, far below: all keys of a row count the same."""
    g, cu = gen(T), [0, T]
    q, k, v = (torch.zeros(T, h, 128, dtype=BF, device="cuda") for h in (2, 1, 1))
    q[..., 7], k[..., 7] = a, b
    v.copy_(torch.randint(-8, 9, v.shape, generator=g, device="cuda"))
    p = gdr.AttnProblem(q, k, v, gdr.AttnPlan(cu), scale=1.0)
    o, lse = torch.empty_like(q), torch.empty(2, T, device="cuda")
    gdr.attn_fwd(p, o, lse)
    count = torch.arange(1, T + 1, device="cuda").double()
    mean = v.double().cumsum(0) / count[:, None, None]

    def near(got, mean):  # one probability, rounded to bf16 for the products, times whole numbers: sums are exact; the quotient is rounded twice
        assert ((got.double() - mean).abs() <= (2.0 ** -7 + 2.0 ** -14) * mean.abs()).all()

    near(o, mean)
    assert ((lse.double() - a * b - count.log()).abs() <= abs(a * b) * 2.0 ** -21 + 2.0 ** -19).all()
    cache, table = pool(g, [T], 1, 16)
    every = gdr.KvProblem(cache, table, None, T, ints(cu))
    gdr.kv_store(every, k, v)
    K, V = torch.empty_like(k), torch.empty_like(v)
    gdr.kv_load(every, K, V)
    assert K.equal(k)
    s = gdr.AttnStep(q[-1:], cache, table, ints([T]), scale=1.0)
    one = torch.empty(1, 2, 128, dtype=BF, device="cuda")
    gdr.attn_step(s, one, s.alloc_workspace())
    near(one, V.double().mean(0))


def test_far_positions_keep_small_angles():
    """Angles by whole-number arithmetic from the frequencies given: far positions chosen so that p f_i comes within 2^-20 to 2^-30
    turns of a whole number, whose sine is then the angle, to a few roundings of itself."""
    freqs = gdr.rope_freqs(16, 10.0)
    exact = [Fraction(x) for x in freqs.tolist()]
    pos, g = [], torch.Generator().manual_seed(3)
    for f in exact:  # denominators of f's continued fraction: p f is nearly whole
        a, b, p0, p1 = f.numerator, f.denominator, 1, 0
        while b:
            a, b, p0, p1 = b, a % b, p1, (a // b) * p1 + p0
            if p1 >= 1 << 31:
                break
            pos += [p1] if p1 > 1 << 12 else []
    pos += torch.randint(0, 2 ** 31 - 1, (200,), generator=g).tolist() + [2 ** 31 - 1, -(2 ** 31)]
    T = len(pos)
    x = torch.zeros(T, 1, 16, device="cuda")
    x[..., :8] = 1.0  # (1, 0) becomes (cos, sin)
    y = torch.empty_like(x)
    gdr.rope_fwd(gdr.RopeProblem(x, None, freqs, positions=torch.tensor(pos, dtype=torch.int32, device="cuda")), y)
    small = 0
    for t, row in enumerate(y[:, 0].double().tolist()):
        for i, f in enumerate(exact):
            turns = pos[t] * f
            turns = float(turns - round(turns))
            small += abs(turns) < 2.0 ** -24
            # the fraction of a turn is rounded to fp32, which is relative to it (2 pi |turns| 2^-24 of angle, at most pi 2^-24), and sine and
            # cosine are good to 4 ulp; near zero turns the angle's error is the sine's, relative, and none of the cosine's
            for got, want in ((row[i], math.cos(2 * math.pi * turns)), (row[8 + i], math.sin(2 * math.pi * turns))):
                assert abs(got - want) <= 2.0 ** -21 * abs(want) + (math.pi * 2.0 ** -24 if abs(turns) > 0.125 else 0.0), (pos[t], i)
    assert small > 20, small
