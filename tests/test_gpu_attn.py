"""The softmax-attention layers' operators on the GPU against fp64 references, with
bounds counted in roundings (tests/attn_ref.py)."""
import math

import numpy as np
import pytest
import torch

import attn_ref as ref
import chunked_gated_delta_14_amd as gdr

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def heads(g, T, H, pad=0, dtype=BF, std=1.0):
    return (torch.randn(T, H * 128 + pad, generator=g, device="cuda") * std).to(dtype)[:, : H * 128].unflatten(1, (H, 128))


def cu_of(lens):
    return [0] + [int(x) for x in np.cumsum(lens)]


# ---- rotary positions ----


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("T,Hq,Hk,D,rot,pad", [(1, 16, 2, 128, 64, 0), (3, 1, 0, 128, 128, 0), (67, 5, 3, 128, 96, 13), (700, 2, 1, 64, 6, 8),
                                               (2500, 3, 1, 128, 2, 0), (41, 2, 2, 130, 130, 5), (9, 40, 40, 128, 30, 0), (5, 1, 1, 1024, 1022, 1)])
def test_rope_positions(dtype, layout, T, Hq, Hk, D, rot, pad):
    g = gen(T + rot)
    q = torch.randn(T, Hq * D + pad, generator=g, device="cuda").to(dtype)[:, : Hq * D].unflatten(1, (Hq, D))
    k = torch.randn(T, Hk * D + pad, generator=g, device="cuda").to(dtype)[:, : Hk * D].unflatten(1, (Hk, D)) if Hk else None
    pos = torch.randint(0, 2 ** 31 - 1, (T,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = 0
    freqs = gdr.rope_freqs(rot, 1e4)
    p = gdr.RopeProblem(q, k, freqs, positions=pos, layout=layout, magnitude=1.25)
    new = lambda x: torch.full(x.shape, float("nan"), dtype=dtype, device="cuda") if x is not None else None  # noqa: E731
    qo, ko = new(q), new(k)
    gdr.rope_fwd(p, qo, ko)
    for x, y in ((q, qo), (k, ko)):
        if x is not None:
            ref.check("fwd", y, *ref.rope(x, pos, freqs, layout == 0, 1.25))
    dq, dk = new(q), new(k)
    gdr.rope_bwd(p, q, k, dq, dk)
    for x, y in ((q, dq), (k, dk)):
        if x is not None:
            ref.check("bwd", y, *ref.rope(x, pos, freqs, layout == 0, 1.25, back=True))
    # in place, out of a wider buffer: bit for bit, and nothing beside it moves
    q2 = q.clone() if not pad else torch.as_strided(q, (T, Hq * D + pad), (Hq * D + pad, 1)).clone()[:, : Hq * D].unflatten(1, (Hq, D))
    p2 = gdr.RopeProblem(q2, None, freqs, positions=pos, layout=layout, magnitude=1.25)
    gdr.rope_fwd(p2, q2)
    assert q2.equal(qo)
    assert qo[..., rot:].equal(q[..., rot:])


@pytest.mark.parametrize("docs", [[1], [64, 1, 0, 65, 200, 7], [3000, 129]])
def test_rope_documents(docs):
    T = sum(docs)
    q = heads(gen(T), T, 3)
    freqs = gdr.rope_freqs(128, 5e5, gdr.GDR_ROPE_BLEND, 8.0)
    qo = torch.empty_like(q)
    gdr.rope_fwd(gdr.RopeProblem(q, None, freqs, plan=gdr.Plan(cu_of(docs))), qo)
    pos = torch.cat([torch.arange(n) for n in docs]).cuda()
    ref.check("q", qo, *ref.rope(q, pos, freqs, True))


# ---- attention over packed documents ----

CASES = [
    # docs, docs_k, Hq, Hkv, causal, window, pad
    ([1], None, 1, 1, True, 0, 0),
    ([2, 1, 0, 3], None, 2, 1, True, 0, 8),
    ([64], None, 2, 2, True, 0, 0),
    ([31, 32, 33, 63, 65, 127, 128, 129], None, 2, 1, True, 0, 64),
    ([257, 500], None, 4, 2, True, 0, 0),
    ([300], None, 3, 1, False, 0, 0),
    ([130, 70, 5], None, 6, 2, True, 1, 0),
    ([400, 129], None, 2, 1, True, 64, 0),
    ([700], None, 8, 1, True, 100, 8),
    ([5, 200, 64, 0, 3], [100, 200, 1, 7, 0], 4, 2, True, 0, 0),       # rows that see no key, a document without keys, one without rows
    ([5, 200, 64, 0, 3], [100, 200, 1, 7, 0], 2, 2, False, 0, 0),
    ([100, 40], [700, 20], 2, 1, True, 50, 0),
    ([1, 1, 1], [1000, 64, 65], 8, 2, True, 0, 0),
    ([1100], None, 2, 2, True, 0, 0),
    # few tiles with many steps: shared by several blocks
    ([2000, 30, 0, 700], None, 4, 1, True, 0, 64),
    ([40, 3], [5000, 1], 8, 2, True, 0, 0),
    ([1500], [2500], 2, 1, False, 0, 8),
    ([3000], None, 1, 1, True, 1500, 0),
]


def attn_inputs(case, seed=0):
    docs, docs_k, Hq, Hkv, causal, window, pad = case
    cu_q, cu_k = cu_of(docs), cu_of(docs if docs_k is None else docs_k)
    g = gen(seed + sum(docs) + Hq)
    q, k, v = heads(g, cu_q[-1], Hq, pad), heads(g, cu_k[-1], Hkv, pad), heads(g, cu_k[-1], Hkv, pad)
    return q, k, v, heads(g, cu_q[-1], Hq).contiguous(), cu_q, cu_k


@pytest.mark.parametrize("case", CASES)
def test_attention(case):
    docs, docs_k, Hq, Hkv, causal, window, pad = case
    q, k, v, do, cu_q, cu_k = attn_inputs(case)
    want = ref.attention(q, k, v, cu_q, cu_k, causal, window, dout=do)
    plan = gdr.AttnPlan(cu_q, None if docs_k is None else cu_k, causal=causal, window=window)
    p = gdr.AttnProblem(q, k, v, plan)
    o = torch.full((q.shape[0], Hq, 128), float("nan"), dtype=BF, device="cuda")
    lse = torch.full((Hq, q.shape[0]), float("nan"), device="cuda")
    gdr.attn_fwd(p, o, lse)
    ref.check("o", o, *want["o"])
    ref.check("lse", lse, *want["lse"])
    ws = p.alloc_workspace().fill_(0xFF)
    base = [torch.full((t.shape[0], t.shape[1] * 128 + pad), float("nan"), dtype=BF, device="cuda") for t in (q, k, v)]
    dq, dk, dv = (b[:, : t.shape[1] * 128].unflatten(1, (t.shape[1], 128)) for b, t in zip(base, (q, k, v)))
    gdr.attn_bwd(p, o, lse, do, dq, dk, dv, ws)
    for name, got in (("dv", dv), ("dq", dq), ("dk", dk)):
        ref.check(name, got, *want[name])
    for b, t in zip(base, (q, k, v)):
        assert torch.isnan(b[:, t.shape[1] * 128:]).all()
    # the same again, bit for bit
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    gdr.attn_fwd(p, o2, lse2)
    dq2, dk2, dv2 = (torch.empty(t.shape, dtype=BF, device="cuda") for t in (q, k, v))
    gdr.attn_bwd(p, o2, lse2, do, dq2, dk2, dv2, ws)
    for x, y in ((o, o2), (lse, lse2), (dq, dq2), (dk, dk2), (dv, dv2)):
        assert x.equal(y)


@pytest.mark.parametrize("docs,window,at", [([300, 40], 0, 130), ([300, 40], 0, 63), ([200, 90], 70, 64), ([1, 1, 129], 0, 1), ([700], 0, 699)])
def test_hidden_values_stay_hidden(docs, window, at):
    """An infinity or NaN in k or v reaches the rows that see it, in the channels that hold it, and no others."""
    cu, inf, nan = cu_of(docs), float("inf"), float("nan")
    g = gen(at)
    q, k, v = heads(g, cu[-1], 2), heads(g, cu[-1], 1), heads(g, cu[-1], 1)
    p = gdr.AttnPlan(cu, window=window)
    doc = next(n for n in range(len(docs)) if cu[n] <= at < cu[n + 1])
    sees = torch.zeros(cu[-1], dtype=torch.bool, device="cuda")
    sees[at: min(cu[doc + 1], at + window) if window else cu[doc + 1]] = True

    def forward(k, v):
        o, lse = torch.empty_like(q), torch.empty(2, cu[-1], device="cuda")
        gdr.attn_fwd(gdr.AttnProblem(q, k, v, p), o, lse)
        return o, lse

    o0, lse0 = forward(k, v)
    poison = {3: inf, 40: -inf, 77: nan, 127: inf}
    v1 = v.clone()
    for c, x in poison.items():
        v1[at, 0, c] = x
    o, lse = forward(k, v1)
    assert lse.equal(lse0) and o[~sees].equal(o0[~sees])
    for c in range(128):
        if c not in poison:
            assert torch.isfinite(o[sees, :, c]).all()
        elif poison[c] != poison[c]:
            assert torch.isnan(o[sees, :, c]).all()
        else:
            assert (o[sees, :, c] == poison[c]).all()
    k1 = k.clone()
    k1[at, 0, 5] = nan
    o, lse = forward(k1, v)
    assert o[~sees].equal(o0[~sees]) and lse[:, ~sees].equal(lse0[:, ~sees])
    assert torch.isnan(o[sees]).all() and torch.isnan(lse[:, sees]).all()


# ---- the cache in 4 bits ----


def pool(g, lens, H, page, spare=3):
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    at = cu_of(need)
    for n in range(len(lens)):
        table[n, : need[n]] = order[at[n]: at[n + 1]]
    cache = gdr.KvCache.empty(sum(need) + spare, H, page)
    for t in (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale):
        t.fill_(0xFF)  # what a page held before does not matter
    return cache, table


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def fill(g, cache, table, lens, std=1.0):
    """Stores random tokens for every sequence; returns the values held, fp64 [T, H, 128]."""
    T, H = sum(lens), cache.H_kv
    k, v = heads(g, T, H, std=std), heads(g, T, H, std=std)
    gdr.kv_store(gdr.KvProblem(cache, table, None, T, ints(cu_of(lens))), k, v)
    return [torch.from_numpy(ref.to_4bit(x.double().cpu().numpy())[0]).cuda() for x in (k, v)]


def test_code_layout():
    """Every code, every scale byte that a store gives, and how bytes hold them."""
    cache = gdr.KvCache.empty(16, 1, 16)
    table = torch.arange(16, dtype=torch.int32, device="cuda")[None]
    n = 253
    x = torch.zeros(n, 1, 128, dtype=torch.float64)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
    for t in range(n):
        x[t, 0] = grid.repeat(8) * 2.0 ** (t - 126)
    x = x.clamp(-torch.finfo(BF).max, torch.finfo(BF).max).to(BF).cuda()
    value, scale, codes = ref.to_4bit(x.double().cpu().numpy())
    p = gdr.KvProblem(cache, table, None, n, ints([0, n]))
    gdr.kv_store(p, x, x)
    got = cache.k_codes.view(256, 64)[:n].cpu().numpy()
    assert (cache.k_scale.view(256, 4)[:n].cpu().numpy() == scale[:, 0]).all()
    assert ((got ^ codes[:, 0]) & ~np.where(value[:, 0, 0::2] == 0, 0x08, 0) & ~np.where(value[:, 0, 1::2] == 0, 0x80, 0) == 0).all()
    y, z = torch.empty_like(x), torch.empty_like(x)
    gdr.kv_load(p, y, z)
    assert y.equal(z) and (y.double().cpu().numpy() == value).all()


@pytest.mark.parametrize("past,new,H,page,pad", [([0], [1], 1, 16, 0), ([0, 3, 15, 16, 100], [5, 0, 1, 33, 28], 3, 16, 8),
                                                 ([7, 200], [300, 1], 8, 64, 0), ([1000], [513], 2, 256, 5), ([31, 0], [1, 1], 4, 32, 0)])
def test_store_and_load(past, new, H, page, pad):
    g = gen(sum(new) + H)
    every = [a + b for a, b in zip(past, new)]
    cache, table = pool(g, every, H, page)
    K, V = heads(g, sum(every), H, pad), heads(g, sum(every), H, pad) * 30
    V[0, 0, 3], V[-1, H - 1, 100] = float("inf"), float("nan")
    cut = [slice(a, a + p) for a, p in zip(cu_of(every), past)]
    tail = [slice(a + p, a + p + n) for a, p, n in zip(cu_of(every), past, new)]
    for part, start, lens in ((cut, None, past), (tail, past, new)):
        k, v = (torch.cat([x[s] for s in part]) for x in (K, V))
        gdr.kv_store(gdr.KvProblem(cache, table, None if start is None else ints(start), sum(lens), ints(cu_of(lens))), k, v)
    k, v = (torch.full((sum(every), H * 128 + pad), 7.0, dtype=BF, device="cuda") for _ in range(2))
    kk, vv = (x[:, : H * 128].unflatten(1, (H, 128)) for x in (k, v))
    gdr.kv_load(gdr.KvProblem(cache, table, None, sum(every), ints(cu_of(every))), kk, vv)
    for got, x in ((kk, K), (vv, V)):
        want = ref.to_4bit(x.double().cpu().numpy())[0]
        assert np.array_equal(got.double().cpu().numpy(), want, equal_nan=True)
    assert (k[:, H * 128:] == 7).all()


def test_places_that_are_not_there():
    g = gen(5)
    cache, table = pool(g, [40, 40, 40, 40], 2, 16)
    table[1, 1], table[2, 0] = -1, cache.n_pages
    before = [t.clone() for t in (cache.k_codes, cache.k_scale)]
    k, v = heads(g, 100, 2), heads(g, 100, 2)
    # sequence 0 starts before its first place, 3 runs past its table; tokens 90.. belong to none; cu is out of [0, T] at its ends
    cu, start = ints([-5, 20, 50, 80, 90]), ints([-3, 0, 0, 45])
    p = gdr.KvProblem(cache, table, start, 100, cu)
    gdr.kv_store(p, k, v)
    want = {}
    for n, (a, b, s) in enumerate(((0, 20, -3), (20, 50, 0), (50, 80, 0), (80, 90, 45))):
        for t in range(a, b):
            at = s + t - a
            if 0 <= at < 48 and 0 <= table[n, at // 16].item() < cache.n_pages:
                want[t] = (table[n, at // 16].item(), at % 16)
    assert 0 < len(want) < 90
    value = ref.to_4bit(k.double().cpu().numpy())[0]
    y, z = (torch.full_like(k, 7.0) for _ in range(2))
    gdr.kv_load(p, y, z)
    touched = torch.zeros(cache.n_pages, 16, dtype=torch.bool, device="cuda")
    for t in range(100):
        if t in want:
            assert (y[t].double().cpu().numpy() == value[t]).all()
            touched[want[t]] = True
        else:
            assert (y[t] == 7).all() and (z[t] == 7).all()
    for x, b in zip((cache.k_codes, cache.k_scale), before):
        assert x.transpose(1, 2)[~touched].equal(b.transpose(1, 2)[~touched])


ATTEND = [
    # lens, runs, Hq, Hkv, page, window, pad
    ([1], None, 1, 1, 16, 0, 0),
    ([31, 32, 33, 1, 0, 127, 128, 129], None, 4, 2, 16, 0, 8),
    ([1000, 5, 300], None, 8, 1, 32, 0, 0),
    ([4096], None, 16, 2, 16, 0, 0),
    ([700, 64, 65], None, 32, 2, 64, 0, 13),
    ([3000, 20, 700], None, 6, 3, 128, 100, 0),
    ([5000, 1, 300], None, 40, 2, 256, 0, 0),       # more heads to a kv head than a product has columns
    ([100, 40, 3, 2000, 0], [4, 1, 8, 3, 2], 4, 2, 16, 0, 0),  # runs, one longer than what is held
    ([500, 33], [8, 0], 8, 1, 64, 20, 8),
    ([300, 260], [40, 1], 2, 2, 32, 0, 0),
]


@pytest.mark.parametrize("case", ATTEND)
def test_attention_step(case):
    lens, runs, Hq, Hkv, page, window, pad = case
    g = gen(sum(lens) + Hq)
    cache, table = pool(g, lens, Hkv, page)
    K, V = fill(g, cache, table, lens)
    rows = runs or [1] * len(lens)
    q = heads(g, sum(rows), Hq, pad)
    p = gdr.AttnStep(q, cache, table, ints(lens), ints(cu_of(rows)) if runs else None, window=window)
    o = torch.full((sum(rows), Hq, 128), float("nan"), dtype=BF, device="cuda")
    gdr.attn_step(p, o, p.alloc_workspace().fill_(0xFF))
    want = ref.attention(q, K, V, cu_of(rows), cu_of(lens), True, window)["o"]
    ref.check("o", o, *want)
    o2 = torch.empty_like(o)
    gdr.attn_step(p, o2, p.alloc_workspace())
    assert o.equal(o2)
