"""Host-side tests of the softmax-attention layers' operators: argument refusals (every
one before any device call, so without a GPU), the tile planner, rope frequencies,
workspace sizes, and the fp64 references' gradients against central differences."""
import ctypes
import math

import numpy as np
import pytest
import torch

import attn_ref as ref
import chunked_gated_delta_14_amd as gdr
from chunked_gated_delta_14_amd import attn

PTR, OUT, OUT2, OUT3 = 4096, 1 << 20, 1 << 21, 1 << 22  # never dereferenced
BIG = 1 << 40


def refused(rc, code, word):
    assert rc == code, (rc, gdr.lib().gdr_last_error().decode())
    assert word in gdr.lib().gdr_last_error().decode(), gdr.lib().gdr_last_error().decode()


def plan(docs, docs_k=None, causal=True, window=0):
    L, ip = gdr.lib(), ctypes.POINTER(ctypes.c_int32)
    cu = np.concatenate([[0], np.cumsum(docs)]).astype(np.int32)
    ck = cu if docs_k is None else np.concatenate([[0], np.cumsum(docs_k)]).astype(np.int32)
    p = attn._CAttnPlan()
    args = (cu.ctypes.data_as(ip), ck.ctypes.data_as(ip), len(docs), int(causal), window)
    assert L.gdr_plan_attn(*args, None, 0, ctypes.byref(p)) == 0
    table = np.zeros(max(p.table_len, 1), np.int32)
    assert L.gdr_plan_attn(*args, table.ctypes.data_as(ip), p.table_len, ctypes.byref(p)) == 0
    return p, table, cu, ck


def rope(**kw):
    f = dict(T=64, N=1, H_q=4, H_k=2, D=128, rot=64, dtype=0, layout=0, n_chunks=1, magnitude=1.0, q_stride=512, k_stride=256, q=PTR,
             k=PTR + 64, positions=None, chunk_table=PTR, freqs=PTR)
    f.update(kw)
    return attn._CRope(**f)


@pytest.mark.parametrize("kw,code,word", [
    (dict(T=-1), 1, "T and N"), (dict(H_q=-1), 1, "H_q and H_k"), (dict(H_q=1 << 17, q_stride=1 << 24), 2, "65536"), (dict(D=1), 1, "D must"),
    (dict(D=1026), 2, "1024"), (dict(rot=0), 1, "rot"), (dict(rot=63), 1, "rot"), (dict(rot=130), 1, "rot"), (dict(dtype=2), 1, "dtype"),
    (dict(layout=2), 1, "layout"), (dict(magnitude=float("nan")), 1, "magnitude"), (dict(freqs=None), 1, "freqs"),
    (dict(freqs=PTR + 4), 1, "aligned"), (dict(n_chunks=0), 1, "n_chunks"), (dict(n_chunks=3), 1, "n_chunks"),
    (dict(chunk_table=None), 1, "positions or chunk_table"), (dict(positions=PTR + 2, chunk_table=None), 1, "aligned"),
    (dict(T=1 << 30, positions=PTR), 2, "launch"),
])
def test_rope_refusals(kw, code, word):
    p = rope(**kw)
    s = 1 << 26
    refused(gdr.lib().gdr_rope_fwd(ctypes.byref(p), OUT, s, OUT2, s, None), code, word)
    refused(gdr.lib().gdr_rope_bwd(ctypes.byref(p), PTR, s, PTR + 64, s, OUT, s, OUT2, s, None), code, word)


def test_rope_call_refusals():
    L, p = gdr.lib(), rope()
    r = ctypes.byref(p)
    refused(L.gdr_rope_fwd(None, OUT, 512, OUT2, 256, None), 1, "NULL")
    refused(L.gdr_rope_fwd(r, None, 512, OUT2, 256, None), 1, "NULL")
    refused(L.gdr_rope_fwd(r, OUT, 511, OUT2, 256, None), 1, "stride")
    refused(L.gdr_rope_fwd(r, OUT, 512, OUT2 + 1, 256, None), 1, "aligned")
    refused(L.gdr_rope_fwd(r, PTR, 520, OUT2, 256, None), 1, "in place")
    refused(L.gdr_rope_fwd(r, OUT, 512, OUT, 256, None), 1, "other side")
    refused(L.gdr_rope_fwd(r, PTR + 64, 512, OUT2, 256, None), 1, "other side")
    refused(L.gdr_rope_bwd(r, OUT, 512, OUT2, 256, PTR, 512, OUT3, 256, None), 1, "is an input")


@pytest.mark.parametrize("args,word", [
    ((0, 1e4, 0, 1., 4096., 1., 32.), "rot"), ((3, 1e4, 0, 1., 4096., 1., 32.), "rot"), ((64, 0., 0, 1., 4096., 1., 32.), "base"),
    ((64, 1e4, 4, 1., 4096., 1., 32.), "scaling"), ((64, 1e4, 1, 0., 4096., 1., 32.), "factor"), ((64, 1e4, 3, 2., 0., 1., 32.), "original"),
    ((64, 1e4, 3, 2., 4096., 32., 32.), "low"), ((64, 1e4, 2, float("inf"), 4096., 1., 32.), "factor"),
])
def test_rope_freqs_refusals(args, word):
    buf = (ctypes.c_double * 600)()
    refused(gdr.lib().gdr_rope_freqs(*args, buf), 1, word)
    refused(gdr.lib().gdr_rope_freqs(64, 1e4, 0, 1., 1., 1., 2., None), 1, "NULL")


@pytest.mark.parametrize("rot", [2, 64, 128, 1024])
def test_rope_freqs(rot):
    i = np.arange(rot // 2)
    f = 1e4 ** (-2.0 * i / rot) / (2 * math.pi)
    get = lambda *a, **k: gdr.rope_freqs(rot, 1e4, *a, device="cpu", **k).numpy()  # noqa: E731
    np.testing.assert_allclose(get(), f, rtol=1e-14)
    np.testing.assert_allclose(get(gdr.GDR_ROPE_LINEAR, 4.0), f / 4, rtol=1e-14)
    base = 1e4 * 8 ** (rot / (rot - 2)) if rot > 2 else 1e4
    np.testing.assert_allclose(get(gdr.GDR_ROPE_BASE, 8.0), base ** (-2.0 * i / rot) / (2 * math.pi), rtol=1e-13)
    if rot > 2:  # the lowest frequency is the one that `linear` would give, the highest stays
        np.testing.assert_allclose(get(gdr.GDR_ROPE_BASE, 8.0)[[0, -1]], [f[0], f[-1] / 8], rtol=1e-13)
    c = np.clip((4096 * f - 1) / 31, 0, 1)
    np.testing.assert_allclose(get(gdr.GDR_ROPE_BLEND, 8.0, original=4096, low=1, high=32), f * ((1 - c) / 8 + c), rtol=1e-14)


@pytest.mark.parametrize("docs,docs_k,causal,window", [
    ([1], None, True, 0), ([0], None, True, 0), ([], None, True, 0), ([300, 0, 64, 1, 129, 2000], None, True, 0), ([300, 5], [40, 700], True, 0),
    ([300, 5, 7], [40, 700, 0], False, 0), ([1000, 30], None, True, 100), ([500, 40], [700, 3], True, 1), ([32674], None, True, 0),
])
def test_planner(docs, docs_k, causal, window):
    p, table, cu, ck = plan(docs, docs_k, causal, window)
    lk = docs if docs_k is None else docs_k
    assert p.n_q_tiles == sum(-(-n // 128) for n in docs) and p.n_k_tiles == sum(-(-n // 256) for n in lk)
    at = 0
    for side, n_tiles, mine, other, size in ((0, p.n_q_tiles, cu, ck, 128), (1, p.n_k_tiles, ck, cu, 256)):
        rows = table[at:at + 8 * n_tiles].reshape(-1, 8)
        at += 8 * n_tiles
        covered, costs = np.zeros(mine[-1], int), []
        for row0, n, other0, L, first, shift, begin, end in rows:
            covered[row0:row0 + n] += 1
            d = int(np.searchsorted(mine, row0, side="right")) - 1
            assert 1 <= n <= size and first == row0 - mine[d] and row0 + n <= mine[d + 1]
            assert other0 == other[d] and L == other[d + 1] - other[d] and shift == lk[d] - docs[d]
            assert 0 <= begin <= max(end, 0) and end <= L and begin % 64 == 0
            # every pair that is seen lies within
            seen = ref.seen_mask(docs[d], lk[d], causal, window, "cpu").numpy() if docs[d] * lk[d] < 3e6 else None
            if seen is not None:
                part = seen[first:first + n] if side == 0 else seen[:, first:first + n].T
                hit = np.flatnonzero(part.any(0))
                if len(hit):
                    assert begin <= hit[0] < begin + 64 and hit[-1] + 1 == end
                else:
                    assert begin >= end or not part.size or not seen.any() or end - begin <= 64
            costs.append(-(-(end - begin) // 64) if end > begin else 0)
        assert (covered == 1).all() and costs == sorted(costs, reverse=True)
        steps, longest = (p.k_steps, p.k_longest) if side else (p.q_steps, p.q_longest)
        assert steps == sum(costs) and longest == max(costs, default=0)
        if side == 0:
            q_costs = costs
    for items, costs in ((p.q_items, q_costs), (p.k_items, costs)):
        for level, n in enumerate(items):
            if not n:
                continue
            got = table[at:at + 2 * n].reshape(-1, 2)
            at += 2 * n
            want = {(t, x, parts) for t, c in enumerate(costs) for parts in [min(max(-(-c // (1 << level)), 1), 64)] for x in range(parts)}
            assert len(got) == len(want) and {(int(t), int(x) & 0xFFFF, int(x) >> 16) for t, x in got} == want
    assert at == p.table_len


def test_planner_refusals():
    L, ip = gdr.lib(), ctypes.POINTER(ctypes.c_int32)
    p = attn._CAttnPlan()

    def call(cu, ck=None, N=None, window=0, causal=1, table=None, capacity=0, out=ctypes.byref(p)):
        cu = np.asarray(cu, np.int32)
        ck = None if ck is None else np.asarray(ck, np.int32).ctypes.data_as(ip)
        return L.gdr_plan_attn(cu.ctypes.data_as(ip), ck, len(cu) - 1 if N is None else N, causal, window, table, capacity, out)

    refused(call([0, 5], N=-1), 1, "N must")
    refused(L.gdr_plan_attn(None, None, 1, 1, 0, None, 0, ctypes.byref(p)), 1, "cu_q is NULL")
    refused(call([1, 5]), 1, "must be 0")
    refused(call([0, 5, 3]), 1, "non-decreasing")
    refused(call([0, 5], [0, -1]), 1, "non-decreasing")
    refused(call([0, 5], window=-1), 1, "window")
    refused(call([0, 5], window=3, causal=0), 2, "causal")
    refused(call([0, (1 << 30) + 1]), 2, "2^30")
    refused(call([0, 5], out=None), 1, "plan is NULL")
    buf = (ctypes.c_int32 * 4)()
    refused(call([0, 5], table=buf, capacity=4), 1, "capacity")


def problem(docs=(300, 20), Hq=4, Hkv=2, **kw):
    p = plan(list(docs))[0]
    T = sum(docs)
    f = dict(T_q=T, T_k=T, N=len(docs), H_q=Hq, H_kv=Hkv, D=128, causal=1, window=0, plan=p, scale=0.1, q_stride=Hq * 128,
             k_stride=Hkv * 128, v_stride=Hkv * 128, q=PTR, k=PTR + 64, v=PTR + 128, tile_table=PTR + 256)
    f.update(kw)
    return attn._CAttn(**f)


def bwd(L, r, o=PTR, lse=PTR, dout=PTR, dq=OUT, dqs=512, dk=OUT2, dks=256, dv=OUT3, dvs=256, ws=1 << 23, n=BIG):
    return L.gdr_attn_bwd(r, o, lse, dout, dq, dqs, dk, dks, dv, dvs, ws, n, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(T_q=-1), 1, "T_q, T_k"), (dict(N=-1), 1, "N must"), (dict(Hq=0), 1, "head counts"), (dict(Hq=3), 2, "multiple"), (dict(D=64), 2, "D = 128"),
    (dict(window=-1), 1, "window"), (dict(window=4, causal=0), 2, "causal"), (dict(scale=0.0), 1, "scale"), (dict(scale=float("inf")), 1, "scale"), (dict(scale=1e30), 1, "scale"),
    (dict(scale=-1.0), 1, "scale"), (dict(scale=float("nan")), 1, "scale"), (dict(q=None), 1, "q must"), (dict(v=None), 1, "k and v"),
    (dict(tile_table=None), 1, "tile_table"), (dict(tile_table=PTR + 2), 1, "aligned"), (dict(q=PTR + 8), 1, "16-byte"), (dict(q_stride=516), 1, "16-byte"),
    (dict(k_stride=248), 1, "16-byte"), (dict(v_stride=1 << 24), 1, "16-byte"), (dict(T_k=1), 1, "plan"), (dict(T_q=600), 1, "plan"),
    (dict(T_q=(1 << 30) + 1), 2, "2^30"),
])
def test_attn_refusals(kw, code, word):
    L, p = gdr.lib(), problem(**kw)
    r = ctypes.byref(p)
    refused(L.gdr_attn_fwd(r, OUT, OUT2, None, 0, None), code, word)
    refused(bwd(L, r), code, word)
    refused(-L.gdr_attn_workspace_bytes(r, 1), code, word)


def test_attn_call_refusals():
    L, p = gdr.lib(), problem()
    r = ctypes.byref(p)
    refused(L.gdr_attn_fwd(None, OUT, OUT2, None, 0, None), 1, "NULL")
    refused(L.gdr_attn_fwd(r, None, OUT2, None, 0, None), 1, "o is NULL")
    refused(L.gdr_attn_fwd(r, OUT + 8, OUT2, None, 0, None), 1, "aligned")
    refused(L.gdr_attn_fwd(r, OUT, OUT2 + 2, None, 0, None), 1, "aligned")
    refused(L.gdr_attn_fwd(r, PTR, OUT2, None, 0, None), 1, "is an input")
    refused(L.gdr_attn_fwd(r, OUT, PTR + 256, None, 0, None), 1, "is an input")
    for word, kw in (("non-NULL", dict(lse=None)), ("non-NULL", dict(dk=None)), ("16-byte", dict(dout=PTR + 8)), ("16-byte", dict(dqs=500)),
                     ("16-byte", dict(dv=OUT3 + 4)), ("is an input", dict(dq=PTR + 64)), ("same memory", dict(dk=OUT3)), ("same memory", dict(dq=OUT2))):
        refused(bwd(L, r, **kw), 1, word)
    need = L.gdr_attn_workspace_bytes(r, 1)
    assert need > 0 and need % 256 == 0
    refused(bwd(L, r, n=need - 1), 3, "too small")
    refused(bwd(L, r, ws=None), 3, "NULL")
    refused(bwd(L, r, ws=(1 << 23) + 16), 3, "aligned")
    # few rows with many keys: the forward has a workspace, which may be left out but not short
    long = problem(docs=(20000,))
    fwd = L.gdr_attn_workspace_bytes(ctypes.byref(long), 0)
    assert fwd > 0 and fwd % 256 == 0
    refused(L.gdr_attn_fwd(ctypes.byref(long), OUT, OUT2, 1 << 23, fwd - 1, None), 3, "too small")
    bad = problem()
    bad.plan.q_items[3] = 1
    refused(L.gdr_attn_fwd(ctypes.byref(bad), OUT, OUT2, None, 0, None), 1, "plan")
    bad = problem()
    bad.plan.k_longest = 1000
    refused(L.gdr_attn_fwd(ctypes.byref(bad), OUT, OUT2, None, 0, None), 1, "plan")


def kv(**kw):
    f = dict(n_pages=10, page=16, H_kv=2, D=128, N=3, max_pages=4, k_codes=PTR, v_codes=PTR + 64, k_scale=PTR + 128, v_scale=PTR + 256, page_table=PTR + 512)
    f.update(kw)
    return attn._CKv(**f)


def step(**kw):
    f = dict(T=3, H_q=4, window=0, scale=0.1, q_stride=512, q=OUT2, lens=OUT3, cu_seqlens=None)
    f.update(kw)
    return attn._CAttnStep(**f)


@pytest.mark.parametrize("kw,code,word", [
    (dict(n_pages=-1), 1, "n_pages"), (dict(N=-1), 1, "N and"), (dict(page=17), 2, "page must"), (dict(page=0), 2, "page must"), (dict(H_kv=0), 1, "H_kv"),
    (dict(D=64), 2, "D = 128"), (dict(k_codes=None), 1, "pool"), (dict(v_scale=None), 1, "pool"), (dict(v_codes=PTR + 8), 1, "16-byte"),
    (dict(page_table=None), 1, "page_table"), (dict(page_table=PTR + 2), 1, "aligned"),
])
def test_kv_refusals(kw, code, word):
    L, c, p = gdr.lib(), kv(**kw), step()
    r = ctypes.byref(c)
    for fn in (L.gdr_kv_store, L.gdr_kv_load):
        refused(fn(r, 3, None, None, OUT, 256, OUT2, 256, None), code, word)
    refused(L.gdr_attn_step_fwd(r, ctypes.byref(p), OUT, 1 << 23, BIG, None), code, word)


def test_kv_call_refusals():
    L, c = gdr.lib(), kv()
    r = ctypes.byref(c)
    for fn in (L.gdr_kv_store, L.gdr_kv_load):
        refused(fn(None, 3, None, None, OUT, 256, OUT2, 256, None), 1, "NULL")
        refused(fn(r, -1, None, None, OUT, 256, OUT2, 256, None), 1, "T must")
        refused(fn(r, 4, None, None, OUT, 256, OUT2, 256, None), 1, "N must equal T")
        refused(fn(r, 3, None, None, None, 256, OUT2, 256, None), 1, "k and v")
        refused(fn(r, 3, None, None, OUT, 255, OUT2, 256, None), 1, "stride")
        refused(fn(r, 3, None, None, OUT, 256, OUT2 + 1, 256, None), 1, "aligned")
        refused(fn(r, 3, None, PTR + 2, OUT, 256, OUT2, 256, None), 1, "aligned")
        refused(fn(r, 1 << 30, PTR, None, OUT, 256, OUT2, 256, None), 2, "launch")
        refused(fn(r, 3, None, None, PTR, 256, OUT2, 256, None), 1, "is an input")
    refused(L.gdr_kv_load(r, 3, None, None, OUT, 256, OUT, 256, None), 1, "same memory")
    same = kv(v_codes=PTR)
    refused(L.gdr_kv_store(ctypes.byref(same), 3, None, None, OUT, 256, OUT2, 256, None), 1, "same memory")


@pytest.mark.parametrize("kw,code,word", [
    (dict(T=-1), 1, "T, N"), (dict(H_q=0), 1, "head counts"), (dict(H_q=3), 2, "multiple"), (dict(window=-1), 1, "window"), (dict(scale=0.0), 1, "scale"),
    (dict(T=4), 1, "N must equal T"), (dict(q_stride=500), 1, "q_stride"), (dict(q=None), 1, "q and o"), (dict(lens=None), 1, "lens"),
    (dict(q=OUT2 + 1), 1, "aligned"), (dict(lens=OUT3 + 2), 1, "aligned"), (dict(q=OUT), 1, "is an input"),
])
def test_step_refusals(kw, code, word):
    L, c, p = gdr.lib(), kv(), step(**kw)
    refused(L.gdr_attn_step_fwd(ctypes.byref(c), ctypes.byref(p), OUT, 1 << 23, BIG, None), code, word)


def test_step_workspace():
    L, c, p = gdr.lib(), kv(max_pages=4000, n_pages=12000), step()
    need = gdr.attn_step_workspace_bytes(3, 3, 4, 2, 4000, 16)
    assert need > 0 and need % 256 == 0
    refused(L.gdr_attn_step_fwd(ctypes.byref(c), ctypes.byref(p), OUT, 1 << 23, need - 1, None), 3, "too small")
    refused(L.gdr_attn_step_fwd(ctypes.byref(c), ctypes.byref(p), OUT + 8, 1 << 23, need, None), 1, "16 bytes")
    refused(L.gdr_attn_step_fwd(ctypes.byref(c), None, OUT, 1 << 23, need, None), 1, "NULL")
    assert gdr.attn_step_workspace_bytes(3, 3, 4, 2, 4, 16) == 0  # one block holds all that such a table can
    with pytest.raises(gdr.GdrError):
        gdr.attn_step_workspace_bytes(3, 3, 5, 2, 4, 16)
    with pytest.raises(gdr.GdrError):
        gdr.attn_step_workspace_bytes(3, 1 << 33, 4, 2, 4, 16)


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 5)])
def test_reference_gradients(causal, window):
    """The references' gradients against central differences."""
    g = torch.Generator().manual_seed(3)
    cu_q, cu_k = [0, 9, 9, 20], [0, 5, 7, 30]
    q, k, v, do = (torch.randn(n, h, 8, generator=g, dtype=torch.float64) for n, h in ((20, 4), (30, 2), (30, 2), (20, 4)))
    out = ref.attention(q, k, v, cu_q, cu_k, causal, window, dout=do)
    f = lambda: (ref.attention(q, k, v, cu_q, cu_k, causal, window)["o"][0] * do).sum().item()  # noqa: E731
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        for _ in range(12):
            i = tuple(int(torch.randint(0, n, (1,), generator=g)) for n in x.shape)
            at, h = x[i].item(), 1e-5
            x[i] = at + h
            up = f()
            x[i] = at - h
            down = f()
            x[i] = at
            assert abs((up - down) / (2 * h) - out[name][0][i].item()) < 1e-8


def test_reference_rope_gradient():
    g = torch.Generator().manual_seed(4)
    x, y = (torch.randn(5, 2, 12, generator=g, dtype=torch.float64) for _ in range(2))
    pos = torch.tensor([0, 1, 5, 100000, 2 ** 31 - 1])
    f = torch.tensor([0.3, 0.01, 1e-5], dtype=torch.float64)
    for half in (True, False):  # a linear map and its transpose
        a = (ref.rope(x, pos, f, half, 1.5)[0] * y).sum()
        b = (x * ref.rope(y, pos, f, half, 1.5, back=True)[0]).sum()
        assert abs(a - b) < 1e-12 * abs(a).clamp_min(1)


def test_reference_4bit():
    x = np.zeros((1, 128))
    x[0, :8] = [6, 5, 2.5, 0.25, -0.75, 3.5, -1.25, 1.75]
    x[0, 32] = 6.1
    x[0, 64] = np.inf
    value, scale, codes = ref.to_4bit(x)
    assert list(value[0, :8]) == [6, 4, 2, 0, -1, 4, -1, 2]  # ties to the even code
    assert value[0, 32] == 6 and list(scale[0]) == [127, 128, 255, 1] and np.isnan(value[0, 64:96]).all()
    assert codes[0, 0] == 7 | 6 << 4 and codes[0, 2] == (2 | 8) | 6 << 4
