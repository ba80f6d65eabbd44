"""The softmax-attention layers' operators as they are used: a layer forwards and
backwards out of one projection buffer, prompts and tokens through the cache, captured
graphs, other streams, far offsets, refusals of the binding."""
import pytest
import torch

import attn_ref as ref
import chunked_gated_delta_14_amd as gdr
from test_gpu_attn import BF, cu_of, fill, gen, heads, ints, pool

pytestmark = pytest.mark.gpu


def split(buf, *counts):
    out, at = [], 0
    for n in counts:
        out.append(buf[:, at * 128: (at + n) * 128].unflatten(1, (n, 128)))
        at += n
    return out


@pytest.mark.parametrize("docs,Hq,Hkv", [([70, 1, 300, 129], 4, 2), ([513], 2, 2)])
def test_layer_forwards_and_backwards(docs, Hq, Hkv):
    """Projection, rope in place, attention, and the way back into one gradient buffer, each step checked on what it was given."""
    T, cu = sum(docs), cu_of(docs)
    g = gen(T)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * 128, generator=g, device="cuda").to(BF)
    raw = qkv.clone()
    q, k, v = split(qkv, Hq, Hkv, Hkv)
    freqs = gdr.rope_freqs(96, 5e5)
    pos = torch.cat([torch.arange(n) for n in docs]).cuda()
    rp = gdr.RopeProblem(q, k, freqs, plan=gdr.Plan(cu))
    gdr.rope_fwd(rp, q, k)
    for x, y in zip(split(raw, Hq, Hkv, Hkv), (q, k)):
        ref.check("rope", y, *ref.rope(x, pos, freqs, True))
    assert v.equal(split(raw, Hq, Hkv, Hkv)[2])
    p = gdr.AttnProblem(q, k, v, gdr.AttnPlan(cu))
    o, lse = torch.empty(T, Hq, 128, dtype=BF, device="cuda"), torch.empty(Hq, T, device="cuda")
    gdr.attn_fwd(p, o, lse)
    do = heads(g, T, Hq).contiguous()
    dqkv = torch.full_like(qkv, float("nan"))
    dq, dk, dv = split(dqkv, Hq, Hkv, Hkv)
    gdr.attn_bwd(p, o, lse, do, dq, dk, dv, p.alloc_workspace())
    want = ref.attention(q, k, v, cu, cu, dout=do)
    for name, x in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        ref.check(name, x, *want[name])
    mid = dqkv.clone()
    gdr.rope_bwd(rp, dq, dk, dq, dk)
    for x, y in zip(split(mid, Hq, Hkv, Hkv), (dq, dk)):
        ref.check("rope backward", y, *ref.rope(x, pos, freqs, True, back=True))
    assert torch.isfinite(dqkv).all()




def test_prompts_then_tokens_in_a_graph():
    """A decode step (rope, store, attention) on static buffers, captured once and replayed; every replay against the
    reference on what the cache then holds, and against the eager step."""
    lens, Hq, Hkv, page, steps = [100, 1, 0, 333, 64], 8, 2, 32, 5
    N, g = len(lens), gen(9)
    cache, table = pool(g, [n + steps + 1 for n in lens], Hkv, page)
    fill(g, cache, table, lens)
    freqs = gdr.rope_freqs(64, 1e6)
    qkv = torch.empty(N, (Hq + 2 * Hkv) * 128, dtype=BF, device="cuda")
    q, k, v = split(qkv, Hq, Hkv, Hkv)
    start, held = ints(lens), ints([n + 1 for n in lens])
    rp = gdr.RopeProblem(q, k, freqs, positions=start)
    store = gdr.KvProblem(cache, table, start, N)
    step = gdr.AttnStep(q, cache, table, held)
    ws = step.alloc_workspace()
    o = torch.zeros(N, Hq, 128, dtype=BF, device="cuda")

    def run():
        gdr.rope_fwd(rp, q, k)
        gdr.kv_store(store, k, v)
        gdr.attn_step(step, o, ws)

    tokens = [torch.randn(N, qkv.shape[1], generator=g, device="cuda").to(BF) for _ in range(steps)]
    state = [t.clone() for t in (cache.k_codes, cache.k_scale, cache.v_codes, cache.v_scale)]
    eager = []
    for t in range(steps):
        qkv.copy_(tokens[t])
        run()
        eager.append(o.clone())
        total = [n + t + 1 for n in lens]
        K, V = (torch.empty(sum(total), Hkv, 128, dtype=BF, device="cuda") for _ in range(2))
        gdr.kv_load(gdr.KvProblem(cache, table, None, sum(total), ints(cu_of(total))), K, V)
        ref.check("o", o, *ref.attention(q, K, V, cu_of([1] * N), cu_of(total))["o"])
        start += 1
        held += 1
    for t, s in zip((cache.k_codes, cache.k_scale, cache.v_codes, cache.v_scale), state):
        t.copy_(s)
    start.copy_(ints(lens))
    held.copy_(ints([n + 1 for n in lens]))
    qkv.copy_(tokens[0])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run()
    for t in range(steps):
        qkv.copy_(tokens[t])
        o.zero_()
        graph.replay()
        assert o.equal(eager[t]), "replay %d" % t
        torch.cuda.synchronize()
        start += 1
        held += 1


def test_training_in_a_graph_and_on_another_stream():
    docs, Hq, Hkv = [1500, 40, 7], 4, 1  # long enough to be shared by several blocks
    cu, g = cu_of(docs), gen(11)
    T = cu[-1]
    q, k, v, do = heads(g, T, Hq), heads(g, T, Hkv), heads(g, T, Hkv), heads(g, T, Hq).contiguous()
    p = gdr.AttnProblem(q, k, v, gdr.AttnPlan(cu))
    assert p._fwd_bytes > 0
    ws = p.alloc_workspace()

    def outputs():
        return [torch.empty(T, Hq, 128, dtype=BF, device="cuda"), torch.empty(Hq, T, device="cuda")] + [
            torch.empty(T, h, 128, dtype=BF, device="cuda") for h in (Hq, Hkv, Hkv)]

    def run(out, stream=None):
        gdr.attn_fwd(p, out[0], out[1], stream=stream)
        gdr.attn_bwd(p, out[0], out[1], do, *out[2:], ws, stream=stream)

    want, other, got = outputs(), outputs(), outputs()
    run(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    run(other, side)
    side.synchronize()
    assert all(x.equal(y) for x, y in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(got)
    base = [t.clone() for t in (q, k, v, do)]
    for t in range(3):
        for x in got:
            x.zero_()
        for x, b in zip((q, k, v, do), base):
            x.copy_(b * (t + 1) * 0.5)
        run(want)
        graph.replay()
        torch.cuda.synchronize()
        assert all(x.equal(y) for x, y in zip(want, got)), "replay %d" % t


def test_far_offsets():
    """Rows 16 MB apart, so that a batch spans more than 4 GB, and pages past 4 GB of a pool."""
    g, T, stride = gen(13), 300, 1 << 23
    far = torch.empty(T, stride, dtype=BF, device="cuda")
    far[:, : 4 * 128] = torch.randn(T, 4 * 128, generator=g, device="cuda").to(BF)
    q, k, v = split(far, 2, 1, 1)
    near = [x.clone() for x in (q, k, v)]
    freqs = gdr.rope_freqs(128)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    do = heads(g, T, 2).contiguous()
    results = []
    for a, b, c in ((q, k, v), near):
        gdr.rope_fwd(gdr.RopeProblem(a, b, freqs, positions=pos), a, b)
        p = gdr.AttnProblem(a, b, c, gdr.AttnPlan([0, T]))
        o, lse = torch.empty(T, 2, 128, dtype=BF, device="cuda"), torch.empty(2, T, device="cuda")
        gdr.attn_fwd(p, o, lse)
        gdr.attn_bwd(p, o, lse, do, *(grads := [torch.empty(x.shape, dtype=BF, device="cuda") for x in near]), p.alloc_workspace())
        results.append([a.clone(), b.clone(), o, lse, *grads])
    assert all(x.equal(y) for x, y in zip(*results))
    del far, q, k, v, a, b, c, p
    torch.cuda.empty_cache()
    n_pages = (1 << 32) // (2 * 256 * 64) + 40  # 4 GB of codes and 40 pages
    cache = gdr.KvCache(*(torch.empty(n_pages, 2, 256, w, dtype=torch.uint8, device="cuda") for w in (64, 4, 64, 4)))
    table = ints([[n_pages - 1, 3, n_pages - 20], [0, n_pages - 7, n_pages // 2]])
    lens = [700, 513]
    K, V = fill(g, cache, table, lens)
    qq = heads(g, 2, 4)
    s = gdr.AttnStep(qq, cache, table, ints(lens))
    o = torch.empty(2, 4, 128, dtype=BF, device="cuda")
    gdr.attn_step(s, o, s.alloc_workspace())
    ref.check("o", o, *ref.attention(qq, K, V, [0, 1, 2], cu_of(lens))["o"])


def test_pages_that_are_not_there_are_hidden():
    g, lens = gen(15), [200, 90]
    cache, table = pool(g, lens, 2, 32)
    K, V = fill(g, cache, table, lens)
    table[0, 2], table[1, 0] = -1, cache.n_pages + 5
    keep = torch.ones(290, dtype=torch.bool, device="cuda")
    keep[64:96] = False
    keep[200:232] = False
    q = heads(g, 2, 4)
    p = gdr.AttnStep(q, cache, table, ints([200, 9999]))  # more than the table holds: clipped to its 224 places
    o = torch.empty(2, 4, 128, dtype=BF, device="cuda")
    gdr.attn_step(p, o, p.alloc_workspace())
    want = ref.attention(q[:1], K[:200][keep[:200]], V[:200][keep[:200]], [0, 1], [0, 168])["o"]
    ref.check("o", o[:1], *want)
    table.fill_(-1)
    gdr.attn_step(p, o, p.alloc_workspace())
    assert (o == 0).all()


def test_rows_without_a_sequence_stay():
    g, lens = gen(17), [50, 70, 20]
    cache, table = pool(g, lens, 1, 16)
    K, V = fill(g, cache, table, lens)
    q = heads(g, 9, 2)
    o = torch.full((9, 2, 128), 7.0, dtype=BF, device="cuda")
    p = gdr.AttnStep(q, cache, table, ints(lens), ints([1, 3, 3, 6]))  # rows 0 and 6.. belong to none, sequence 1 has none
    gdr.attn_step(p, o, p.alloc_workspace())
    assert (o[0] == 7).all() and (o[6:] == 7).all()
    want = ref.attention(torch.cat([q[1:3], q[3:6]]), torch.cat([K[:50], K[120:]]), torch.cat([V[:50], V[120:]]), [0, 2, 5], [0, 50, 70])["o"]
    ref.check("o", o[1:6], *want)


def test_stale_pages_hold_anything():
    """What lies behind a sequence's last token in its page, NaN scales among it, does not matter."""
    g, lens = gen(19), [17, 33, 1]
    cache, table = pool(g, lens, 2, 64)  # filled with 0xFF: every scale a NaN
    K, V = fill(g, cache, table, lens)
    q = heads(g, 3, 8)
    p = gdr.AttnStep(q, cache, table, ints(lens))
    o = torch.empty(3, 8, 128, dtype=BF, device="cuda")
    gdr.attn_step(p, o, p.alloc_workspace())
    ref.check("o", o, *ref.attention(q, K, V, [0, 1, 2, 3], cu_of(lens))["o"])


@pytest.mark.parametrize("scale", [1e-3, 1.0, 30.0])
def test_scores_of_any_size(scale):
    """Nearly even and nearly one-hot probabilities, and scores far beyond exp's range."""
    g, cu = gen(21), [0, 200, 270]
    q, k, v, do = heads(g, 270, 2), heads(g, 270, 1), heads(g, 270, 1), heads(g, 270, 2).contiguous()
    p = gdr.AttnProblem(q, k, v, gdr.AttnPlan(cu), scale=scale)
    o, lse = torch.empty_like(q).contiguous(), torch.empty(2, 270, device="cuda")
    gdr.attn_fwd(p, o, lse)
    grads = [torch.empty(x.shape, dtype=BF, device="cuda") for x in (q, k, v)]
    gdr.attn_bwd(p, o, lse, do, *grads, p.alloc_workspace())
    want = ref.attention(q, k, v, cu, cu, scale=scale, dout=do)
    for name, x in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
        ref.check(name, x, *want[name])


def test_nothing_to_do():
    e = lambda *s, dtype=BF: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    freqs = gdr.rope_freqs(64)
    gdr.rope_fwd(gdr.RopeProblem(e(0, 2, 128), None, freqs, positions=e(0, dtype=torch.int32)), e(0, 2, 128))
    p = gdr.AttnProblem(e(0, 2, 128), e(0, 1, 128), e(0, 1, 128), gdr.AttnPlan([0, 0]))
    gdr.attn_fwd(p, e(0, 2, 128), e(2, 0, dtype=torch.float32))
    gdr.attn_bwd(p, e(0, 2, 128), e(2, 0, dtype=torch.float32), e(0, 2, 128), e(0, 2, 128), e(0, 1, 128), e(0, 1, 128), p.alloc_workspace())
    # keys without queries: their gradients are zeros
    p = gdr.AttnProblem(e(0, 2, 128), e(5, 1, 128).zero_(), e(5, 1, 128).zero_(), gdr.AttnPlan([0, 0], [0, 5]))
    dk, dv = e(5, 1, 128).fill_(7), e(5, 1, 128).fill_(7)
    gdr.attn_bwd(p, e(0, 2, 128), e(2, 0, dtype=torch.float32), e(0, 2, 128), e(0, 2, 128), dk, dv, p.alloc_workspace())
    assert (dk == 0).all() and (dv == 0).all()
    cache = gdr.KvCache.empty(0, 1)
    gdr.kv_store(gdr.KvProblem(cache, e(0, 4, dtype=torch.int32), None, 0), e(0, 1, 128), e(0, 1, 128))
    s = gdr.AttnStep(e(2, 1, 128).zero_(), cache, ints([[0, 0], [0, 0]]), ints([5, 5]))  # a pool without pages
    o = e(2, 1, 128).fill_(7)
    gdr.attn_step(s, o, s.alloc_workspace())
    assert (o == 0).all()


def test_binding_refusals():
    g = gen(23)
    q, k = heads(g, 10, 2), heads(g, 10, 1)
    freqs, plan = gdr.rope_freqs(64), gdr.AttnPlan([0, 10])
    pos = torch.arange(10, dtype=torch.int32, device="cuda")

    def refuses(word, f):
        with pytest.raises(gdr.GdrError, match=word):
            f()

    refuses("on a GPU", lambda: gdr.RopeProblem(q.cpu(), None, freqs, positions=pos))
    refuses("int32", lambda: gdr.RopeProblem(q, None, freqs, positions=pos.long()))
    refuses("either", lambda: gdr.RopeProblem(q, None, freqs))
    refuses("float64", lambda: gdr.RopeProblem(q, None, freqs.float(), positions=pos))
    refuses("shape", lambda: gdr.RopeProblem(q, k[:5], freqs, positions=pos))
    refuses("bfloat16 or float32", lambda: gdr.RopeProblem(q.half(), None, freqs, positions=pos))
    refuses("10 tokens|holds", lambda: gdr.RopeProblem(q, None, freqs, plan=gdr.Plan([0, 9])))
    rp = gdr.RopeProblem(q, k, freqs, positions=pos)
    refuses("k_out is None", lambda: gdr.rope_fwd(rp, q))
    refuses("shape", lambda: gdr.rope_fwd(rp, k, k))
    refuses("holds", lambda: gdr.AttnProblem(q[:9], k, k, plan))
    refuses("bfloat16", lambda: gdr.AttnProblem(q.float(), k, k, plan))
    refuses("16-byte", lambda: gdr.AttnProblem(torch.empty(10, 260, dtype=BF, device="cuda")[:, 4:].unflatten(1, (2, 128)), k, k, plan))
    refuses("16-byte", lambda: gdr.AttnProblem(torch.empty(10, 260, dtype=BF, device="cuda")[:, :256].unflatten(1, (2, 128)), k, k, plan))
    refuses("multiple", lambda: gdr.AttnProblem(heads(g, 10, 3), heads(g, 10, 2), heads(g, 10, 2), plan))
    refuses("causal", lambda: gdr.AttnPlan([0, 10], causal=False, window=5))
    refuses("N\\+1", lambda: gdr.AttnPlan([0, 10], [0, 5, 10]))
    p = gdr.AttnProblem(q, k, k, plan)
    o, lse = torch.empty_like(q), torch.empty(2, 10, device="cuda")
    refuses("is an input", lambda: gdr.attn_fwd(p, q, lse))
    refuses("float32", lambda: gdr.attn_fwd(p, o, lse.double()))
    refuses("too small", lambda: gdr.attn_bwd(p, o, lse, o.clone(), q.clone(), k.clone(), k.clone(), torch.empty(64, dtype=torch.uint8, device="cuda")))
    cache, table = gdr.KvCache.empty(4, 1, 16), ints([[0, 1], [2, 3]])
    refuses("page must", lambda: gdr.kv_store(gdr.KvProblem(gdr.KvCache.empty(4, 1, 24), table, None, 2), k[:2], k[:2]))
    refuses("uint8", lambda: gdr.KvCache(cache.k_codes.int(), cache.k_scale, cache.v_codes, cache.v_scale))
    refuses("shape", lambda: gdr.KvCache(cache.k_codes, cache.k_scale[:3], cache.v_codes, cache.v_scale))
    refuses("int32", lambda: gdr.KvProblem(cache, table.long(), None, 2))
    refuses("N must equal T", lambda: gdr.kv_store(gdr.KvProblem(cache, table, None, 3), k[:3], k[:3]))
    refuses("shape", lambda: gdr.kv_store(gdr.KvProblem(cache, table, None, 2), q[:2], q[:2]))
    refuses("shape", lambda: gdr.AttnStep(q[:2], cache, table, ints([1])))
    refuses("N must equal T", lambda: gdr.attn_step(s := gdr.AttnStep(q[:3], cache, table, ints([1, 1])), torch.empty_like(q[:3]), s.alloc_workspace()))
