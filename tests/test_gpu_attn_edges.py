"""Calls that the attention layers' documentation allows and that stand at its borders:
a side without heads, many heads to a kv head, thousands of tiny documents, one row with very many
keys, windows past everything, an output left out, extreme lengths and windows of the step."""
import pytest
import torch

import attn_ref as ref
import chunked_gated_delta_14_amd as gdr
from test_gpu_attn import BF, cu_of, fill, gen, heads, ints, pool

pytestmark = pytest.mark.gpu


def test_rope_without_query_heads():
    g = gen(1)
    k = heads(g, 33, 3)
    q = torch.empty(33, 0, 128, dtype=BF, device="cuda")
    pos = torch.arange(33, dtype=torch.int32, device="cuda") - 7  # positions may be negative
    freqs = gdr.rope_freqs(100)
    out = torch.empty_like(k)
    gdr.rope_fwd(gdr.RopeProblem(q, k, freqs, positions=pos), q, out)
    ref.check("k", out, *ref.rope(k, pos, freqs, True))


@pytest.mark.parametrize("docs,docs_k,Hq,Hkv,causal,window", [
    ([200, 31], None, 24, 1, True, 0), ([130], None, 64, 2, True, 0), ([1], [20000], 4, 2, True, 0), ([70, 70], None, 2, 1, True, 1 << 30),
    ([3, 2, 1, 0] * 700, None, 2, 1, True, 0), ([600], [5], 2, 2, True, 0),
])
def test_attention_borders(docs, docs_k, Hq, Hkv, causal, window):
    cu, ck = cu_of(docs), cu_of(docs_k or docs)
    g = gen(Hq + cu[-1])
    q, k, v, do = heads(g, cu[-1], Hq), heads(g, ck[-1], Hkv), heads(g, ck[-1], Hkv), heads(g, cu[-1], Hq).contiguous()
    p = gdr.AttnProblem(q, k, v, gdr.AttnPlan(cu, ck if docs_k else None, causal=causal, window=window))
    o, lse = torch.empty(cu[-1], Hq, 128, dtype=BF, device="cuda"), torch.empty(Hq, cu[-1], device="cuda")
    gdr.attn_fwd(p, o, lse)
    alone = torch.empty_like(o)
    gdr.attn_fwd(p, alone)  # without lse
    assert alone.equal(o)
    grads = [torch.empty(x.shape, dtype=BF, device="cuda") for x in (q, k, v)]
    gdr.attn_bwd(p, o, lse, do, *grads, p.alloc_workspace())
    want = ref.attention(q, k, v, cu, ck, causal, window, dout=do)
    for name, x in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
        ref.check(name, x, *want[name])


def test_shared_and_whole_tiles_agree():
    """Sums joined from parts against one block's, through the C entry without a workspace."""
    g, T = gen(3), 2600
    q, k, v = heads(g, T, 2), heads(g, T, 1), heads(g, T, 1)
    p = gdr.AttnProblem(q, k, v, gdr.AttnPlan([0, T]))
    assert p._fwd_bytes > 0
    o, lse, o2, lse2 = (torch.empty(*s, dtype=d, device="cuda") for s, d in (((T, 2, 128), BF), ((2, T), torch.float32)) * 2)
    gdr.attn_fwd(p, o, lse)
    stream = torch.cuda.current_stream().cuda_stream
    assert gdr.lib().gdr_attn_fwd(p.cstruct, o2.data_ptr(), lse2.data_ptr(), None, 0, stream) == 0
    # Probabilities are rounded to bf16 relative to the maximum that a block holds, which parts have of their own: a factor
    # 2^x between them, x no whole number, so P and P 2^x round apart, by up to 2^-8 of P each.  The two results
    # differ by up to both sides' bounds, not by one rounding of the output: each is held to its own.
    want = ref.attention(q, k, v, [0, T], [0, T])
    for a, b in ((o, lse), (o2, lse2)):
        ref.check("o", a, *want["o"])
        ref.check("lse", b, *want["lse"])


@pytest.mark.parametrize("window", [1, 2 ** 31 - 1])
def test_step_borders(window):
    g, lens, runs = gen(5), [5000, 40, 1], [2, 1, 1]
    cache, table = pool(g, lens, 1, 128)
    K, V = fill(g, cache, table, lens)
    q = heads(g, 4, 3)
    held = ints(lens)
    p = gdr.AttnStep(q, cache, table, held, ints(cu_of(runs)), window=window)
    o = torch.empty(4, 3, 128, dtype=BF, device="cuda")
    ws = p.alloc_workspace()
    gdr.attn_step(p, o, ws)
    ref.check("o", o, *ref.attention(q, K, V, cu_of(runs), cu_of(lens), True, window)["o"])
    held.copy_(ints([-5, 0, -(2 ** 31)]))  # sequences that hold nothing
    gdr.attn_step(p, o, ws)
    assert (o == 0).all()
