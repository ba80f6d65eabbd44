"""The attention layers' operators where a formula's terms cancel or leave the ordinary
range: rows that see one key."""
import pytest
import torch

import attn_ref as ref
import chunked_gated_delta_14_amd as gdr
from test_gpu_attn import BF, cu_of, gen, heads

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
