"""Host-side limits of the softmax-attention layers' operators, without a GPU: every
refusal here stands for sizes that the kernels' 32-bit arithmetic would not hold."""
import ctypes
import random

import numpy as np
import pytest
import torch

import chunked_gated_delta_14_amd as gdr
from test_attn_host import BIG, OUT, kv, plan, problem, refused, step


@pytest.mark.parametrize("page,max_pages,T", [(256, 1 << 23, 3), (16, (1 << 26) + 1, 3), (256, (1 << 31) - 1, 3), (16, 4, (1 << 30) + 1)])
def test_step_places_past_32_bits(page, max_pages, T):
    """Places are held with 32 bits, up to a block's share past the last: tables of more than 2^30 places are refused."""
    L, c, p = gdr.lib(), kv(page=page, max_pages=max_pages, N=T), step(T=T)
    refused(L.gdr_attn_step_fwd(ctypes.byref(c), ctypes.byref(p), OUT, 1 << 23, BIG, None), 2, "2^30")
    refused(-L.gdr_attn_step_workspace_bytes(T, T, 4, 2, max_pages, page), 2, "2^30")
    assert L.gdr_attn_step_workspace_bytes(3, 3, 4, 2, (1 << 30) // page, page) > 0


LONG_AMONG_SHORT = [  # rows, keys, query heads, kv heads
    ([16] + [512] * 120, [200000] + [512] * 120, 16, 4), ([1] + [2000] * 30, [128000] + [2000] * 30, 8, 2),
    ([300] + [64] * 2000, [65536] + [64] * 2000, 8, 2), ([32768] + [64] * 3500, None, 4, 1), ([8192], None, 16, 4),
    ([1] + [64] * 256, [131072] + [64] * 256, 32, 8), ([128] + [100] * 2000, [1 << 20] + [100] * 2000, 8, 1), ([128] + [512] * 16, [131072] + [512] * 16, 16, 4),
]


@pytest.mark.parametrize("docs,docs_k,Hq,Hkv", LONG_AMONG_SHORT)
def test_workspaces_hold_parts_not_batches(docs, docs_k, Hq, Hkv):
    """Slots and heads: at most 2731 of 65 KB for queries, 1024 of 256 KB for keys, whatever else the batch holds."""
    L, (c, _, cu, ck) = gdr.lib(), plan(docs, docs_k)
    p = problem(Hq=Hq, Hkv=Hkv, T_q=int(cu[-1]), T_k=int(ck[-1]), N=len(docs), plan=c)
    fwd, bwd = (L.gdr_attn_workspace_bytes(ctypes.byref(p), i) for i in (0, 1))
    assert 0 < fwd <= 2731 * 65 * 1024
    assert bwd <= 2 * (4 * int(cu[-1]) * Hq + 255) + 2731 * 64 * 1024 + 1024 * 256 * 1024


def test_lists_of_parts():
    """Every part of every tile once, a tile's parts in a row, and all of several parts within the slots that a workspace has."""
    r = random.Random(5)
    for _ in range(150):
        n = r.randint(0, 6)
        docs = [r.choice([0, 1, r.randint(1, 700), r.randint(1, 3000)]) for _ in range(n)]
        docs_k = [r.choice([0, x, r.randint(1, 20000)]) for x in docs] if r.random() < 0.7 else None
        causal = r.random() < 0.8
        p, table, _, _ = plan(docs, docs_k, causal, r.randint(1, 5000) if causal and r.random() < 0.4 else 0)
        tiles = (p.n_q_tiles, p.n_k_tiles)
        at, first = 8 * sum(tiles), 0
        for items, count in zip((p.q_items, p.k_items), tiles):
            entries = table[8 * first: 8 * (first + count)].reshape(-1, 8)
            steps = [max(0, -(-int(e[7] - e[6]) // 64)) for e in entries]
            first += count
            for level, m in enumerate(items):
                rows = table[at: at + 2 * m].reshape(-1, 2)
                at += 2 * m
                seen, i, last = set(), 0, 0
                while i < m:
                    tile, parts = int(rows[i, 0]), int(rows[i, 1]) >> 16
                    assert 0 <= tile < count and tile not in seen
                    assert parts == min(max(-(-steps[tile] // (1 << level)), 1), 64)
                    assert [(int(t), int(x) & 0xFFFF, int(x) >> 16) for t, x in rows[i: i + parts]] == [(tile, x, parts) for x in range(parts)]
                    seen.add(tile)
                    i += parts
                    last = i if parts > 1 else last
                assert len(seen) == (count if m else 0)
                assert last <= (2 * sum(steps)) // (1 << level)
        assert at == p.table_len


@pytest.mark.parametrize("cu", [
    torch.tensor([0, (1 << 32) + 5, (1 << 32) + 9]), np.array([0, 5, (1 << 33) + 9]), [0, 5, 1 << 40], np.array([0, -(1 << 32), 9]), [0, 2.5, 9.9],
    torch.tensor([0.0, 5.0, 9.0]),
])
def test_plan_takes_ints_of_32_bits(cu):
    """Wider ones would be cut to their low bits, and parts of tokens to whole ones, without a word."""
    for args in ((cu, None), ([0, 5, 9], cu)):
        with pytest.raises(gdr.GdrError, match="32 bits|ints"):
            gdr.AttnPlan(*args, device="cpu")


@pytest.mark.parametrize("cu", [[0, 5, 9], (0, 5, 9), np.array([0, 5, 9], np.uint8), torch.tensor([0, 5, 9]), torch.tensor([0, 5, 9], dtype=torch.int32)])
def test_plan_takes_ints_of_any_kind(cu):
    p = gdr.AttnPlan(cu, device="cpu")
    assert (p.N, p.T_q, p.T_k) == (2, 9, 9)


def test_forward_outputs_are_two():
    L, p = gdr.lib(), problem()
    refused(L.gdr_attn_fwd(ctypes.byref(p), OUT, OUT, None, 0, None), 1, "same memory")
