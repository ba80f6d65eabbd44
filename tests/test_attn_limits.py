"""Host-side limits of the softmax-attention layers' operators, without a GPU: every
refusal here stands for sizes that the kernels' 32-bit arithmetic would not hold."""
import ctypes

import pytest

import chunked_gated_delta_14_amd as gdr
from test_attn_host import BIG, OUT, kv, refused, step


@pytest.mark.parametrize("page,max_pages,T", [(256, 1 << 23, 3), (16, (1 << 26) + 1, 3), (256, (1 << 31) - 1, 3), (16, 4, (1 << 30) + 1)])
def test_step_places_past_32_bits(page, max_pages, T):
    """Places are held with 32 bits, up to a block's share past the last: tables of more than 2^30 places are refused."""
    L, c, p = gdr.lib(), kv(page=page, max_pages=max_pages, N=T), step(T=T)
    refused(L.gdr_attn_step_fwd(ctypes.byref(c), ctypes.byref(p), OUT, 1 << 23, BIG, None), 2, "2^30")
    refused(-L.gdr_attn_step_workspace_bytes(T, T, 4, 2, max_pages, page), 2, "2^30")
    assert L.gdr_attn_step_workspace_bytes(3, 3, 4, 2, (1 << 30) // page, page) > 0
