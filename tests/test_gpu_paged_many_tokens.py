"""Single-token attention over pages for batches above 2^19 tokens, where the
launch of the merge kernel passes 65535 groups of 8 tokens."""
import pytest
import torch

import mla_latent_space_lca_b200 as lca

import paged_ref as ref
from test_gpu_paged import DEV, SCALE, i32, status_ok

pytestmark = pytest.mark.gpu


def test_more_than_65535_groups_of_tokens():
    T, page = 8 * 65535 + 13, 64
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 30 GB: 32 KB of partial outputs and 22 KB of inputs and results a token")
    g = torch.Generator(device=DEV).manual_seed(7)
    pages = torch.randn(5, page, 576, generator=g, device=DEV).to(torch.bfloat16)
    table = i32([[3, 1], [0, 4]])
    first = T // 3
    start, lens = i32([0, first, T]), i32([first, T - first])   # tokens past the table's 128 rows attend all of them
    q = torch.empty(T, 16, 576, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    w_uv = (torch.randn(16, 512, 128, generator=g, device=DEV) / 512 ** 0.5).to(torch.bfloat16)
    out = lca.mla_paged_attn(pages, table, lens, start, q, w_uv, 1)
    status_ok()
    assert torch.isfinite(out).all()
    tokens = sorted({0, 1, 70, first - 1, first, first + 100, *range(4096, T, 65536), 8 * 65535 - 1, 8 * 65535,
                     8 * 65535 + 1, T - 1})
    want = torch.cat([ref.attention(pages, table[b:b + 1], i32([t - int(start[b]) + 1]), i32([0, 1]), q[t:t + 1], w_uv,
                                    SCALE) for t in tokens for b in [int(t >= first)]])
    ref.assert_attention(out[tokens], want)
