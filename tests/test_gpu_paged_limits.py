"""The paged cache at the edges of what its documentation allows: a pool whose
offsets pass 32 bits, the largest pages, pages shared by sequences, many
sequences, other scales, graphs replayed side by side."""
import random

import pytest
import torch

import mla_latent_space_lca_b200 as lca

import paged_ref as ref
from test_gpu_paged import DEV, SCALE, check_attn, i32, make, status_ok

pytestmark = pytest.mark.gpu
HINTS = [1, 9]


def test_a_pool_beyond_32_bit_offsets():
    # 4.5 million rows: 5.2 GB, 2.6 * 2^30 elements; the pages lie in random
    # order, the last ones of the pool among them
    page, n_pages = 64, 70_000
    g = torch.Generator(device=DEV).manual_seed(1)
    pages = torch.zeros(n_pages, page, 576, dtype=torch.bfloat16, device=DEV)
    ctx, new = [3000, 0, 777], [1, 130, 5]
    order = [n_pages - 1 - 7 * k for k in range(60)] + [n_pages // 2 + k for k in range(20)]
    random.Random(1).shuffle(order)
    table = torch.full((3, 64), -1, dtype=torch.int32, device=DEV)
    used = 0
    for b, c in enumerate(ctx):
        n = -(-c // page)
        table[b, :n] = i32(order[used:used + n])
        pages[table[b, :n].long()] = torch.randn(n, page, 576, generator=g, device=DEV).to(torch.bfloat16)
        used += n
    rows = torch.randn(136, 576, generator=g, device=DEV).to(torch.bfloat16)
    lens, start, slots, _, _, counts = lca.lca_page_tables(i32(ctx), i32(new), i32(order), i32([used]), table, page, 136)
    assert counts.tolist()[1] == counts.tolist()[3] == 0
    lca.lca_append_paged(pages, rows, slots)
    assert torch.equal(pages.view(-1, 576)[slots], rows) and slots.max() > 1 << 22
    q = torch.randn(136, 16, 576, generator=g, device=DEV).to(torch.bfloat16)
    w_uv = (torch.randn(16, 512, 128, generator=g, device=DEV) / 512 ** 0.5).to(torch.bfloat16)
    want = ref.attention(pages, table, lens, start, q, w_uv, SCALE)
    for hint in HINTS:
        ref.assert_attention(lca.mla_paged_attn(pages, table, lens, start, q, w_uv, hint), want)
    status_ok()


@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("page", [4096, 65536])
def test_large_pages(page, hint):
    check_attn(*make([9000, 70, 4097], [3, 1, 12], page, seed=page, extra_pages=1), hint)


@pytest.mark.parametrize("hint", HINTS)
def test_pages_shared_by_sequences(hint):
    # two sequences with the same first pages, one that holds a page twice
    pages, table, lens, start, q, w_uv = make([500, 450, 300], [2, 9, 1], 32, seed=3)
    table[1, :12] = table[0, :12]
    table[2, 5] = table[2, 1]
    check_attn(pages, table, lens, start, q, w_uv, hint)


@pytest.mark.parametrize("hint", HINTS)
def test_many_sequences_few_with_tokens(hint):
    rng = random.Random(2)
    new = [rng.choice([0, 0, 0, 0, 0, 0, 0, 0, 1, 3]) for _ in range(9000)]
    lens = [n + rng.randrange(30) for n in new]
    check_attn(*make(lens, new, 16, seed=8, pad=5), hint)


@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("scale", [1e-30, 1e-3, 3.0])
def test_other_scales(scale, hint):
    # (weights of few rows: their roundings need not average out; 2^-8 each, and the result's)
    args = make([700, 90], [3, 2], 64, seed=6)
    out = lca.mla_paged_attn(*args, hint, scale=scale)
    status_ok()
    ref.assert_attention(out, ref.attention(*args, scale), rel=2.004 * 2.0 ** -8 * 1.01)


def test_graphs_side_by_side():
    """Two captured calls with a workspace each, replayed at the same time on
    two streams; a third graph shares the first one's inputs, not its scratch."""
    batches = [(make([3000, 800, 64], [40, 3, 1], 32, seed=1), 40), (make([5000, 60, 900], [1, 1, 1], 16, seed=2), 1)]
    batches.append((batches[0][0], 7))
    graphs, outs = [], []
    for args, hint in batches:
        lca.mla_paged_attn(*args, hint)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(lca.mla_paged_attn(*args, hint))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for o in outs:
        o.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    status_ok()
    for o, (args, _) in zip(outs, batches):
        ref.assert_attention(o, ref.attention(*args, SCALE))
