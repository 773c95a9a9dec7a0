"""Attention of several new tokens a sequence over pages: work cut over SM
pairs (many query tiles a pair, one query tile over many), tile borders, plans
above their shared-memory sizes, capture, streams."""
import random

import pytest
import torch

import mla_latent_space_lca_b200 as lca

import paged_ref as ref
from test_gpu_paged import DEV, SCALE, Server, check_attn, i32, make, status_ok

pytestmark = pytest.mark.gpu


def sampled(pages, table, lens, start, q, w_uv, tokens):
    """ref.attention of some tokens of the batch."""
    out = torch.full((q.shape[0], 16, 128), float("nan"), dtype=torch.float64, device=DEV)
    bounds = start.tolist()
    for t in tokens:
        b = next(i for i in range(len(bounds) - 1) if bounds[i] <= t < bounds[i + 1])
        n = int(lens[b]) - (bounds[b + 1] - t) + 1
        out[t] = ref.attention(pages, table[b:b + 1], i32([n]), i32([0, 1]), q[t:t + 1], w_uv, SCALE)[0]
    return out


# ------------------------------------------------------------------ tile borders
@pytest.mark.parametrize("n", [1, 7, 8, 9, 16, 17])
@pytest.mark.parametrize("rows", [127, 128, 129, 143, 144, 145, 255, 256, 257, 384])
def test_rows_and_tokens_at_tile_borders(rows, n):
    check_attn(*make([rows, max(rows - 1, n)], [n, n], 16, seed=rows + n), 17)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_every_length_of_a_prompt(page):
    # each token's row count is another: 1 .. 300
    check_attn(*make([300], [300], page, seed=page), 300)


# ------------------------------------------------------------------ cutting the work
@pytest.mark.parametrize("lens,new", [
    ([746, 97, 71, 266], [700, 1, 1, 1]),          # several short pieces a pair, the last of each cut
    ([40, 300, 513, 700], [40, 300, 513, 700]),    # prompts from their first token on
    ([4000], [3]), ([9000, 20], [9, 20]),          # one query tile over many pairs
    ([1500] * 7, [8] * 7), ([129] * 90, [2] * 90), ([30] * 200, [3] * 200),
])
def test_uneven_work(lens, new):
    for page in (16, 64):
        check_attn(*make(lens, new, page, seed=len(lens)), max(new))


def test_long_rows_few_tokens():
    args = make([60000, 31, 20001], [4, 2, 11], 64, seed=12)
    check_attn(*args, 11)


def test_plan_above_its_shared_memory():
    # more than 1024 sequences, more than 1024 query tiles, both
    rng = random.Random(4)
    new = [rng.choice([0, 1, 2, 9]) for _ in range(1500)]
    lens = [n + rng.randrange(40) for n in new]
    args = make(lens, new, 16, seed=3)
    check_attn(*args, 9)
    args = make([9100, 60], [9100, 60], 64, seed=5)
    out = lca.mla_paged_attn(*args, 9100)
    status_ok()
    ref.assert_attention(out, sampled(*args, [0, 1, 7, 8, 500, 1023, 1024, 4095, 5000, 8191, 8192, 9099, 9100, 9159]))


def test_maximum_that_keeps_moving():
    # every cache tile brings a new maximum for every row, most of them above
    # the step of 2^8 that rescales what is there
    pages, table, lens, start, q, w_uv = make([2000], [17], 64, seed=21)
    ids = table[0, :-(-2000 // 64)].long()
    ramp = torch.linspace(0, 150, ids.numel() * 64, device=DEV).view(-1, 64, 1)
    mean = q.float().mean((0, 1))
    unit = mean / mean.norm() ** 2 / SCALE
    q = (q.float() * 0.05 + mean * 1.0).to(torch.bfloat16)
    pages[ids] = (pages[ids].float() * 0.2 + ramp * unit).to(torch.bfloat16)
    pages[ids[-1], 2000 % 64:] = float("nan")
    check_attn(pages, table, lens, start, q, w_uv, 17)


@pytest.mark.parametrize("n", [2, 8, 20])
def test_non_finite_rows_behind_every_token(n):
    # the rows between a token and the last one of its query tile, and the
    # page's rest, hold infinities of either sign and NaN in all columns
    pages, table, lens, start, q, w_uv = make([130 + n], [n], 64, seed=n)
    want = ref.attention(pages, table, lens, start, q, w_uv, SCALE)
    page, row = int(table[0, (130 + n - 1) // 64]), (130 + n - 1) % 64
    for value in (float("inf"), -float("inf"), float("nan")):
        pages[page, row] = value   # the last token's own row
        out = lca.mla_paged_attn(pages, table, lens, start, q, w_uv, n)
        status_ok()
        ref.assert_attention(out[:n - 1], want[:n - 1])
        assert not torch.isfinite(out[n - 1:].float()).any()


# ------------------------------------------------------------------ streams, graphs, workspaces
def test_two_batches_at_once():
    a, b = make([3000, 800], [30, 9], 32, seed=1), make([500, 2600, 90], [40, 3, 1], 16, seed=2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):   # workspaces allocated on the current stream, used on another, freed at once
        x = lca.mla_paged_attn(*a, 30, stream=s1)
        y = lca.mla_paged_attn(*b, 40, stream=s2)
        torch.empty(1 << 22, device=DEV).fill_(float("nan"))
    torch.cuda.synchronize()
    status_ok()
    ref.assert_attention(x, ref.attention(*a, SCALE))
    ref.assert_attention(y, ref.attention(*b, SCALE))


def test_one_workspace_from_call_to_call():
    # calls of other shapes before it leave nothing that matters in it
    shapes = [make([900, 70], [33, 2], 16, seed=1), make([5000], [2], 64, seed=2), make([64] * 20, [5] * 20, 32, seed=3)]
    ws = max((lca.paged_workspace(a[1].shape[0], a[4].shape[0], 99) for a in shapes), key=torch.Tensor.numel)
    ws.fill_(255)
    for a in shapes + shapes[::-1]:
        ref.assert_attention(lca.mla_paged_attn(*a, 99, ws=ws), ref.attention(*a, SCALE))
    status_ok()


def test_captured_step_of_drafted_tokens():
    """Four drafted tokens a sequence and step, captured once: lengths, pages
    and slots move on the device."""
    s = Server(3, 16, 60, seed=2)
    first = [20, 133, 5]
    rows, q = s.inputs(sum(first))
    s.step(i32(first), rows, q, max(first))
    s.keep(first, rows)
    new, batch = i32([4, 4, 4]), [4, 4, 4]
    rows, q = s.inputs(14)   # two rows of no sequence behind them
    state = s.lens.clone(), s.taken.clone(), s.table.clone(), s.pages.clone()

    def restore():
        for t, v in zip((s.lens, s.taken, s.table, s.pages), state):
            t.copy_(v)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s.step(new, rows, q, 4)
    torch.cuda.synchronize()
    restore()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, start, _ = s.step(new, rows, q, 4)
    restore()
    for _ in range(15):
        r, x = s.inputs(14)
        rows.copy_(r)
        q.copy_(x)
        out[12:] = 7.0
        graph.replay()
        s.keep(batch, r[:12])
        ref.assert_attention(out[:12], s.expect(batch, x[:12]))
        assert (out[12:] == 7.0).all()
    status_ok()
    assert s.lens.tolist() == [80, 193, 65]


def test_refusals_on_the_gpu():
    pages, table, lens, start, q, w_uv = make([40], [4], 16)
    with pytest.raises(TypeError):
        lca.mla_paged_attn(pages, table, lens, start, q.float(), w_uv, 4)
    with pytest.raises(ValueError):
        lca.mla_paged_attn(pages, table, lens, start, q[:, :8], w_uv, 4)
    with pytest.raises(ValueError):
        lca.mla_paged_attn(pages, table, lens, start[:1], q, w_uv, 4)
    with pytest.raises(ValueError):
        lca.mla_paged_attn(pages.transpose(0, 1), table, lens, start, q, w_uv, 4)
    with pytest.raises((TypeError, ValueError)):
        lca.mla_paged_attn(pages, table, lens.cpu(), start, q, w_uv, 4)
    with pytest.raises(lca._lib.LcaError):
        lca.mla_paged_attn(pages, table, lens, start, q, w_uv, 4, ws=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(lca._lib.LcaError):
        lca.mla_paged_attn(pages, table, lens, start, q, w_uv, 4, scale=-0.1)
    with pytest.raises(lca._lib.LcaError):
        lca.mla_paged_attn(pages, table, lens, start, q, w_uv, 0)
    empty = lca.mla_paged_attn(pages, table, lens, i32([0, 0]), q[:0], w_uv, 4)
    assert empty.shape == (0, 16, 128)


@pytest.mark.parametrize("B", [127, 128, 129, 300, 1030])
def test_single_tokens_of_many_sequences(B):
    # up to 128 tokens and sequences the attention kernel lists its items itself
    rng = random.Random(B)
    new = [rng.choice([0, 1, 1, 1]) for _ in range(B)]
    lens = [n + rng.randrange(200) for n in new]
    check_attn(*make(lens, new, 16, seed=B, pad=2), 1)


@pytest.mark.parametrize("new", [[128], [1] * 128, [129], [0] * 127 + [5], [60, 0, 68]])
def test_item_lists_at_their_size(new):
    check_attn(*make([n + 50 for n in new], new, 32, seed=len(new)), 1)
