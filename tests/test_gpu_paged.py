"""The paged cache on the GPU: page tables, append and attention over pages,
each against tests/paged_ref.py, and a serving loop of the three."""
import random

import pytest
import torch

import mla_latent_space_lca_b200 as lca

import paged_ref as ref

pytestmark = pytest.mark.gpu
SCALE = 1.0 / 192.0 ** 0.5
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def status_ok():
    rc, detail = lca.device_status()
    assert rc == 0, hex(detail)


# ------------------------------------------------------------------ tables
def guarded(n, dtype, fill):
    buf = torch.full((n + 16,), fill, dtype=dtype, device=DEV)
    return buf, buf[8:8 + n]


def check_tables(ctx, new, free, taken, blocks, page, max_tokens, seed=0, inplace=False):
    rng = random.Random(seed)
    B = len(ctx)
    table = [[rng.randrange(1000, 2000) for _ in range(blocks)] for _ in range(B)]
    dt = i32(table)
    dctx, dtaken = i32(ctx), i32([taken])
    want = ref.tables(ctx, new, free, taken, table, page, max_tokens)
    bufs = {k: guarded(n, d, f) for k, n, d, f in (
        ("seq_lens", B, torch.int32, -77), ("q_start", B + 1, torch.int32, -77),
        ("slot_map", max_tokens, torch.int64, -77), ("positions", max_tokens, torch.int32, -77),
        ("taken_out", 1, torch.int32, -77), ("counts", 4, torch.int32, -77))}
    outs = {k: v[1] for k, v in bufs.items()}
    if inplace:
        outs["seq_lens"], outs["taken_out"] = dctx, dtaken
    got = lca.lca_page_tables(dctx, i32(new), i32(free), dtaken, dt, page, max_tokens, **outs)
    for g, w, name in zip(got, want, ("seq_lens", "q_start", "slot_map", "positions", "taken_out", "counts")):
        assert g.cpu().tolist() == (w if isinstance(w, list) else [w]), name
    assert dt.cpu().tolist() == want[6]
    for k, (buf, _) in bufs.items():
        assert (buf[:8] == -77).all() and (buf[-8:] == -77).all(), k


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("B,page,lo,hi,max_tokens", [
    (1, 16, 1, 1, 1), (1, 64, 1, 1, 3), (3, 16, 0, 40, 128), (33, 32, 0, 7, 300), (1025, 16, 0, 5, 4000),
    (2500, 128, 0, 3, 9000), (7, 16, 200, 900, 8000), (64, 64, 1, 1, 64),
])
def test_tables(B, page, lo, hi, max_tokens, inplace):
    rng = random.Random(B)
    ctx = [rng.choice([0, 1, page - 1, page, page + 1, rng.randrange(20 * page)]) for _ in range(B)]
    new = [rng.randint(lo, hi) for _ in range(B)]
    blocks = 20 + -(-hi // page) + 1
    check_tables(ctx, new, rng.sample(range(1 << 20), B * (hi // page + 2) + 5), 2, blocks, page, max_tokens,
                 inplace=inplace)


@pytest.mark.parametrize("max_tokens", [0, 5, 64, 3000])
def test_tables_without_room(max_tokens):
    # a list that runs out, rows beyond the table, lengths below zero and huge
    ctx = [-3, 15, 2 ** 31 - 1, 60, 0, 64, 10]
    new = [20, 2 ** 31 - 1, 5, 9, -4, 3, 2 ** 31 - 1]
    check_tables(ctx, new, [11, 12, 13], 1, 4, 16, max_tokens)
    check_tables(ctx, new, [11, 12, 13], 99, 4, 16, max_tokens)
    check_tables(ctx, new, [], 0, 4, 16, max_tokens)


def test_tables_largest_batch():
    rng = random.Random(5)
    B = 8192
    check_tables([rng.randrange(100) for _ in range(B)], [rng.randrange(4) for _ in range(B)],
                 rng.sample(range(1 << 20), 9000), 0, 8, 16, 20000)
    with pytest.raises(lca._lib.LcaError):
        lca.lca_page_tables(i32([0] * 8193), i32([0] * 8193), i32([1]), i32([0]), i32([[0]] * 8193), 16, 4)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("T", [1, 3, 5, 64, 1001, 20000])
@pytest.mark.parametrize("pitch", [576, 640])
def test_append(T, pitch):
    g = torch.Generator(device=DEV).manual_seed(T)
    n_pages, page = T // 16 + 3, 32
    pages = torch.randn(n_pages, page, 576, generator=g, device=DEV).to(torch.bfloat16)
    rows = torch.randn(T, pitch, generator=g, device=DEV).to(torch.bfloat16)[:, :576]
    slots = torch.randperm(n_pages * page, generator=g, device=DEV)[:T]
    if T > 2:   # slots that are no slots
        slots[0], slots[T // 2], slots[T - 1] = -1, n_pages * page, 2 ** 40
    want = pages.clone()
    good = (slots >= 0) & (slots < n_pages * page)
    want.view(-1, 576)[slots[good]] = rows[good]
    lca.lca_append_paged(pages, rows, slots)
    assert torch.equal(pages, want)


# ------------------------------------------------------------------ attention
def make(lens, new, page, seed=0, spread=1.0, extra_pages=3, pad=0):
    """Random pages in random order; rows past each sequence's end (the rest
    of its last page, and pages of no sequence) are NaN."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    need = [-(-max(n, 0) // page) for n in lens]
    n_pages = sum(need) + extra_pages
    pages = torch.randn(n_pages, page, 576, generator=g, device=DEV).to(torch.bfloat16)
    perm = torch.randperm(n_pages, generator=g, device=DEV).tolist()
    blocks = max(need + [1]) + 1
    table = [[-1] * blocks for _ in lens]
    k = 0
    for b, n in enumerate(lens):
        for j in range(need[b]):
            table[b][j] = perm[k]
            k += 1
        if n > 0 and n % page:
            pages[table[b][need[b] - 1], n % page:] = float("nan")
    for p in perm[k:]:
        pages[p] = float("nan")
    T = sum(new) + pad
    q = (torch.randn(T, 16, 576, generator=g, device=DEV) * spread).to(torch.bfloat16)
    w_uv = (torch.randn(16, 512, 128, generator=g, device=DEV) / 512 ** 0.5).to(torch.bfloat16)
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    return pages, i32(table), i32(lens), i32(start), q, w_uv


def check_attn(pages, table, lens, start, q, w_uv, max_new, rel=ref.TOKEN_REL):
    T = q.shape[0]
    buf = torch.full((T + 2, 16, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lca.mla_paged_attn(pages, table, lens, start, q, w_uv, max_new, out=buf[1:T + 1])
    want = ref.attention(pages, table, lens, start, q, w_uv, SCALE)
    status_ok()
    ref.assert_attention(buf[1:T + 1], want, rel)
    dead = torch.isnan(want).flatten(1).all(1)
    assert (buf[1:T + 1][dead] == 7.0).all() and (buf[0] == 7.0).all() and (buf[-1] == 7.0).all()


HINTS = [1, 9]   # both kernels, whatever the batch holds


@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 1024])
@pytest.mark.parametrize("lens,new", [
    ([1], [1]), ([2], [2]), ([63], [1]), ([64], [1]), ([65], [3]), ([17, 1, 400], [1, 1, 1]),
    ([129, 64, 1000], [5, 9, 1]), ([300], [33]), ([8], [8]), ([40, 7], [40, 7]),
])
def test_attention_sizes(page, lens, new, hint):
    check_attn(*make(lens, new, page, seed=len(lens) + page), hint)


@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("seed", range(6))
def test_attention_ragged(seed, hint):
    rng = random.Random(seed)
    B = rng.randint(1, 40)
    new = [rng.choice([0, 1, 1, 2, 5, 17]) for _ in range(B)]
    lens = [n + rng.choice([0, 1, rng.randrange(3000)]) for n in new]
    if sum(new) == 0:
        new[0], lens[0] = 1, lens[0] + 1
    check_attn(*make(lens, new, rng.choice([16, 32, 64, 256]), seed=seed, pad=rng.choice([0, 3])), hint)


@pytest.mark.parametrize("hint", HINTS)
def test_attention_tokens_with_nothing_to_attend(hint):
    # lengths below the number of new tokens (positions below 0), zero and negative
    args = make([3, 0, -5, 70], [8, 2, 1, 3], 16, seed=3, pad=2)
    check_attn(*args, hint)


@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("page", [16, 64, 128])
def test_attention_missing_pages(page, hint):
    pages, table, lens, start, q, w_uv = make([700, 700, 90, 200], [1, 12, 3, 2], page, seed=9)
    n = pages.shape[0]
    table[0, 0], table[0, 2], table[1, 1] = -1, n, 2 ** 31 - 1   # entries that name no page
    table[1, -3:] = -(2 ** 31)
    table[2] = -1                                                # a sequence without any
    check_attn(pages, table, lens, start, q, w_uv, hint)


@pytest.mark.parametrize("hint", HINTS)
def test_attention_table_shorter_than_the_length(hint):
    pages, table, lens, start, q, w_uv = make([200, 60], [4, 2], 16, seed=4)
    check_attn(pages, table[:, :5].contiguous(), lens, start, q, w_uv, hint)


@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("bad", [[0, 5, 3, 8], [2, 4, 4, 7], [-3, 2, 5, 100], [0, 0, 0, 0], [5, 4, 3, 2]])
def test_attention_offsets_out_of_order(bad, hint):
    # the first row of no sequence, overlapping and decreasing offsets, rows
    # beyond the batch: whatever they say, only rows of the batch are touched
    pages, table, lens, start, q, w_uv = make([90, 90, 90], [3, 3, 2], 32, seed=6)
    buf = torch.full((10, 16, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lca.mla_paged_attn(pages, table, lens, i32(bad), q, w_uv, hint, out=buf[1:9])
    status_ok()
    assert (buf[0] == 7.0).all() and (buf[-1] == 7.0).all()
    if bad == sorted(bad) and bad[0] >= 0:
        want = ref.attention(pages, table, lens, i32(bad), q, w_uv, SCALE)
        ref.assert_attention(buf[1:9], want)
        assert (buf[1:9][torch.isnan(want).flatten(1).all(1)] == 7.0).all()


@pytest.mark.parametrize("hint", HINTS)
def test_attention_large_logits(hint):
    # logits up to several hundred: near one-hot weights, a moving maximum.
    # fp32 logits of size z carry z * 576 * 2^-24 at most, and as much
    # relative error of a weight: with |z| <= 400 that is 1.4e-2 at the very
    # worst; the mean square over a sum of 576 terms is sqrt(576) * 2^-24 * 400
    args = make([900, 2000], [2, 7], 32, seed=8, spread=25.0)
    check_attn(*args, hint)


@pytest.mark.parametrize("hint", HINTS)
def test_attention_growing_logits(hint):
    # every tile's maximum above the last one's by more than the rescale step
    pages, table, lens, start, q, w_uv = make([1500], [6], 16, seed=2)
    ids = table[0, :-(-1500 // 16)].long()
    ramp = torch.linspace(0, 60, ids.numel() * 16, device=DEV).view(-1, 16, 1)
    unit = q[0, 0].float() / q[0, 0].float().norm() ** 2 / SCALE
    pages[ids] = (pages[ids].float() * 0.2 + ramp * unit).to(torch.bfloat16)
    pages[ids[-1], 1500 % 16:] = float("nan")
    check_attn(pages, table, lens, start, q, w_uv, hint)


@pytest.mark.parametrize("hint", HINTS)
def test_attention_later_rows_that_are_not_finite(hint):
    # row 70 of the sequence holds NaN and infinities: the tokens before it
    # must not see them, the token itself and those after it do
    pages, table, lens, start, q, w_uv = make([75], [12], 16, seed=5)
    pages[int(table[0, 70 // 16]), 70 % 16, 100] = float("nan")
    pages[int(table[0, 72 // 16]), 72 % 16, 300] = float("inf")
    out = lca.mla_paged_attn(pages, table, lens, start, q, w_uv, hint)
    status_ok()
    want = ref.attention(pages, table, lens, start, q, w_uv, SCALE)
    ref.assert_attention(out[:7], want[:7])   # positions 63 .. 69
    assert torch.isnan(out[7:].float()).all()


@pytest.mark.parametrize("hint", HINTS)
def test_attention_repeats_bit_for_bit(hint):
    args = make([4000, 130, 2222], [1, 20, 3], 64, seed=11)
    first = lca.mla_paged_attn(*args, hint)
    for _ in range(3):
        assert torch.equal(first, lca.mla_paged_attn(*args, hint))


def test_attention_two_streams_at_once():
    a, b = make([3000, 800], [1, 1], 32, seed=1), make([500, 2600, 90], [40, 3, 1], 16, seed=2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(s1):
            x = lca.mla_paged_attn(*a, 1)
        y = lca.mla_paged_attn(*b, 40, stream=s2)
    torch.cuda.synchronize()
    status_ok()
    ref.assert_attention(x, ref.attention(*a, SCALE))
    ref.assert_attention(y, ref.attention(*b, SCALE))


# ------------------------------------------------------------------ together
class Server:
    """A cache in pages, kept by the three operators; the rows as appended
    are kept beside it, sequence by sequence."""

    def __init__(self, B, page, blocks, seed=0):
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.page, self.B = page, B
        n_pages = B * blocks
        self.pages = torch.full((n_pages, page, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
        self.free = torch.randperm(n_pages, generator=self.g, device=DEV).to(torch.int32)
        self.taken, self.lens = i32([0]), i32([0] * B)
        self.table = torch.full((B, blocks), -1, dtype=torch.int32, device=DEV)
        self.w_uv = (torch.randn(16, 512, 128, generator=self.g, device=DEV) / 512 ** 0.5).to(torch.bfloat16)
        self.rows = [[] for _ in range(B)]

    def inputs(self, T):
        r = torch.randn(T, 576, generator=self.g, device=DEV).to(torch.bfloat16)
        return r, torch.randn(T, 16, 576, generator=self.g, device=DEV).to(torch.bfloat16)

    def step(self, new, rows, q, max_new, **kw):
        _, start, slots, _, _, counts = lca.lca_page_tables(
            self.lens, new, self.free, self.taken, self.table, self.page, rows.shape[0], seq_lens=self.lens,
            taken_out=self.taken, **kw)
        lca.lca_append_paged(self.pages, rows, slots)
        return lca.mla_paged_attn(self.pages, self.table, self.lens, start, q, self.w_uv, max_new), start, counts

    def keep(self, new, rows):
        t = 0
        for b, n in enumerate(new):
            self.rows[b].append(rows[t:t + n])
            t += n

    def expect(self, new, q):
        out, t = [], 0
        for b, n in enumerate(new):
            r = torch.cat(self.rows[b]).double()
            for i in range(n):
                m = r[: len(r) - n + i + 1]
                p = torch.softmax((q[t].double() @ m.T) * SCALE, -1)
                out.append(torch.einsum("hc,hcv->hv", p @ m[:, :512], self.w_uv.double()))
                t += 1
        return torch.stack(out)


@pytest.mark.parametrize("page", [16, 64])
def test_serving_loop(page):
    s = Server(4, page, 1200 // page + 1, seed=page)
    for new in ([37, 0, 1, 260], [1, 90, 1, 1], [1, 1, 1, 1], [0, 1, 64, 1], [5, 3, 2, 1], [1, 1, 1, 1],
                [1, 0, 0, 0], [700, 1, 1, 1]):
        rows, q = s.inputs(sum(new))
        out, start, counts = s.step(i32(new), rows, q, max(new))
        s.keep(new, rows)
        assert counts.cpu().tolist()[:2] == [sum(new), 0] and counts[3] == 0
        ref.assert_attention(out, s.expect(new, q))
    status_ok()
    # the same cache, contiguous, through the decode that was there before:
    # its o enters W_UV rounded to bf16, one rounding more than here
    b = 3
    r = torch.cat(s.rows[b])[None].contiguous()
    old = lca.mla_decode_attn(r, q[-1:], s.w_uv)
    assert ((old[0].double() - s.expect(new, q)[-1]).norm() / old.double().norm()).item() < 2 * ref.TOKEN_REL


def test_serving_loop_captured():
    """One decode step, captured once and replayed: the lengths, pages and
    slots move on the device."""
    s = Server(3, 16, 40, seed=1)
    first = [20, 33, 5]
    rows, q = s.inputs(sum(first))
    s.step(i32(first), rows, q, max(first))
    s.keep(first, rows)
    new = i32([1, 1, 1])
    rows, q = s.inputs(3)
    side = torch.cuda.Stream()
    state = s.lens.clone(), s.taken.clone(), s.table.clone(), s.pages.clone()
    with torch.cuda.stream(side):
        s.step(new, rows, q, 1)   # warm-up, undone
    torch.cuda.synchronize()
    for t, v in zip((s.lens, s.taken, s.table, s.pages), state):
        t.copy_(v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _, _ = s.step(new, rows, q, 1)
    for t, v in zip((s.lens, s.taken, s.table, s.pages), state):
        t.copy_(v)
    for _ in range(20):
        r, x = s.inputs(3)
        rows.copy_(r)
        q.copy_(x)
        graph.replay()
        s.keep([1, 1, 1], r)
        ref.assert_attention(out, s.expect([1, 1, 1], x))
    status_ok()
    assert s.lens.cpu().tolist() == [40, 53, 25]
