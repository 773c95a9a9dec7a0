"""Results and scratch that a call makes itself for a stream given to it: they
never lie in memory that work queued on the current stream still uses."""
import pytest
import torch

import mla_latent_space_lca_b200 as lca

import paged_ref as ref
from test_gpu_paged import DEV, SCALE, make, status_ok

pytestmark = pytest.mark.gpu
DELAY = 100_000_000   # clock cycles, 50 ms and more


class Pending:
    """Blocks of the given sizes that are free again for the current stream's
    next allocation while that stream has yet to read and write them."""

    def __init__(self, sizes):
        blocks = [torch.empty(n, dtype=torch.uint8, device=DEV).fill_(5) for n in sizes]
        self.kept = [torch.zeros(n, dtype=torch.uint8, device=DEV) for n in sizes]
        torch.cuda.synchronize()
        torch.cuda._sleep(DELAY)
        for b, k in zip(blocks, self.kept):
            k.copy_(b)
            b.fill_(255)

    def check(self):
        torch.cuda.synchronize()
        assert all((k == 5).all() for k in self.kept)


def nbytes(t):
    return t.numel() * t.element_size()


@pytest.mark.parametrize("lens,new,max_new", [([900, 4000, 70], [1, 1, 1], 1), ([900, 4000, 70], [40, 3, 1], 40)])
def test_attention_on_a_stream_given(lens, new, max_new):
    args = make(lens, new, 32, seed=max_new)
    T = args[4].shape[0]
    want = ref.attention(*args, SCALE)
    s2 = torch.cuda.Stream()
    torch.cuda.synchronize()
    pending = Pending([nbytes(lca.paged_workspace(3, T, max_new)), T * 16 * 128 * 2])
    out = lca.mla_paged_attn(*args, max_new, stream=s2)
    pending.check()
    status_ok()
    ref.assert_attention(out, want)


def test_tables_on_a_stream_given():
    B, T, page = 700, 400_000, 16   # (above 1 MB the freed blocks are sure to be the next ones handed out)
    ctx = torch.arange(B, dtype=torch.int32, device=DEV) % 50
    new = torch.full((B,), 7, dtype=torch.int32, device=DEV)
    free = torch.arange(3000, dtype=torch.int32, device=DEV)
    taken = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = torch.arange(B * 4, dtype=torch.int32, device=DEV).view(B, 4) + 5000
    want = ref.tables(ctx.tolist(), new.tolist(), free.tolist(), 0, table.tolist(), page, T)
    s2 = torch.cuda.Stream()
    pending = Pending([4 * B, 4 * (B + 1), 8 * T, 4 * T, 4, 16])
    got = lca.lca_page_tables(ctx, new, free, taken, table, page, T, stream=s2)
    pending.check()
    for g, w in zip(got, want):
        assert g.tolist() == (w if isinstance(w, list) else [w])
    assert table.tolist() == want[6]


def test_a_result_still_read_by_the_current_stream():
    # a result freed here while the current stream has yet to read it: the
    # next call on the other stream must not get its memory
    args = make([300, 90], [3, 2], 16, seed=1)
    other = make([300, 90], [3, 2], 16, seed=2)
    want = ref.attention(*args, SCALE)
    s2 = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = lca.mla_paged_attn(*args, 3, stream=s2)
    kept = torch.zeros_like(out)
    torch.cuda.current_stream().wait_stream(s2)
    torch.cuda._sleep(DELAY)
    kept.copy_(out)
    del out
    again = lca.mla_paged_attn(*other, 3, stream=s2)
    torch.cuda.synchronize()
    status_ok()
    ref.assert_attention(kept, want)
    ref.assert_attention(again, ref.attention(*other, SCALE))


def decode_inputs(B=3, L=5000, seed=4):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *shape: torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    return {"cache": r(B, L, 576), "ring": r(B, 16, 16, 576), "q": r(B, 16, 576),
            "w_uv": (r(16, 512, 128).float() / 512 ** 0.5).to(torch.bfloat16),
            "lens": torch.tensor([L, 70, L - 1300][:B], dtype=torch.int32, device=DEV)}


CONTIGUOUS = {
    "mla_decode_attn": lambda s, **k: lca.mla_decode_attn(s["cache"], s["q"], s["w_uv"], **k),
    "lca_condense": lambda s, **k: lca.lca_condense(s["cache"], s["ring"], **k),
    "lca_decode_attn": lambda s, **k: lca.lca_decode_attn(s["cache"], s["rep"], s["q"], s["w_uv"], **k),
    "lca_decode_stored": lambda s, **k: lca.lca_decode_stored(s["cache"], s["rep"], s["q"], s["w_uv"], **k),
    "lca_decode": lambda s, **k: lca.lca_decode(s["cache"], s["ring"], s["q"], s["w_uv"], **k),
    "lca_decode_varlen": lambda s, **k: lca.lca_decode_varlen(s["cache"], s["lens"], s["ring"], s["q"], s["w_uv"], **k),
    "lca_decode_stored_varlen": lambda s, **k: lca.lca_decode_stored_varlen(s["cache"], s["rep"], s["lens"], s["q"],
                                                                            s["w_uv"], **k),
    "lca_decode_shard": lambda s, **k: lca.lca_decode_shard(s["cache"], s["ring"], s["q"], 5000, 0, **k),
    "lca_combine_shards": lambda s, **k: lca.lca_combine_shards(s["parts"], s["w_uv"], 3, **k),
    "lca_prefill_block": lambda s, **k: lca.lca_prefill_block(s["cache"][:1], s["q_all"], s["w_uv"], 1200, 64, **k),
}
OPS = {"mla_decode_attn": 0, "lca_condense": 1, "lca_decode_attn": 2, "lca_decode_stored": 2, "lca_decode": 3,
       "lca_decode_varlen": 3, "lca_decode_stored_varlen": 2, "lca_decode_shard": 3, "lca_prefill_block": 4}


@pytest.mark.parametrize("name", list(CONTIGUOUS))
def test_contiguous_calls_on_a_stream_given(name):
    s = decode_inputs()
    s["rep"] = lca.lca_condense(s["cache"], s["ring"])
    s["parts"] = lca.lca_decode_shard(s["cache"], s["ring"], s["q"], 5000, 0)[None]
    s["q_all"] = torch.randn(1, 5000, 16, 576, device=DEV).to(torch.bfloat16)
    call = CONTIGUOUS[name]
    want = call(s)
    sizes = [nbytes(want)]
    if name in OPS:
        B, q_len = (1, 64) if name == "lca_prefill_block" else (3, 0)
        sizes.append(nbytes(lca.workspace(OPS[name], B, 5000, q_len)))
    s2 = torch.cuda.Stream()
    torch.cuda.synchronize()
    pending = Pending(sizes)
    got = call(s, stream=s2)
    pending.check()
    status_ok()
    assert torch.equal(got, want)


def test_captured_on_a_stream_that_joins_the_capture():
    args = make([900, 300, 64], [1, 7, 3], 32, seed=9)
    s = decode_inputs()
    want, plain = ref.attention(*args, SCALE), lca.lca_decode(s["cache"], s["ring"], s["q"], s["w_uv"])
    lca.mla_paged_attn(*args, 7)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        out = lca.mla_paged_attn(*args, 7, stream=side)
        again = lca.mla_paged_attn(*args, 1, stream=side)
        fused = lca.lca_decode(s["cache"], s["ring"], s["q"], s["w_uv"], stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for t in (out, again, fused):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        status_ok()
        ref.assert_attention(out, want)
        ref.assert_attention(again, want)
        assert torch.equal(fused, plain)
