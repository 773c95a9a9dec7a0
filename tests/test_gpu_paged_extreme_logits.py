"""Attention over pages with logits of any size that fp32 holds.

The logits' own rounding in fp32 is at most 576 * 2^-24 = 3.5e-5 of the sum of
their products' magnitudes.  Looked at are the tokens' heads whose largest logit
is above all others by twice that and 200 more, in 64 bits: their weights are
one-hot.  Such a result is a row through W_UV, off by one rounding of its one
weight to bf16 (against the fp32 sum that holds the same weight) and by the
result's own, 2^-8 of the value each at most, which is 2.004 * 2^-8 together;
1 % more is for the 32-bit part."""
import pytest
import torch

import mla_latent_space_lca_b200 as lca

import paged_ref as ref
from test_gpu_paged import DEV, SCALE, make, status_ok

pytestmark = pytest.mark.gpu
HINTS = [1, 9]
REL = 2.004 * 2.0 ** -8 * 1.01


def check(pages, table, lens, start, q, w_uv, hint):
    rows = pages[table[0, : -(-int(lens[0]) // pages.shape[1])].long()].reshape(-1, 576)[: int(lens[0])].double()
    n = q.shape[0]
    sure = torch.zeros(n, 16, dtype=torch.bool, device=DEV)
    for i in range(n):
        m = rows[: len(rows) - n + i + 1]
        top = (q[i].double() @ m.T * SCALE).topk(2, -1).values
        error = 3.5e-5 * SCALE * (q[i].double().abs() @ m.abs().T).amax(-1)
        sure[i] = top[:, 0] - top[:, 1] > 2 * error + 200
    assert sure.float().mean() > 0.5
    out = lca.mla_paged_attn(pages, table, lens, start, q, w_uv, hint)
    status_ok()
    want = ref.attention(pages, table, lens, start, q, w_uv, SCALE)[sure]
    got = out.double()[sure]
    assert torch.isfinite(got).all()
    assert ((got - want).norm(dim=1) / want.norm(dim=1)).max() <= REL


@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("size", [1e2, 1e3, 1e4, 3e4, 1e5, 3e5, 1e6, 1e9, 1e13])
def test_logits_up_to(size, hint):
    pages, table, lens, start, q, w_uv = make([30], [7], 16, seed=3)
    pages = (pages.float() * size).to(torch.bfloat16)
    q = (q.float() * size).to(torch.bfloat16)
    check(pages, table, lens, start, q, w_uv, hint)


@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("exponent", [20, 26, 29, 30, 31, 32, 40, 60])
@pytest.mark.parametrize("steps", [1, 40])
def test_logits_that_differ_in_their_last_bits(steps, exponent, hint):
    # one product per logit, so that fp32 holds it exactly: 300 rows whose
    # bf16 values step down from row 250, in both directions
    pages, table, lens, start, q, w_uv = make([300], [9], 16, seed=5)
    ids = table[0, : -(-300 // 16)].long()
    rows = pages[ids].reshape(-1, 576)
    near = (torch.arange(rows.shape[0], device=DEV) - 250).abs()
    rows[:, 0] = (2.0 ** (exponent // 2) * (2 - 2.0 ** -7 * (1 + (steps * near).clamp(max=126)))).to(torch.bfloat16)
    pages[ids] = rows.view(-1, 16, 576)
    pages[ids[-1], 300 % 16:] = float("nan")
    q.zero_()
    q[:, :, 0] = 2.0 ** (exponent - exponent // 2 + 4)
    check(pages, table, lens, start, q, w_uv, hint)


def ramp(lens, new, page, first, last, seed, size=1.0):
    """Rows along one direction: logits from `first` to `last` by position."""
    pages, table, lens, start, q, w_uv = make([lens], [new], page, seed=seed)
    ids = table[0, : -(-int(lens[0]) // page)].long()
    unit = q[0, 0].float() / q[0, 0].float().norm()
    q[:] = (unit * size).to(torch.bfloat16)
    z = torch.linspace(first, last, ids.numel() * page, dtype=torch.float64, device=DEV)
    pages[ids] = (z.view(-1, page, 1) * unit.double() / (SCALE * size)).to(torch.bfloat16)
    return pages, table, lens, start, q, w_uv


@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("first,last", [(-3e33, -1e32), (-1e32, -3e33), (-1e25, -1e24), (3e35, -3e35), (-3e35, 3e35)])
def test_logits_of_any_sign(first, last, hint):
    check(*ramp(20, 5, 16, first, last, seed=2, size=1e15), hint)
