"""Plain implementations of the paged-cache operators for the tests: page
tables in Python integers, attention in 64 bits from the definition."""
import math

import torch

H, DC, D, DV = 16, 512, 576, 128


def tables(ctx, new, free, taken, table, page, max_tokens):
    """(seq_lens, q_start, slots, positions, taken_out, counts, table) of
    lists; `table` (list of lists) is changed in place."""
    cap = len(table[0]) * page
    lens, start, slots, positions = [], [0], [], []
    asked = kept = 0
    used = min(max(taken, 0), len(free))
    first = used
    for b, (c, n) in enumerate(zip(ctx, new)):
        c = min(max(c, 0), cap)
        asked += max(n, 0)
        n = min(max(n, 0), cap - c, max_tokens - kept)
        for k in range(-(-c // page), -(-(c + n) // page)):
            table[b][k] = free[used] if used < len(free) else -1
            used += 1
        for p in range(c, c + n):
            pg = table[b][p // page]
            slots.append(pg * page + p % page if pg >= 0 else -1)
            positions.append(p)
        kept += n
        lens.append(c + n)
        start.append(kept)
    got = min(used, len(free))
    pad = max_tokens - kept
    return (lens, start, slots + [-1] * pad, positions + [-1] * pad, got,
            [kept, min(asked - kept, 2 ** 31 - 1), got - first, used - got], table)


def attention(pages, table, lens, q_start, q, w_uv, scale):
    """out [T, 16, 128] in 64 bits; rows of no sequence are NaN."""
    T, (n_pages, page, _) = q.shape[0], pages.shape
    out = torch.full((T, H, DV), math.nan, dtype=torch.float64, device=q.device)
    w = w_uv.double()
    table = table.cpu().tolist()
    for b, row in enumerate(table):
        q0, q1 = int(q_start[b]), int(q_start[b + 1])
        for t in range(max(q0, 0), min(q1, T)):
            pos = int(lens[b]) - (q1 - q0) + t - q0
            want = min(pos + 1, len(row) * page)
            rows = [pages[row[k], : min(page, want - k * page)] for k in range(-(-max(want, 0) // page))
                    if 0 <= row[k] < n_pages]
            if not rows:
                out[t] = 0
                continue
            r = torch.cat(rows).double()
            p = torch.softmax((q[t].double() @ r.T) * scale, -1)
            out[t] = torch.einsum("hc,hcv->hv", p @ r[:, :DC], w)
    return out


# Between fp32 logits and the bf16 result there are two roundings to bf16: the
# softmax weights' and the result's own.  A rounding is off by at most 2^-8 of
# the value, by 2^-8 / sqrt(3) in the mean square.  For latents of independent
# signs the weights' roundings add up in the mean square like the terms of o
# themselves, so each contributes at most 2^-8 / sqrt(3) of the result's norm
# over a token's 2048 values: 2^-8 * sqrt(2 / 3) = 3.2e-3 together.  Half as
# much again covers the scatter of a finite sample and the 32-bit part.
TOKEN_REL = 1.5 * 2.0 ** -8 * math.sqrt(2 / 3)


def assert_attention(got, want, rel=TOKEN_REL):
    """Token by token, in the 2-norm; rows of no sequence are not looked at."""
    assert got.dtype == torch.bfloat16 and got.shape == want.shape
    live = ~torch.isnan(want).flatten(1).all(1)
    g, w = got[live].double().flatten(1), want[live].flatten(1)
    assert torch.isfinite(g).all()
    err = (g - w).norm(dim=1) / w.norm(dim=1).clamp(min=1e-30)
    assert err.numel() == 0 or err.max().item() <= rel, (err.max().item(), int(err.argmax()))
    zero = w.norm(dim=1) == 0
    assert (g[zero] == 0).all()
