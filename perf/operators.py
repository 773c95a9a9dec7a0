"""What is measured of the paged latent cache: the page tables built from
request lengths, the append of new rows through the slot map, and MLA
attention of each sequence's new tokens over its pages.

`run` computes a case either in its plain form (elementary torch operations,
fp32, rounded once at the end) or, with `own` set, through the framework's
entry points.  A cache row is [c (512) | k^R (64)] bf16, 16 query heads, value
width 128 after W_UV, as everywhere in this framework.
"""
import math

import torch

own = False

HEADS, D_C, D_R, D_V = 16, 512, 64, 128
D = D_C + D_R
SCALE = 1.0 / math.sqrt(192.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the bookkeeping of one user's next token: pure latency
        {"name": "tables_b1_n1", "op": "tables", "batch": 1, "ctx": 4096, "ctx_hi": 4096, "new": 1,
         "new_hi": 1, "last": 0, "page": 64},
        # a large mixed batch: 512 requests, short and long chunks, small pages
        {"name": "tables_b512_mixed", "op": "tables", "batch": 512, "ctx": 0, "ctx_hi": 8000, "new": 1,
         "new_hi": 250, "last": 0, "page": 16},
        # one decode step's rows of 32 sequences
        {"name": "append_b32_n1", "op": "append", "batch": 32, "ctx": 900, "ctx_hi": 5000, "new": 1, "new_hi": 1,
         "last": 0, "page": 64},
        # the rows of several long prompt chunks
        {"name": "append_b9_chunks", "op": "append", "batch": 9, "ctx": 0, "ctx_hi": 4001, "new": 1500,
         "new_hi": 2200, "last": 0, "page": 16},
        # one token of one short sequence: latency
        {"name": "attn_b1_l4k_n1", "op": "attn", "batch": 1, "ctx": 4095, "ctx_hi": 4095, "new": 1, "new_hi": 1,
         "last": 0, "page": 64},
        # the decode of the framework's own benchmark, over pages: 8 x 128K
        {"name": "attn_b8_l128k_n1", "op": "attn", "batch": 8, "ctx": 131071, "ctx_hi": 131071, "new": 1,
         "new_hi": 1, "last": 0, "page": 64},
        # a ragged serving batch of 32 up to 32K, small pages
        {"name": "attn_b32_ragged_n1", "op": "attn", "batch": 32, "ctx": 700, "ctx_hi": 32767, "new": 1,
         "new_hi": 1, "last": 0, "page": 16},
        # several tokens a sequence at once (drafted tokens to be verified)
        {"name": "attn_b16_n2to5", "op": "attn", "batch": 16, "ctx": 1000, "ctx_hi": 16000, "new": 2, "new_hi": 5,
         "last": 0, "page": 32},
        # a prompt's chunk of 2048 tokens over the 30720 before it
        {"name": "attn_b1_chunk2048", "op": "attn", "batch": 1, "ctx": 30720, "ctx_hi": 30720, "new": 2048,
         "new_hi": 2048, "last": 0, "page": 64},
        # prompts from their first token on, odd lengths
        {"name": "attn_b4_prompts", "op": "attn", "batch": 4, "ctx": 0, "ctx_hi": 0, "new": 611, "new_hi": 1733,
         "last": 0, "page": 128},
        # one token for each of 15 sequences beside one prompt's chunk
        {"name": "attn_b16_mixed", "op": "attn", "batch": 16, "ctx": 2000, "ctx_hi": 12000, "new": 1, "new_hi": 1,
         "last": 700, "page": 64},
        # a whole serving step: tables, append, attention
        {"name": "step_b24_n1", "op": "step", "batch": 24, "ctx": 300, "ctx_hi": 9000, "new": 1, "new_hi": 1,
         "last": 0, "page": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["tables", "append", "attn", "attn", "attn", "attn", "step"])
    page = rng.choice([16, 32, 64, 128])
    if op in ("tables", "append"):
        batch = _log(rng, 1, 512)
        hi = _log(rng, 1, min(4096, (65536 if op == "tables" else 18000) // batch))
        ctx_hi = _log(rng, 1, 8000)
        return {"op": op, "batch": batch, "ctx": rng.randrange(ctx_hi + 1), "ctx_hi": ctx_hi,
                "new": rng.randint(1, hi), "new_hi": hi, "last": 0, "page": page}
    kind = rng.choice(["one", "few", "chunk", "mixed"]) if op == "attn" else "one"
    if kind in ("one", "few"):
        batch = _log(rng, 1, 64)
        ctx_hi = _log(rng, 16, min(131071, (1 << 20) // batch - 16))
        hi = 1 if kind == "one" else rng.randint(2, 12)
        if hi * batch * ctx_hi > 1 << 25:
            ctx_hi = max(16, (1 << 25) // (hi * batch))
        return {"op": op, "batch": batch, "ctx": rng.randrange(ctx_hi // 8, ctx_hi + 1), "ctx_hi": ctx_hi,
                "new": 1 if kind == "one" else rng.randint(2, hi), "new_hi": hi, "last": 0, "page": page}
    if kind == "chunk":
        batch = rng.randint(1, 4)
        hi = _log(rng, 17, 2048 // batch)
        ctx_hi = _log(rng, 1, 30000)
        return {"op": op, "batch": batch, "ctx": rng.randrange(ctx_hi + 1), "ctx_hi": ctx_hi,
                "new": rng.randint(13, hi), "new_hi": hi, "last": 0, "page": page}
    batch = rng.randint(2, 32)
    ctx_hi = _log(rng, 64, 12000)
    return {"op": op, "batch": batch, "ctx": rng.randrange(ctx_hi // 4, ctx_hi + 1), "ctx_hi": ctx_hi, "new": 1,
            "new_hi": rng.randint(1, 3), "last": _log(rng, 17, 1024), "page": page}


def _lengths(case):
    """(cached tokens, new tokens) of each sequence, from the case alone."""
    b = case["batch"]
    lo, hi = min(case["ctx"], case["ctx_hi"]), max(case["ctx"], case["ctx_hi"])
    nlo, nhi = min(case["new"], case["new_hi"]), max(case["new"], case["new_hi"])
    ctx = [hi if i == 0 else lo + int((hi - lo) * ((i * 0.6180339887) % 1.0)) for i in range(b)]
    new = [nhi if i == 0 else nlo + int((nhi - nlo + 1) * ((i * 0.7548776662) % 1.0)) for i in range(b)]
    if case["last"]:
        new[-1] = case["last"]
    return ctx, new


def work(case):
    ctx, new = _lengths(case)
    tokens, rows, page = sum(new), sum(c + n for c, n in zip(ctx, new)), case["page"]
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
    fresh = sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(ctx, new))
    held = sum(-(-(c + n) // page) for c, n in zip(ctx, new))
    # lengths in; seq_lens, q_start, slots (8), positions (4) and new table entries out
    tables = {"bytes": 16 * case["batch"] + 12 * tokens + 8 * fresh + 32, "flops": 2 * tokens}
    append = {"bytes": tokens * (2 * 2 * D + 8), "flops": 0}
    # the cache once, the tables' entries, queries in, W_UV, outputs in bf16
    attn = {"bytes": rows * 2 * D + 4 * held + tokens * HEADS * (2 * D + 2 * D_V) + 2 * HEADS * D_C * D_V,
            "flops": 2 * HEADS * (pairs * (D + D_C) + tokens * D_C * D_V)}
    if case["op"] == "step":
        return {k: tables[k] + append[k] + attn[k] for k in ("bytes", "flops")}
    return {"tables": tables, "append": append, "attn": attn}[case["op"]]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    ctx, new = _lengths(case)
    b, page = case["batch"], case["page"]
    tokens = sum(new)
    lens = [c + n for c, n in zip(ctx, new)]
    held = [-(-n // page) for n in (lens if case["op"] in ("append", "attn") else ctx)]
    blocks = max(-(-n // page) for n in lens) + 1
    n_pages = sum(-(-n // page) for n in lens) + 7
    # pages in the order in which a long-running server hands them out: any
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((b, blocks), -1, dtype=torch.int32, device=dev)
    at = torch.arange(blocks, device=dev)[None, :] < torch.tensor(held, device=dev)[:, None]
    table[at] = perm[:sum(held)]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s = {"op": case["op"], "page": page, "tokens": tokens, "max_new": max(new), "table": table, "ctx": i32(ctx),
         "new": i32(new), "lens": i32(lens), "q_start": i32(start), "made": {}}
    if case["op"] in ("tables", "step"):
        s["free"] = perm[sum(held):].contiguous()
        s["taken"] = i32([3])   # a server does not start from a fresh list
    if case["op"] != "tables":
        s["pages"] = torch.empty(n_pages, page, D, dtype=torch.bfloat16, device=dev)
        for i in range(0, n_pages, 4096):   # latents of unit variance; a rotated N(0, 1) key is N(0, 1)
            s["pages"][i:i + 4096] = torch.randn(min(4096, n_pages - i), page, D, generator=g, device=dev)
    if case["op"] in ("append", "step"):
        s["rows"] = torch.randn(tokens, D, generator=g, device=dev).to(torch.bfloat16)
    if case["op"] == "append":
        pos = torch.cat([torch.arange(c, c + n) for c, n in zip(ctx, new)]).to(dev)
        seq = torch.repeat_interleave(torch.arange(b), torch.tensor(new)).to(dev)
        s["slots"] = table[seq, pos // page].long() * page + pos % page
    if case["op"] in ("attn", "step"):
        # logits of standard deviation 1.7: neither uniform nor one-hot weights
        s["q"] = torch.randn(tokens, HEADS, D, generator=g, device=dev).to(torch.bfloat16)
        s["w_uv"] = (torch.randn(HEADS, D_C, D_V, generator=g, device=dev) / math.sqrt(D_C)).to(torch.bfloat16)
        # sequences with as many new tokens as each other, for the plain form
        s["groups"] = [(n, torch.tensor([i for i in range(b) if new[i] == n], device=dev),
                        max(lens[i] for i in range(b) if new[i] == n)) for n in sorted(set(new)) if n]
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "tables":
        return _plain_tables(s)
    if s["op"] == "append":
        return _plain_append(s["pages"], s["rows"], s["slots"])
    if s["op"] == "attn":
        return _plain_attn(s, s["lens"], s["q_start"])
    lens, q_start, slots, positions, taken, counts, table = _plain_tables(s)
    _plain_append(s["pages"], s["rows"], slots)
    return _plain_attn(s, lens, q_start), lens, q_start, slots, positions, taken, counts, table


def _run_own(s):
    import mla_latent_space_lca_b200 as lca
    made, b = s["made"], s["table"].shape[0]
    if not made:   # buffers that a program keeps from step to step
        dev = s["table"].device
        if s["op"] in ("tables", "step"):
            for name, n, kind in (("seq_lens", b, torch.int32), ("q_start", b + 1, torch.int32),
                                  ("slot_map", s["tokens"], torch.int64), ("positions", s["tokens"], torch.int32),
                                  ("taken_out", 1, torch.int32), ("counts", 4, torch.int32)):
                made[name] = torch.empty(n, dtype=kind, device=dev)
        if s["op"] in ("attn", "step"):
            made["out"] = torch.empty(s["tokens"], HEADS, D_V, dtype=torch.bfloat16, device=dev)
            made["ws"] = lca.paged_workspace(b, s["tokens"], s["max_new"], device=dev)
    lens, q_start, slots = s["lens"], s["q_start"], s.get("slots")
    if s["op"] in ("tables", "step"):
        names = ("seq_lens", "q_start", "slot_map", "positions", "taken_out", "counts")
        lca.lca_page_tables(s["ctx"], s["new"], s["free"], s["taken"], s["table"], s["page"], s["tokens"],
                            **{n: made[n] for n in names})
        tables = tuple(made[n] for n in names) + (s["table"],)
        lens, q_start, slots = tables[:3]
        if s["op"] == "tables":
            return tables
    if s["op"] in ("append", "step"):
        lca.lca_append_paged(s["pages"], s["rows"], slots)
        if s["op"] == "append":
            return s["pages"]
    out = lca.mla_paged_attn(s["pages"], s["table"], lens, q_start, s["q"], s["w_uv"], s["max_new"], scale=SCALE,
                             out=made["out"], ws=made["ws"])
    return out if s["op"] == "attn" else (out,) + tables


def _plain_tables(s):
    page, table, free = s["page"], s["table"], s["free"]
    b, blocks = table.shape
    ctx = s["ctx"].long().clamp(0, blocks * page)
    want = torch.minimum(s["new"].long().clamp(min=0), blocks * page - ctx)
    end = torch.cumsum(want, 0).clamp(max=s["tokens"])
    start = torch.cat([end.new_zeros(1), end[:-1]])
    lens = ctx + end - start
    old, have = (ctx + page - 1) // page, (lens + page - 1) // page
    need = have - old
    taken = s["taken"].long().clamp(0, free.numel())
    first = taken + torch.cumsum(need, 0) - need
    block = torch.arange(blocks, device=table.device)[None, :]
    fresh = (block >= old[:, None]) & (block < have[:, None])
    pick = first[:, None] + block - old[:, None]
    page_of = free[pick.clamp(0, free.numel() - 1)]
    table.copy_(torch.where(fresh, torch.where(pick < free.numel(), page_of, -1), table))
    t = torch.arange(s["tokens"], device=table.device)
    seq = torch.searchsorted(end, t, right=True).clamp(max=b - 1)
    used = t < end[-1]
    pos = ctx[seq] + t - start[seq]
    held = table[seq, (pos // page).clamp(0, blocks - 1)].long()
    slots = torch.where(used & (held >= 0), held * page + pos % page, -1)
    total = need.sum()
    got = torch.minimum(total, free.numel() - taken[0])
    counts = torch.stack([end[-1], s["new"].long().clamp(min=0).sum() - end[-1], got, total - got])
    return (lens.int(), torch.cat([start, end[-1:]]).int(), slots, torch.where(used, pos, -1).int(),
            (taken + got).int(), counts.int(), table)


def _plain_append(pages, rows, slots):
    pages.view(-1, D)[slots] = rows
    return pages


def _plain_attn(s, lens, q_start):
    page, table = s["page"], s["table"]
    out = torch.empty(s["tokens"], HEADS, D_V, dtype=torch.bfloat16, device=table.device)
    w_uv = s["w_uv"].float()
    for n, idx, longest in s["groups"]:
        ids = table[idx, :-(-longest // page)].clamp(min=0)
        rows = s["pages"][ids].reshape(len(idx), -1, D)[:, :longest].float()
        token = q_start[idx].long()[:, None] + torch.arange(n, device=table.device)
        q = s["q"][token].float().reshape(len(idx), n * HEADS, D)
        z = (torch.bmm(q, rows.transpose(1, 2)) * SCALE).view(len(idx), n, HEADS, longest)
        pos = lens[idx][:, None] - n + torch.arange(n, device=table.device)
        z.masked_fill_((torch.arange(longest, device=table.device) > pos[:, :, None])[:, :, None], -math.inf)
        z -= z.amax(-1, keepdim=True)
        z.exp_()
        z /= z.sum(-1, keepdim=True)
        o = torch.bmm(z.view(len(idx), n * HEADS, longest), rows[:, :, :D_C])
        o = o.view(-1, HEADS, D_C).transpose(0, 1)
        out[token.reshape(-1)] = torch.bmm(o, w_uv).transpose(0, 1).to(torch.bfloat16)
    return out


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    ctx, new = _lengths(case)
    page = case["page"]
    tables = None
    if case["op"] in ("tables", "step"):
        table, free, used = s["table"].cpu().clone(), s["free"].cpu().tolist(), int(s["taken"])
        slots, positions, began, first = [], [], [], used
        for b, (c, n) in enumerate(zip(ctx, new)):
            began.append(len(slots))
            for p in range(c, c + n):
                if p % page == 0:
                    table[b, p // page] = free[used] if used < len(free) else -1
                    used += 1
            ids = table[b].tolist()
            slots += [ids[p // page] * page + p % page if ids[p // page] >= 0 else -1 for p in range(c, c + n)]
            positions += list(range(c, c + n))
        got = min(used, len(free))
        i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
        tables = (i32([c + n for c, n in zip(ctx, new)]), i32(began + [len(slots)]), torch.tensor(slots),
                  i32(positions), i32([got]), i32([len(slots), 0, got - first, used - got]), table)
        if case["op"] == "tables":
            return tables
        slots = torch.tensor(slots, device="cuda")
    else:
        table, slots = s["table"], s.get("slots")
    pages = s["pages"].clone()
    if case["op"] in ("append", "step"):
        good = slots >= 0
        pages.view(-1, D).index_copy_(0, slots[good], s["rows"][good])
        if case["op"] == "append":
            return pages
    outs, w_uv, t, ids = [], s["w_uv"].double(), 0, table.cpu()
    for b, (c, n) in enumerate(zip(ctx, new)):
        rows = torch.cat([pages[i] for i in ids[b, :-(-(c + n) // page)].tolist()])[:c + n].double()
        for i in range(0, n, 64):
            m = min(64, n - i)
            z = torch.einsum("thd,ld->thl", s["q"][t + i:t + i + m].double(), rows) / math.sqrt(192.0)
            hidden = torch.ones(m, c + n, dtype=torch.bool, device="cuda").triu(c + i + 1)
            p = torch.softmax(z.masked_fill(hidden[:, None], -math.inf), -1)
            o = torch.einsum("thl,lc->thc", p, rows[:, :D_C])
            outs.append(torch.einsum("thc,hcv->thv", o, w_uv))
        t += n
    out = torch.cat(outs)
    return out if case["op"] == "attn" else (out,) + tables
