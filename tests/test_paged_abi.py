"""Refusals of the paged-cache entry points, on the host (no GPU): every
invalid argument is rejected before anything is launched."""
import pytest
import torch

import mla_latent_space_lca_b200 as lca
from mla_latent_space_lca_b200 import _lib

from paged_ref import tables

A = 0x7F0000000000   # never dereferenced
INV, MIS, WS, UNS = (_lib.LCA_ERR_INVALID_ARG, _lib.LCA_ERR_MISALIGNED, _lib.LCA_ERR_WORKSPACE,
                     _lib.LCA_ERR_UNSUPPORTED)


def call(fn, order, base, kw):
    a = dict(base)
    a.update(kw)
    return fn(*[a[k] for k in order])


TABLES = dict(ctx=A, new=A, free=A, n_free=100, taken=A, table=A, B=4, blocks=16, page=64, tokens=128, lens=A,
              start=A, slots=A, pos=A, out=A, counts=A, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(ctx=None), INV), (dict(new=None), INV), (dict(taken=None), INV), (dict(table=None), INV),
    (dict(lens=None), INV), (dict(start=None), INV), (dict(out=None), INV), (dict(free=None), INV),
    (dict(slots=None), INV), (dict(B=0), INV), (dict(blocks=0), INV), (dict(page=0), INV), (dict(tokens=-1), INV),
    (dict(n_free=-1), INV), (dict(n_free=1 << 31), INV), (dict(page=48), UNS), (dict(page=8), UNS),
    (dict(page=1 << 17), UNS), (dict(B=_lib.PAGED_MAX_BATCH + 1), UNS), (dict(tokens=1 << 30), UNS),
    (dict(blocks=1 << 26), UNS), (dict(slots=A + 4), MIS), (dict(ctx=A + 2), MIS), (dict(counts=A + 1), MIS),
])
def test_page_tables_refusals(lcalib, kw, status):
    assert call(lcalib.lca_page_tables, list(TABLES), TABLES, kw) == status


APPEND = dict(rows=A, pitch=576, slots=A, T=4, pages=A, n_pages=10, page=64, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=None), INV), (dict(slots=None), INV), (dict(pages=None), INV), (dict(T=-1), INV),
    (dict(n_pages=0), INV), (dict(page=0), INV), (dict(pitch=568), INV), (dict(pitch=580), MIS),
    (dict(page=24), UNS), (dict(n_pages=1 << 40), INV), (dict(rows=A + 8), MIS), (dict(pages=A + 2), MIS),
    (dict(slots=A + 4), MIS), (dict(T=0), _lib.LCA_OK),
])
def test_append_refusals(lcalib, kw, status):
    assert call(lcalib.lca_append_paged, list(APPEND), APPEND, kw) == status


ATTN = dict(pages=A, n_pages=10, page=64, table=A, blocks=4, lens=A, start=A, q=A, w_uv=A, B=2, T=2, max_new=1,
            scale=0.07, out=A, ws=A, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(pages=None), INV), (dict(table=None), INV), (dict(lens=None), INV), (dict(start=None), INV),
    (dict(q=None), INV), (dict(w_uv=None), INV), (dict(out=None), INV), (dict(B=0), INV), (dict(T=-1), INV),
    (dict(n_pages=0), INV), (dict(blocks=0), INV), (dict(max_new=0), INV), (dict(scale=0.0), INV),
    (dict(scale=float("nan")), INV), (dict(page=20), UNS), (dict(n_pages=1 << 26), UNS), (dict(blocks=1 << 26), UNS),
    (dict(T=1 << 27), UNS), (dict(T=1 << 20, blocks=1 << 20), UNS), (dict(pages=A + 8), MIS), (dict(q=A + 2), MIS),
    (dict(out=A + 4), MIS), (dict(table=A + 2), MIS), (dict(ws=None), WS), (dict(ws_bytes=100), WS),
    (dict(ws=A + 128), MIS), (dict(T=0), _lib.LCA_OK),
])
def test_attention_refusals(lcalib, kw, status):
    assert call(lcalib.mla_paged_attn, list(ATTN), ATTN, kw) == status


def test_workspace_bytes(lcalib):
    assert lcalib.mla_paged_workspace_bytes(0, 4, 1) == 0
    assert lcalib.mla_paged_workspace_bytes(4, 0, 1) == 0
    assert lcalib.mla_paged_workspace_bytes(4, 4, 0) == 0
    for T in (1, 7, 4096):
        for new in (1, 5):
            n = lcalib.mla_paged_workspace_bytes(3, T, new)
            assert n > 0 and n % 256 == 0


def test_bindings_refuse_host_tensors(lcalib):
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError):
        lca.lca_page_tables(i, i, i, i[:1], i.view(4, 1), 16, 8)
    with pytest.raises(TypeError):
        lca.lca_append_paged(torch.zeros(2, 16, 576, dtype=torch.bfloat16),
                             torch.zeros(2, 576, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64))


def test_reference_tables_by_hand():
    # 2 sequences, pages of 16: 15 + 3 rows need one page more, 16 + 1 one too
    t = [[7, -1, -1], [5, -1, -1]]
    got = tables([15, 16], [3, 1], [9, 8, 4], 1, t, 16, 6)
    assert got == ([18, 17], [0, 3, 4], [7 * 16 + 15, 8 * 16, 8 * 16 + 1, 4 * 16, -1, -1],
                   [15, 16, 17, 16, -1, -1], 3, [4, 0, 2, 0], [[7, 8, -1], [5, 4, -1]])
    # the list runs out, and the batch has room for two tokens only
    t = [[7, -1], [5, -1]]
    got = tables([16, 15], [1, 9], [], 0, t, 16, 2)
    assert got == ([17, 16], [0, 1, 2], [-1, 5 * 16 + 15], [16, 15], 0, [2, 8, 0, 1], [[7, -1], [5, -1]])
