"""Size limits of the paged-cache entry points at their edges, on the host (no
GPU): what is refused, and what is not refused for its size."""
import pytest

from mla_latent_space_lca_b200 import _lib

from test_paged_abi import ATTN, TABLES, call

OK, WS, UNS = _lib.LCA_OK, _lib.LCA_ERR_WORKSPACE, _lib.LCA_ERR_UNSUPPORTED


@pytest.mark.parametrize("page", [16, 64, 65536])
def test_rows_of_a_cache(lcalib, page):
    # ws=None: a size that is accepted goes on to the workspace check
    most = (2 ** 31 - 1024) // page
    for key in ("n_pages", "blocks"):
        assert call(lcalib.mla_paged_attn, list(ATTN), ATTN, {"page": page, "max_new": 4, key: most, "ws": None}) == WS
        assert call(lcalib.mla_paged_attn, list(ATTN), ATTN, {"page": page, "max_new": 4, key: most + 1, "ws": None}) == UNS


def test_single_tokens_are_bounded_by_their_tiles(lcalib):
    kw = dict(T=1 << 14, blocks=1 << 16, page=64, ws=None)   # 2^14 tokens x 2^16 tiles
    assert call(lcalib.mla_paged_attn, list(ATTN), ATTN, dict(kw, max_new=1)) == UNS
    assert call(lcalib.mla_paged_attn, list(ATTN), ATTN, dict(kw, max_new=2)) == WS
    assert call(lcalib.mla_paged_attn, list(ATTN), ATTN, dict(kw, blocks=(1 << 16) - 1, max_new=1)) == WS


def test_workspace_grows_with_the_batch(lcalib):
    size = lcalib.mla_paged_workspace_bytes
    for new in (1, 2, 4096):
        last = 0
        for T in (1, 8, 9, 4096, 1 << 20):
            n = size(64, T, new)
            assert n >= last
            last = n
    assert size(1, (1 << 27) - 1, 4) > 0 and size(1, 1 << 27, 4) == 0
    # o as two bf16 values a token, whatever else
    assert size(8, 1000, 4) > 1000 * 16 * 2 * 512 * 2


def test_tables_at_their_limits(lcalib):
    most = 0x7FFFFFFF // 64
    assert call(lcalib.lca_page_tables, list(TABLES), TABLES, dict(blocks=most + 1)) == UNS
    assert call(lcalib.lca_page_tables, list(TABLES), TABLES, dict(tokens=1 << 30)) == UNS
