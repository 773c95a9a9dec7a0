"""lca_append_paged of a single row that is a slice of a wider one."""
import pytest
import torch

import mla_latent_space_lca_b200 as lca

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width", [577, 580, 583, 584])
def test_append_of_one_row_whatever_its_stride(width):
    pages = torch.zeros(3, 16, 576, dtype=torch.bfloat16, device="cuda")
    rows = torch.randn(1, width, device="cuda").to(torch.bfloat16)[:, :576]
    lca.lca_append_paged(pages, rows, torch.tensor([20], device="cuda"))
    want = torch.zeros_like(pages)
    want[1, 4] = rows[0]
    assert torch.equal(pages, want)


def test_rows_at_a_pitch_that_is_no_multiple_of_16_bytes_are_refused():
    pages = torch.zeros(3, 16, 576, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(lca._lib.LcaError):
        lca.lca_append_paged(pages, torch.zeros(2, 580, device="cuda").bfloat16()[:, :576],
                             torch.tensor([1, 2], device="cuda"))
