"""What the bindings of the paged cache pass on to the library, and what they
refuse, on the host (no GPU): tensors without memory on a CUDA device."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import mla_latent_space_lca_b200 as lca
from mla_latent_space_lca_b200 import api


@pytest.fixture
def calls(monkeypatch, lcalib):
    """The arguments of every call that reaches the library."""
    made = []

    def on(dev, stream, fn, *args):
        made.append(args)
        return 0

    monkeypatch.setattr(api, "_on", on)
    with FakeTensorMode():
        yield made


def cuda(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
@pytest.mark.parametrize("width", [576, 577, 580, 584, 1000])
@pytest.mark.parametrize("T", [0, 1])
def test_append_of_one_row_whatever_its_stride(calls, T, width):
    lca.lca_append_paged(cuda(4, 16, 576), cuda(T, width)[:, :576], cuda(T, dtype=torch.int64))
    assert len(calls) == 1 and calls[0][1] % 8 == 0 and calls[0][3] == T


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_append_keeps_the_pitch_of_several_rows(calls):
    lca.lca_append_paged(cuda(4, 16, 576), cuda(3, 640)[:, :576], cuda(3, dtype=torch.int64))
    lca.lca_append_paged(cuda(4, 16, 576), cuda(3, 580)[:, :576], cuda(3, dtype=torch.int64))   # the library refuses it
    assert [c[1] for c in calls] == [640, 580]


def attention_args(T=6, B=2):
    i32 = lambda *shape: cuda(*shape, dtype=torch.int32)  # noqa: E731
    return cuda(4, 16, 576), i32(B, 2), i32(B), i32(B + 1), cuda(T, 16, 576), cuda(16, 512, 128)


def test_workspace_without_memory_of_its_own(calls):
    # as many bytes as it needs by its shape, one by its memory
    ws = cuda(1, dtype=torch.uint8).expand(1 << 30)
    with pytest.raises(ValueError, match="ws"):
        lca.mla_paged_attn(*attention_args(), 3, ws=ws)
    with pytest.raises((TypeError, ValueError), match="ws"):
        lca.mla_paged_attn(*attention_args(), 3, ws=torch.empty(1 << 30, dtype=torch.uint8))
    assert not calls


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
@pytest.mark.parametrize("max_new", [2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 40])
def test_most_new_tokens_beyond_32_bits(calls, max_new):
    # any number: 2^32 + 1 is not the single-token form's 1, nor 2^32 no number at all
    lca.mla_paged_attn(*attention_args(), max_new)
    (args,) = calls
    assert args[10:12] == (6, 2 ** 31 - 1)   # T, max_new
    assert lca.paged_workspace(2, 6, max_new).numel() == lca.paged_workspace(2, 6, 2).numel() == args[15]


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
@pytest.mark.parametrize("page_size", [2 ** 32 + 16, 2 ** 31, -2 ** 32 + 64])
def test_page_size_beyond_32_bits(calls, page_size):
    i32 = lambda *shape: cuda(*shape, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="page_size"):
        lca.lca_page_tables(i32(2), i32(2), i32(9), i32(1), i32(2, 4), page_size, 8)
    assert not calls


def test_workspace_on_the_device_named(monkeypatch, lcalib):
    asked = []
    monkeypatch.setattr(api.torch, "empty", lambda *a, **kw: asked.append(kw["device"]))
    lca.paged_workspace(1, 1, 1, device=0)   # whichever device is current
    lca.workspace(3, 1, 2048, device=0)
    lca.paged_workspace(1, 1, 1)
    assert asked == [0, 0, "cuda"]
