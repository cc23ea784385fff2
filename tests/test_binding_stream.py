"""The stream that the binding hands to the library, on the CPU."""
import types

import pytest
import torch

import mxfp4_sparse_paged_gb300 as m
from mxfp4_sparse_paged_gb300 import build as B_


@pytest.fixture(autouse=True)
def other_torch(monkeypatch):
    """A torch without the call that gives the current stream's address."""
    B_.build()
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)


def test_the_public_call_gives_the_current_stream(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=4096))
    assert m._stream(None) == 4096


@pytest.mark.parametrize("error", [RuntimeError, AssertionError])
def test_arguments_are_looked_at_where_there_is_no_cuda(monkeypatch, error):
    def none():
        raise error("no CUDA")

    monkeypatch.setattr(torch.cuda, "current_stream", none)
    i32 = torch.int32
    with pytest.raises(ValueError, match="CUDA tensor"):
        m.mx4_free_pages(torch.zeros((2, 3), dtype=i32), torch.zeros(2, dtype=i32),
                         torch.zeros(5, dtype=i32), torch.zeros(5, dtype=i32), torch.zeros(1, dtype=i32))
