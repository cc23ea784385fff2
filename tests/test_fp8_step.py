"""The state of a step over the 8-bit cache, on the CPU: calls are refused there at their first
device check, before any kernel."""
import pytest
import torch

from mxfp4_sparse_paged_gb300 import build
from mxfp4_sparse_paged_gb300.fp8_step import Fp8Caches, Fp8Step


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def step_of(lens=(130, 257), blocks=4, q=1, pages=7, table=((3, 5, -1), (1, 6, 2)), **kw):
    caches = Fp8Caches(pages, 2, device="cpu")
    return Fp8Step(caches, torch.tensor(table, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32), q, 4,
                   blocks, **kw)


def rows(T, H=4, Hkv=2):
    bf = torch.bfloat16
    return (torch.zeros((T, H, 128), dtype=bf), torch.zeros((T, Hkv, 128), dtype=bf),
            torch.zeros((T, Hkv, 128), dtype=bf), torch.zeros((T, 128), dtype=bf), torch.zeros((T, 128)))


def test_refused_calls_leave_the_lengths():
    """Any exception of a step or an append, whichever of its calls refuses: seq_lens as before."""
    for blocks in (0, 4):
        step = step_of(blocks=blocks)
        with pytest.raises((ValueError, TypeError)):
            step.run(*rows(2))
        assert step.seq_lens.tolist() == [130, 257]
        q, k, v, _, idx_k = rows(5)
        with pytest.raises((ValueError, TypeError)):
            step.append(k, v, idx_k, torch.tensor([0, 3, 5], dtype=torch.int32),
                        torch.tensor([3, 2], dtype=torch.int32))
        assert step.seq_lens.tolist() == [130, 257]


@pytest.mark.parametrize("kw", [dict(blocks=2), dict(blocks=1, first=0, last=2), dict(blocks=-1),
                                dict(blocks=4, first=-1), dict(blocks=4, last=-1), dict(blocks=4, first=3, last=2)])
def test_choices_of_blocks_are_refused_at_once(kw):
    with pytest.raises(ValueError, match="blocks"):
        step_of(**kw)


@pytest.mark.parametrize("kw", [dict(blocks=3), dict(blocks=0), dict(blocks=1, first=0, last=1),
                                dict(blocks=5, first=3, last=2), dict(blocks=2, first=0, last=0)])
def test_choices_of_blocks(kw):
    assert step_of(**kw).blocks == kw["blocks"]


def test_8_bit_caches_do_not_fork():
    """mx4_fork_pages copies MXFP4 rows: children of an 8-bit cache are refused, not left with a page
    whose rows and scales are another's."""
    from mxfp4_sparse_paged_gb300.speculate import PageBook
    table = torch.tensor([[0, 1]], dtype=torch.int32)
    book = PageBook(4, table)
    with pytest.raises(ValueError, match="MXFP4"):
        book.fork(torch.zeros(2, dtype=torch.int32), table, torch.tensor([130], dtype=torch.int32),
                  Fp8Caches(4, device="cpu"))
