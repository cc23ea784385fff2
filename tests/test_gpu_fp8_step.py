"""A step over the 8-bit cache when something is wrong: refused calls, sequences without a page."""
import pytest
import torch

import mxfp4_sparse_paged_gb300 as m
from mxfp4_sparse_paged_gb300.fp8_step import Fp8Caches, Fp8Step
from test_gpu_fp8_kv import clean, flagged  # noqa: F401 (clean: a fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, H, HKV, PROMPT = 3, 8, 2, 250


def filled(seed=0, lens=(PROMPT,) * B, table=((3, 5, 0), (1, 6, 2), (4, 7, 8)), **kw):
    """A step after its prompts, and the inputs of three steps."""
    g = torch.Generator(DEV).manual_seed(seed)
    caches = Fp8Caches(9, HKV, index_scale=0.02)
    step = Fp8Step(caches, torch.tensor(table, dtype=torch.int32, device=DEV),
                   torch.zeros(B, dtype=torch.int32, device=DEV), heads=H, blocks=2, first=0, last=1,
                   phases=m.rope_phases(m.rope_frequencies(128)[0].to(DEV)), **kw)
    draw = lambda *s: torch.randn(s, generator=g, device=DEV)
    n = sum(lens)
    cu = torch.tensor([0] + list(lens), device=DEV).cumsum(0).to(torch.int32)
    step.append(draw(n, HKV, 128), draw(n, HKV, 128), draw(n, 128), cu,
                torch.tensor(lens, dtype=torch.int32, device=DEV))
    T = B * step.q
    ins = [(draw(T, H, 128), draw(T, HKV, 128), draw(T, HKV, 128), draw(T, 128).to(torch.bfloat16), draw(T, 128))
           for _ in range(3)]
    return step, ins


def test_a_refused_step_is_run_again():
    """Arguments of a wrong shape, in each place: the lengths stay, and the steps that follow give
    the bits of steps that nothing refused."""
    step, ins = filled()
    other, _ = filled()
    for x in ins:
        for i in range(5):
            bad = list(x)
            bad[i] = x[i][:, :-1].contiguous() if i in (0, 3, 4) else x[i][:-1].contiguous()
            before = step.seq_lens.tolist()
            with pytest.raises((ValueError, TypeError)):
                step.run(*bad)
            assert step.seq_lens.tolist() == before
        assert torch.equal(step.run(*x), other.run(*x))
        assert torch.equal(step.seq_lens, other.seq_lens) and torch.equal(step.lse, other.lse)
    m.mx4_check_status()
