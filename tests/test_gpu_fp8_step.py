"""A step over the 8-bit cache when something is wrong: refused calls, sequences without a page."""
import pytest
import torch

import mxfp4_sparse_paged_gb300 as m
from mxfp4_sparse_paged_gb300.fp8_step import Fp8Caches, Fp8Step
from test_gpu_fp8_kv import clean, flagged  # noqa: F401 (clean: a fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, H, HKV, PROMPT = 3, 8, 2, 250


def filled(seed=0, lens=(PROMPT,) * B, table=((3, 5, 0), (1, 6, 2), (4, 7, 8)), blocks=2, **kw):
    """A step after its prompts, and the inputs of three steps."""
    g = torch.Generator(DEV).manual_seed(seed)
    caches = Fp8Caches(9, HKV, index_scale=0.02)
    step = Fp8Step(caches, torch.tensor(table, dtype=torch.int32, device=DEV),
                   torch.zeros(B, dtype=torch.int32, device=DEV), heads=H, blocks=blocks, first=0, last=1,
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


@pytest.mark.parametrize("q", [1, 3])
@pytest.mark.parametrize("blocks", [0, 2])
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("page", [-1, 9, None])
def test_a_sequence_without_a_page_sits_out(q, blocks, captured, page):
    """The second of three has no page for its tokens past 256 (no entry, one past the pool, the
    table's end): from there its length and its bytes stay and its results are zeros; with a page it
    goes on as if it had waited.  The others: the results of steps in which nothing is wrong."""
    first = 256 - PROMPT  # tokens until the page ends
    lens = (PROMPT + first,) * B
    if page is None:
        lens = (PROMPT, 3 * 128 - q + 1, PROMPT)
    step, ins = filled(lens=lens, q_per_seq=q, blocks=blocks)
    other, _ = filled(lens=lens, q_per_seq=q, blocks=blocks)
    good = step.block_table.clone()
    if page is not None:
        step.block_table[1, 2] = page
    run = step.run
    if captured:
        held = [x.clone() for x in ins[0]]
        keep = step.seq_lens.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step.run(*held)

        def run(*x):
            for a, b in zip(held, x):
                a.copy_(b)
            graph.replay()
            return step.out
        assert torch.equal(step.seq_lens, keep)

    def same(a, b):
        """Lists: bit for bit.  Dense calls cut a batch by its units, so that fp32 sums go another way
        (2^-20) and a bf16 number may be the next one (2^-7)."""
        a, b = a.double(), b.double()
        return bool(((a - b).abs() <= (0.0 if blocks else 2.0**-7 if a.dim() == 3 else 2.0**-20) * b.abs()).all())
    mine = slice(q, 2 * q)
    rest = [t for t in range(B * q) if not q <= t < 2 * q]
    pages = good[1].long()
    for x in ins[:2]:
        had = [p[pages].clone() for p in step.caches.kv()]
        want = other.run(*x)
        m.mx4_check_status() if page is not None else flagged(0x5)
        got = run(*x)
        flagged(0x5)  # bad-slot, bad-len
        assert step.seq_lens[1] == lens[1]
        assert torch.equal(step.seq_lens[::2], other.seq_lens[::2])
        assert same(got[rest], want[rest]) and same(step.lse[rest], other.lse[rest])
        assert (got[mine] == 0).all() and (step.lse[mine] == -float("inf")).all()
        if blocks:
            assert (step.block_idx[mine] == -1).all()
        assert all(torch.equal(a, p[pages]) for a, p in zip(had, step.caches.kv()))
    if page is None:
        return
    step.block_table.copy_(good)
    waited, _ = filled(lens=lens, q_per_seq=q, blocks=blocks)
    got, want = run(*ins[2]), waited.run(*ins[2])
    assert same(got[mine], want[mine]) and step.seq_lens[1] == lens[1] + q
    m.mx4_check_status()


def test_a_prompt_without_a_page_sits_out():
    """Prompts of which one reaches past its pages, one past the rows, one brings nothing."""
    g = torch.Generator(DEV).manual_seed(1)
    i = dict(dtype=torch.int32, device=DEV)
    for cu, new, out in (([0, 300, 600, 650], [300, 300, 50], [1]), ([0, 300, 300, 651], [300, 0, 351], [2]),
                         ([0, 385, 400, 640], [385, 15, 240], [0])):
        caches = Fp8Caches(9, HKV)
        table = torch.tensor([[3, 5, 0], [1, 6, -1], [4, 7, 8]], **i)
        step = Fp8Step(caches, table, torch.zeros(B, **i), heads=H, blocks=0)
        k, v = (torch.randn((650, HKV, 128), generator=g, device=DEV) for _ in range(2))
        step.append(k, v, torch.randn((650, 128), generator=g, device=DEV), torch.tensor(cu, **i), torch.tensor(new, **i))
        flagged(0x4 if cu[-1] > 650 else 0x5)
        assert step.seq_lens.tolist() == [0 if s in out else n for s, n in enumerate(new)]
        for s in out:
            held = table[s][table[s] >= 0].long()
            assert (caches.k_pages[held] == 255).all() and (caches.v_scales[held] == 255).all()
