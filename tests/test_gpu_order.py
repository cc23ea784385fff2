"""Calls back to back on one stream, without a synchronisation between them: each reads what the
one before it wrote."""
import numpy as np
import pytest
import torch

import _spec_ref as R
import mxfp4_sparse_paged_gb300 as m

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = "cuda"


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


class Select:
    """Index pages, queries and buffers of index_topk over B sequences."""

    def __init__(self, seed, lens, k, ld):
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.k, self.ld = np.asarray(lens, np.int32), k, ld
        B = len(lens)
        self.bt, self.P = R.block_table(rng, lens)
        self.idx = dev(R.random_pages(rng, self.P, 1)[:, 0])
        self.iq = torch.randn((40, B, 128), generator=torch.Generator(device=DEV).manual_seed(seed),
                              device=DEV).to(torch.bfloat16)
        self.scores = torch.zeros((B, ld), device=DEV)
        need = m.index_topk_workspace(B, k, ld)
        self.ws = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None

    def call(self, i, table, lens, out):
        m.index_topk(self.iq[i], 1, self.idx, table, lens, self.scores, self.k, out, self.ws)


def test_short_rows_of_wide_scores_are_selected_after_they_are_written():
    # no row is long enough for the filter that the width of the scores asks for: its kernels have
    # nothing to do between the scorer and the selection
    a = Select(1, [int(x) for x in np.random.default_rng(1).integers(100, 8000, 64)], 60, 20000)
    table, lens = dev(a.bt), dev(a.lens)
    got = [torch.full((64, a.k), -7, dtype=torch.int32, device=DEV) for _ in range(40)]
    for i in range(40):
        a.call(i, table, lens, got[i])
    for i in range(40):
        want = torch.empty_like(got[i])
        m.index_score(a.iq[i], 1, a.idx, table, lens, a.scores)
        torch.cuda.synchronize()
        m.topk_select(a.scores, lens, 1, a.k, want, a.ws)
        torch.cuda.synchronize()
        assert torch.equal(got[i], want)
    assert m.mx4_check_status() == 0


@pytest.mark.parametrize("ld", [1024, 20000])  # without and with the filter's kernels
@pytest.mark.parametrize("call", ["index_topk", "topk_select", "index_score"])
def test_lengths_that_accept_wrote_are_read_by_the_selection(ld, call):
    # rows shorter than k, so that the selection shows the length that was read; a different
    # number of accepted rows every time
    B, N, k = 64, 16, 512
    a = Select(2, [int(x) for x in np.random.default_rng(2).integers(N + 1, 400, B)], k, ld)
    table, lens, pool = dev(a.bt), dev(a.lens), torch.zeros((a.P, 1, 8704), dtype=torch.uint8, device=DEV)
    path = dev(np.tile(np.arange(N, dtype=np.int32), (B, 1)))
    acc = dev(a.rng.integers(0, N + 1, (40, B)).astype(np.int32))
    new = torch.zeros((B,), dtype=torch.int32, device=DEV)
    out = [torch.full((B, k), -7, dtype=torch.int32, device=DEV) for _ in range(40)]
    marked = [torch.full((B, ld), -7.0, device=DEV) for _ in range(40 if call == "index_score" else 0)]
    for i in range(40):
        m.mx4_accept_rows(path, acc[i], lens, table, pool, pool, None, new)
        if call == "index_topk":
            a.call(i, table, new, out[i])
        elif call == "topk_select":
            m.topk_select(a.scores, new, 1, k, out[i], a.ws)
        else:
            m.index_score(a.iq[i], 1, a.idx, table, new, marked[i])
    assert m.mx4_check_status() == 0
    for i in range(40):
        n = lens - N + acc[i]
        if call == "index_score":
            assert torch.equal((marked[i] != -7.0).sum(1).to(torch.int32), n)
        else:
            at = torch.arange(k, device=DEV)
            assert torch.equal(out[i], torch.where(at < n[:, None], at, -1).to(torch.int32))


def test_tables_and_lengths_that_fork_wrote_are_read_by_the_selection():
    # children of other rows every time, in the same tables: the scores are those of the parents
    B, n, k, ld = 6, 48, 40, 20000
    a = Select(3, [300, 128, 5000, 77, 1000, 9000], k, ld)
    P = a.P + 4 * n
    idx = torch.zeros((P, 8704), dtype=torch.uint8, device=DEV)
    idx[:a.P] = a.idx
    a.idx = idx
    kp = torch.zeros((P, 1, 8704), dtype=torch.uint8, device=DEV)
    refs = torch.zeros((P,), dtype=torch.int32, device=DEV)
    refs[torch.from_numpy(a.bt[a.bt >= 0]).long().to(DEV)] = 1
    left = np.setdiff1d(np.arange(P), a.bt[a.bt >= 0]).astype(np.int32)
    fl = dev(np.concatenate((left, np.full(P - len(left), -1, np.int32))))
    fc = dev(np.array([len(left)], np.int32))
    table, lens = dev(a.bt), dev(a.lens)
    child = torch.zeros((n, a.bt.shape[1]), dtype=torch.int32, device=DEV)
    cl = torch.zeros((n,), dtype=torch.int32, device=DEV)
    rows = dev(a.rng.integers(0, B, (40, n)).astype(np.int32))
    iq = torch.randn((B, 128), generator=torch.Generator(device=DEV).manual_seed(4), device=DEV).to(torch.bfloat16)
    need = m.index_topk_workspace(n, k, ld)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    scores = torch.zeros((n, ld), device=DEV)
    out = [torch.full((n, k), -7, dtype=torch.int32, device=DEV) for _ in range(40)]
    q = [iq[rows[i].long()].contiguous() for i in range(40)]
    torch.cuda.synchronize()
    for i in range(40):
        m.mx4_fork_pages(rows[i], table, lens, refs, fl, fc, kp, kp, idx, child, cl)
        m.index_topk(q[i], 1, idx, child, cl, scores, k, out[i], ws)
        m.mx4_free_pages(child, cl, refs, fl, fc)
    assert m.mx4_check_status() == 0 and int(fc) == len(left)
    want = torch.empty((B, k), dtype=torch.int32, device=DEV)
    m.index_topk(iq, 1, idx, table, lens, scores[:B], k, want, ws)
    torch.cuda.synchronize()
    for i in range(40):
        assert torch.equal(out[i], want[rows[i].long()])
