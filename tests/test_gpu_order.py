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
