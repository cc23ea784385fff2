"""Indices that the speculative step's torch code uses, on the CPU: none reaches a gather out of
range (which on a GPU ends the process), and what is bad is left for the calls to report."""
import types

import numpy as np
import pytest
import torch

import _spec_ref as R
from mxfp4_sparse_paged_gb300 import build as B_, speculate
from mxfp4_sparse_paged_gb300.speculate import SpeculativeStep, tree_masks


@pytest.fixture(scope="module", autouse=True)
def lib():
    B_.build()


def step_of(table, seq_lens, nodes, P):
    pool = torch.zeros((P, 1, 8704), dtype=torch.uint8)
    caches = types.SimpleNamespace(num_pages=P, k_pages=pool, v_pages=pool)
    return SpeculativeStep(caches, torch.tensor(table, dtype=torch.int32),
                           torch.tensor(seq_lens, dtype=torch.int32), nodes)


def test_slots_of_a_table_with_room():
    s = step_of([[3, 5], [7, 0]], [126, 10], 4, 8)
    s.n_nodes[1] = 2
    assert s.slots().tolist() == [3 * 128 + 126, 3 * 128 + 127, 5 * 128, 5 * 128 + 1,
                                  7 * 128 + 10, 7 * 128 + 11, -1, -1]


def test_slots_past_a_table_and_without_a_page_are_flagged_by_the_insert():
    # the last rows of a full table; a row whose next page is none; a page outside the pool; a
    # negative length: slots that no pool has (mx4_insert reports those), none negative, which
    # the insert would skip
    P = 8
    s = step_of([[3, 5], [7, -1], [1, P + 3], [2, 4], [6, -1]], [254, 127, 127, -1, 300], 4, P)
    bad = lambda x: x >= P * 128
    got = s.slots().view(5, 4).tolist()
    assert got[0][:2] == [5 * 128 + 126, 5 * 128 + 127] and all(map(bad, got[0][2:]))
    assert got[1][0] == 7 * 128 + 127 and all(map(bad, got[1][1:]))
    assert got[2][0] == 1 * 128 + 127 and all(map(bad, got[2][1:]))
    assert bad(got[3][0]) and got[3][1:] == [2 * 128, 2 * 128 + 1, 2 * 128 + 2]
    assert all(map(bad, got[4]))
    s.n_nodes.zero_()
    assert s.slots().tolist() == [-1] * 20


def test_tree_masks_of_parents_that_are_none():
    # parents past the nodes, after their node, below -1: roots of their own, as verify_drafts
    # takes their nodes out (and reports them); the root's own entry is not read
    parents = np.array([[-1, 0, 64, 2, -7], [9, 0, 2, 3, 1], [1 << 30, 5, 1, -(1 << 31), 4]], np.int32)
    plain = np.array([[-1, 0, -1, 2, -1], [-1, 0, -1, -1, 1], [-1, -1, 1, -1, -1]], np.int32)
    want = np.stack([R.masks_of(p) for p in plain]).view(np.int64)
    got = tree_masks(torch.from_numpy(parents))
    assert np.array_equal(got.numpy(), want)


def test_a_sequence_with_a_node_without_a_page_sits_the_step_out(monkeypatch):
    # the insert gets its slots (and reports them), every other call sees no nodes of it: its
    # length stays, where a refused path would count the nodes as cached
    s = step_of([[3, 5], [7, -1], [1, 2]], [254, 127, 200], 4, 8)
    seen = {}
    s.caches.insert_rows = lambda k, v, i, slots: seen.update(slots=slots)
    monkeypatch.setattr(speculate, "tree_paged_decode", lambda *a, **kw: seen.update(
        lens=a[4].tolist(), n_nodes=kw["n_nodes"].tolist()))
    k = torch.zeros((3, 4, 1, 128))
    s.attend(None, k, k, k[:, :, 0], n_nodes=torch.tensor([4, 2, 3], dtype=torch.int32))
    assert seen["n_nodes"] == [0, 0, 3] and seen["lens"] == [254, 127, 203]
    assert [int(x) for x in (seen["slots"].view(3, 4) >= 8 * 128).sum(1)] == [2, 1, 0]
    s.attend(None, k, k, k[:, :, 0], n_nodes=torch.tensor([2, 1, 4], dtype=torch.int32))
    assert seen["n_nodes"] == [2, 1, 4] and seen["lens"] == [256, 128, 204]
