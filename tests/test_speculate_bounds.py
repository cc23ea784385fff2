"""Indices that the speculative step's torch code uses, on the CPU: none reaches a gather out of
range (which on a GPU ends the process), and what is bad is left for the calls to report."""
import types

import numpy as np
import pytest
import torch

import _spec_ref as R
from mxfp4_sparse_paged_gb300 import build as B_, speculate
from mxfp4_sparse_paged_gb300.speculate import PageBook, SpeculativeStep, tree_masks


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


# ------------------------------------------------------------------ PageBook

@pytest.fixture
def host_pages(monkeypatch):
    """mx4_fork_pages and mx4_free_pages by the plain implementations, on host tensors."""
    def fork(rows, bt, lens, refs, fl, fc, k, v, idx, child, child_lens):
        c, cl, r, n, _ = R.fork(rows.numpy(), bt.numpy(), lens.numpy(), refs.numpy(), fl.numpy(),
                                int(fc), [])
        for dst, src in ((child, c), (child_lens, cl), (refs, r)):
            dst.copy_(torch.from_numpy(src))
        fc.fill_(n)

    def free(tables, lens, refs, fl, fc):
        assert all((t[:(L + 127) // 128] >= 0).all() for t, L in zip(tables, lens.tolist()))
        r, f, n = R.free(tables.numpy(), lens.numpy(), refs.numpy(), fl.numpy(), int(fc))
        refs.copy_(torch.from_numpy(r))
        fl.copy_(torch.from_numpy(f))
        fc.fill_(n)

    monkeypatch.setattr(speculate, "mx4_fork_pages", fork)
    monkeypatch.setattr(speculate, "mx4_free_pages", free)
    return types.SimpleNamespace(fp8_idx_pages=None, k_pages=None, v_pages=None, idx_pages=None)


def test_ended_sequences_give_all_their_pages_back(host_pages):
    # pages ahead of a sequence's length, for its next drafts, were counted with the others
    table = torch.tensor([[3, 5, 9], [7, 1, -1], [2, -1, -1]], dtype=torch.int32)
    lens = torch.tensor([130, 128, 5], dtype=torch.int32)
    book = PageBook(12, table)
    assert int(book.free_count) == 6
    children, cl = book.fork(torch.tensor([0, 1, 1], dtype=torch.int32), table, lens, host_pages)
    assert int(book.free_count) == 5 and cl.tolist() == [130, 128, 128]
    book.free(children, cl)
    book.free(table, lens)
    assert int(book.free_count) == 12 and not book.ref_counts.any()


def test_sequences_grow_by_pages_off_the_stack(host_pages):
    # a child of a full page has no page for its next token: it takes one, in row order from the
    # top, and all pages come back in the end
    table = torch.tensor([[3, 5, -1], [7, -1, -1]], dtype=torch.int32)
    lens = torch.tensor([250, 128], dtype=torch.int32)
    book = PageBook(10, table)
    assert book.free_list.tolist() == [0, 1, 2, 4, 6, 8, 9, -1, -1, -1]
    children, cl = book.fork(torch.tensor([1, 0, 1], dtype=torch.int32), table, lens, host_pages)
    assert children.tolist() == [[7, -1, -1], [3, 9, -1], [7, -1, -1]]
    book.grow(children, cl, 6)
    assert children.tolist() == [[7, 8, -1], [3, 9, -1], [7, 6, -1]] and int(book.free_count) == 4
    book.grow(children, cl, 7)  # 250 + 7: one more for the second row alone
    assert children.tolist() == [[7, 8, -1], [3, 9, 4], [7, 6, -1]] and int(book.free_count) == 3
    assert [int(book.ref_counts[p]) for p in (7, 8, 3, 9, 4, 6, 0)] == [3, 1, 2, 1, 1, 1, 0]
    # as many as the table and the stack have: rows in order, no page twice
    book.grow(table, torch.tensor([250, 384], dtype=torch.int32), 1 << 20)
    assert table.tolist() == [[3, 5, 2], [7, 1, 0]] and int(book.free_count) == 0
    book.grow(children, cl, 200)
    assert children.tolist() == [[7, 8, -1], [3, 9, 4], [7, 6, -1]] and int(book.free_count) == 0
    book.free(children, cl)
    book.free(table, lens)
    assert int(book.free_count) == 10 and not book.ref_counts.any()


def test_growing_takes_no_page_from_a_bad_stack_or_for_a_bad_length():
    table = torch.tensor([[3, -1], [0, -1], [1, -1]], dtype=torch.int32)
    book = PageBook(6, table)
    book.free_list[book.free_count - 1] = 77
    book.grow(table, torch.tensor([128, -300, 128], dtype=torch.int32), 1)
    assert table.tolist() == [[3, -1], [0, -1], [1, 4]] and int(book.free_count) == 1
    book.free_count.fill_(-3)
    book.grow(table, torch.tensor([128, 128, 128], dtype=torch.int32), 1)
    assert table.tolist() == [[3, -1], [0, -1], [1, 4]]


def test_page_ids_outside_the_pool_are_refused():
    with pytest.raises(ValueError, match="page 6 of a pool of 6"):
        PageBook(6, torch.tensor([[3, 5], [6, -1]], dtype=torch.int32))
