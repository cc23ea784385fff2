"""One speculative decode step over resident MXFP4 page caches, and the pages' book-keeping.

`SpeculativeStep` holds the buffers of a step in which every sequence checks a tree of up to
N drafted tokens (a root, the last token known to stand, and drafts under it): the nodes' rows
are inserted at the end of each sequence (mx4_insert through the shared page-128 slot mapping,
"vllm.models.minimax_m3.amd.mono.dispatch", _slots_shared), all nodes attend at once
(tree_paged_decode), and once the model has turned that into probabilities, verify_drafts
decides which nodes stand and mx4_accept_rows moves their rows together.  All on the current
stream, nothing is read back: sequence lengths stay on the device.

`PageBook` holds the references and the free stack of a pool: sequences branch (mx4_fork_pages),
grow and end (mx4_free_pages).
"""
from __future__ import annotations

import math

import torch

from . import (HEAD_DIM, PAGE_TOKENS, mx4_accept_rows, mx4_fork_pages, mx4_free_pages,
               tree_paged_decode, tree_paged_decode_workspace, verify_drafts)


def tree_masks(parents: torch.Tensor) -> torch.Tensor:
    """int64 [B, N] masks of int32 [B, N] parents (before their nodes; -1: none): bit i of
    word (s, j) set where i is j or an ancestor of j.  A parent that is not before its node is
    none (verify_drafts reports it); parents[:, 0] is not read."""
    B, N = parents.shape
    node = torch.arange(N + 1, device=parents.device)
    # column N: no node.  Each pass doubles the ancestors in a mask and how far `up` leads.
    up = torch.full((B, N + 1), N, dtype=torch.int64, device=parents.device)
    up[:, 1:N] = torch.where((parents >= 0) & (parents < node[:N]), parents, N)[:, 1:]
    masks = torch.where(node < N, torch.ones_like(node) << node.clamp_max(N - 1), 0).expand(B, -1)
    for _ in range((N - 1).bit_length()):
        masks = masks | masks.gather(1, up)
        up = up.gather(1, up)
    return masks[:, :N].contiguous()


class SpeculativeStep:
    """Buffers and calls of speculative steps of `block_table`'s sequences, N nodes each at most.

    seq_lens (int32 [B], device): tokens known to stand and cached; the root's token is not
    among them until its step has run."""

    def __init__(self, caches, block_table, seq_lens, nodes: int, heads: int = 16,
                 scale: float = 1.0 / math.sqrt(HEAD_DIM), window: int = 0, sinks: int = 0):
        dev = block_table.device
        B, self.N, self.H = block_table.shape[0], nodes, heads
        self.caches, self.block_table, self.scale = caches, block_table, scale
        self.window, self.sinks = window, sinks
        self.seq_lens = seq_lens.clone()
        self.with_nodes = torch.empty_like(self.seq_lens)
        self.n_nodes = torch.full((B,), nodes, dtype=torch.int32, device=dev)
        self.out = torch.empty((B, nodes, heads, HEAD_DIM), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((B, nodes, heads), dtype=torch.float32, device=dev)
        self.path = torch.empty((B, nodes), dtype=torch.int32, device=dev)
        self.n_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
        self.next_token = torch.empty((B,), dtype=torch.int32, device=dev)
        self.node = torch.arange(nodes, device=dev)
        need = tree_paged_decode_workspace(B, nodes, heads, caches.k_pages.shape[1])
        self.ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)

    def slots(self) -> torch.Tensor:
        """int64 [B * N] page-128 slots of this step's nodes, -1 past a sequence's n_nodes.  A node
        past the table, or where that has no page, gets a slot past the pool, which the insert
        reports (bad-slot)."""
        W = self.block_table.shape[1]
        pos = self.seq_lens[:, None].long() + self.node
        live = self.node < self.n_nodes[:, None]
        page = self.block_table.gather(1, (pos // PAGE_TOKENS).clamp(0, W - 1)).long()
        there = (pos >= 0) & (pos < W * PAGE_TOKENS) & (page >= 0)
        page = torch.where(there, page, self.caches.num_pages)
        return torch.where(live, page * PAGE_TOKENS + pos % PAGE_TOKENS, -1).flatten()

    def attend(self, q, k, v, idx_k, parents=None, n_nodes=None):
        """Insert the nodes' rows (fp32 k, v [B, N, Hkv, 128], idx_k [B, N, 128]) and attend:
        q bf16 [B, N, H, 128]; parents int32 [B, N] (None: chains); n_nodes int32 [B] (None:
        N each).  Returns out, bf16 [B, N, H, 128].  A sequence with a node that has no page
        (reported: bad-slot) sits the step out: its n_nodes become 0, its length stays."""
        if n_nodes is not None:
            self.n_nodes.copy_(n_nodes)
        else:
            self.n_nodes.fill_(self.N)
        slots = self.slots()
        lost = slots.view(-1, self.N).amax(1) >= self.caches.num_pages * PAGE_TOKENS
        self.n_nodes.masked_fill_(lost, 0)
        torch.add(self.seq_lens, self.n_nodes, out=self.with_nodes)
        self.caches.insert_rows(k.flatten(0, 1), v.flatten(0, 1), idx_k.flatten(0, 1), slots)
        tree_paged_decode(q, self.caches.k_pages, self.caches.v_pages, self.block_table,
                          self.with_nodes, self.scale, self.out, self.ws,
                          tree_mask=None if parents is None else tree_masks(parents),
                          n_nodes=self.n_nodes, window=self.window, sinks=self.sinks, lse=self.lse)
        return self.out

    def verify(self, target, draft, tokens, parents, u_accept, u_sample):
        """Which nodes stand, given the target's probabilities after each node, the draft's
        (None: drafts that were looked up), the drafted tokens and the random numbers; their
        rows move together and seq_lens grows by them.  Returns (path, n_accepted, next_token);
        next_token is the next step's root."""
        verify_drafts(target, draft, tokens, parents, u_accept, u_sample, self.path,
                      self.n_accepted, self.next_token, n_nodes=self.n_nodes)
        c = self.caches
        mx4_accept_rows(self.path, self.n_accepted, self.with_nodes, self.block_table, c.k_pages,
                        c.v_pages, c.idx_pages, self.seq_lens, n_nodes=self.n_nodes)
        if c.fp8_idx_pages is not None:
            mx4_accept_rows(self.path, self.n_accepted, self.with_nodes, self.block_table, None,
                            None, c.fp8_idx_pages, self.seq_lens, n_nodes=self.n_nodes)
        return self.path, self.n_accepted, self.next_token


class PageBook:
    """References and free stack of a pool whose table rows `tables` (int32 [n, W], -1 past a
    sequence's pages) are in use."""

    def __init__(self, num_pages: int, tables: torch.Tensor):
        dev = tables.device
        self.ref_counts = torch.zeros((num_pages,), dtype=torch.int32, device=dev)
        used = tables[tables >= 0].long()
        if used.numel() and int(used.max()) >= num_pages:
            raise ValueError(f"tables hold page {int(used.max())} of a pool of {num_pages}")
        self.ref_counts.index_add_(0, used, torch.ones_like(used, dtype=torch.int32))
        free = (self.ref_counts == 0).nonzero()[:, 0].to(torch.int32)
        self.free_list = torch.full((num_pages,), -1, dtype=torch.int32, device=dev)
        self.free_list[:free.numel()] = free
        self.free_count = torch.tensor([free.numel()], dtype=torch.int32, device=dev)

    def fork(self, rows, block_table, seq_lens, caches):
        """(tables int32 [n, W], lens int32 [n]) of children of block_table's rows."""
        if caches.fp8_idx_pages is not None:
            raise ValueError("caches with a second index pool do not fork")
        n = rows.shape[0]
        tables = torch.empty((n, block_table.shape[1]), dtype=torch.int32, device=rows.device)
        lens = torch.empty((n,), dtype=torch.int32, device=rows.device)
        mx4_fork_pages(rows, block_table, seq_lens, self.ref_counts, self.free_list,
                       self.free_count, caches.k_pages, caches.v_pages, caches.idx_pages, tables,
                       lens)
        return tables, lens

    def grow(self, tables, seq_lens, tokens):
        """Rows of `tables` that end before seq_lens + tokens get pages off the stack, row after
        row from the top.  Where the table or the stack ends an entry stays -1: a step whose
        nodes come there reports it."""
        W, P = tables.shape[1], self.free_list.shape[0]
        need = (seq_lens.long() + tokens + PAGE_TOKENS - 1) // PAGE_TOKENS
        want = (torch.arange(W, device=tables.device) < need[:, None]) & (tables < 0)
        want &= seq_lens[:, None] >= 0
        have = self.free_count.long().clamp(0, P)
        at = have - want.flatten().cumsum(0)  # place in the stack, below 0 past its end
        take = want.flatten() & (at >= 0)
        page = self.free_list.gather(0, at.clamp(0, P - 1)).long()
        ok = take & (page >= 0) & (page < P)
        tables.copy_(torch.where(ok.view_as(want), page.view_as(want), tables))
        self.ref_counts.index_add_(0, page.clamp(0, P - 1), ok.to(torch.int32))
        self.free_count.copy_(have - take.sum())

    def free(self, tables, seq_lens):
        """The pages of ended sequences' table rows go back, those ahead of seq_lens too."""
        col = torch.arange(1, tables.shape[1] + 1, dtype=torch.int32, device=tables.device)
        held = torch.where(tables >= 0, col, 0).amax(1) * PAGE_TOKENS
        # (a negative length stays, for the call to report)
        lens = torch.where(seq_lens < 0, seq_lens, torch.maximum(seq_lens, held))
        mx4_free_pages(tables, lens, self.ref_counts, self.free_list, self.free_count)
