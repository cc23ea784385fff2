"""A decode step over the 8-bit K/V cache: append, choice of blocks, attention.

`Fp8Caches` holds the pools: E4M3 K and V pages with a scale for every 32 tokens and head, and the
fp8 index pages that share their page ids ("vllm.models.minimax_m3.amd.mono.dispatch",
_config_refusal: fp8 K/V and index caches; _slots_shared).  `Fp8Step` holds the buffers of steps in
which every sequence brings q tokens: their K heads turn by their positions and are appended with V
(fp8_rope_append) and the index keys (fp8_index_insert); index scores choose blocks of 128 tokens
for each of them (index_block_score_fp8, block_topk), and attention reads those (fp8_block_decode),
or everything (fp8_paged_decode).  All on the current stream; lengths stay on the device, so a step
can be captured into a CUDA graph.

A sequence with a new token that has no page (past the table, or no entry of the pool there) sits a
step or an append out: its length and its K/V rows stay, its results are zeros, and mx4_check_status
reports it (bad-slot, bad-len).
"""
from __future__ import annotations

import math

import torch

from . import (FP8_PAGE_BYTES, HEAD_DIM, PAGE_TOKENS, block_topk, fp8_block_decode,
               fp8_block_decode_workspace, fp8_index_insert, fp8_paged_decode,
               fp8_paged_decode_workspace, fp8_rope_append, index_block_score_fp8)


class Fp8Caches:
    """Resident pools, poisoned (0xFF: NaN) until written."""

    def __init__(self, num_pages: int, kv_heads: int = 1, index_scale: float = 1.0, device="cuda"):
        self.num_pages, self.index_scale = num_pages, index_scale
        u8 = dict(dtype=torch.uint8, device=device)
        self.k_pages = torch.full((num_pages, kv_heads, FP8_PAGE_BYTES), 0xFF, **u8)
        self.v_pages = torch.full_like(self.k_pages, 0xFF)
        self.k_scales = torch.full((num_pages, kv_heads, 4), 0xFF, **u8)
        self.v_scales = torch.full_like(self.k_scales, 0xFF)
        self.idx_pages = torch.full((num_pages, FP8_PAGE_BYTES), 0xFF, **u8)

    def kv(self):
        return self.k_pages, self.v_pages, self.k_scales, self.v_scales


class Fp8Step:
    """Buffers and calls of decode steps of `block_table`'s sequences, q_per_seq tokens each.

    seq_lens (int32 [B], device): tokens cached so far.  blocks: how many blocks a token reads, the
    first `first` and last `last` in any case (0: all tokens, `first` and `last` unused).  phases (int64, rope_phases): how the
    heads turn, None: not at all."""

    def __init__(self, caches: Fp8Caches, block_table, seq_lens, q_per_seq: int = 1, heads: int = 16,
                 blocks: int = 16, first: int = 1, last: int = 2, phases=None, interleaved=False,
                 factor: float = 1.0, scale: float = 1.0 / math.sqrt(HEAD_DIM)):
        dev, (B, W) = block_table.device, block_table.shape
        if blocks < 0 or (blocks > 0 and (first < 0 or last < 0 or first + last > blocks)):
            raise ValueError(f"blocks = {blocks}, of which the first {first} and the last {last} in any case")
        self.caches, self.block_table, self.q, self.scale = caches, block_table, q_per_seq, scale
        self.blocks, self.first, self.last = blocks, first, last
        self.phases, self.interleaved, self.factor = phases, interleaved, factor
        self.seq_lens = seq_lens.clone()
        self.now = torch.empty_like(self.seq_lens)   # with a step's tokens, 0 where it is sat out
        self.next = torch.empty_like(self.seq_lens)  # what seq_lens is after it
        T, Hkv = B * q_per_seq, caches.k_pages.shape[1]
        self.cu_step = torch.arange(0, T + 1, q_per_seq, dtype=torch.int32, device=dev)
        t = torch.arange(T, device=dev)
        self.row_seq, self.row_back = t // q_per_seq, t % q_per_seq - q_per_seq  # of a step's rows
        self.q_out = torch.empty((T, heads, HEAD_DIM), dtype=torch.bfloat16, device=dev)
        self.out = torch.empty_like(self.q_out)
        self.lse = torch.empty((T, heads), dtype=torch.float32, device=dev)
        need = fp8_paged_decode_workspace(T, q_per_seq, heads, Hkv)
        if blocks:
            self.scores = torch.empty((T, W), dtype=torch.float32, device=dev)
            self.block_idx = torch.empty((T, blocks), dtype=torch.int32, device=dev)
            need = fp8_block_decode_workspace(T, blocks, heads, Hkv)
        self.ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)

    def slots(self, cu_new, T: int, lens=None) -> torch.Tensor:
        """int64 [T] page-128 slots of the rows that cu_new gives the sequences' last positions (of
        `lens`, None: seq_lens), -1 for rows of none.  A row past the table, or where that has no
        page, gets a slot past the pool, which the insert reports (bad-slot)."""
        lens = self.seq_lens if lens is None else lens
        B, dev = self.block_table.shape[0], self.block_table.device
        t = torch.arange(T, device=dev, dtype=cu_new.dtype)
        s = torch.searchsorted(cu_new, t, right=True).sub_(1)
        live = (s >= 0) & (s < B)
        s = s.clamp_(0, B - 1)
        return torch.where(live, self._slots(s, t - cu_new[s + 1], lens), -1)

    def _slots(self, seq, back, lens):
        """Slots of the rows of sequences `seq` at lens + back, past the pool where there is no page."""
        W = self.block_table.shape[1]
        pos = lens[seq].long() + back
        page = self.block_table[seq, (pos // PAGE_TOKENS).clamp(0, W - 1)].long()
        there = (pos >= 0) & (pos < W * PAGE_TOKENS) & (page >= 0)
        return torch.where(there, page, self.caches.num_pages) * PAGE_TOKENS + pos % PAGE_TOKENS

    def append(self, k, v, idx_k, cu_new, new, q=None, q_out=None, positions=None):
        """`new` (int32 [B]) more tokens a sequence, the rows of k, v [T, Hkv, 128] and idx_k fp32
        [T, 128] that cu_new (int32 [B + 1]) gives it; q [T, H, 128] turned into q_out.  A call
        that is refused (an exception) leaves the lengths as they were."""
        torch.add(self.seq_lens, new, out=self.now)
        T = k.shape[0]
        slots = self.slots(cu_new, T, self.now)
        # rows without a page ahead of each row; a sequence whose rows cross one, or the end, is out
        before = torch.nn.functional.pad((slots >= self.caches.num_pages * PAGE_TOKENS).cumsum(0), (1, 0))
        at = cu_new.long()
        n = before[at.clamp(0, T)]
        self._write(k, v, idx_k, cu_new, q, q_out, positions, slots, (n[1:] != n[:-1]) | (at[1:] > T))
        self.seq_lens.copy_(self.next)

    def _write(self, k, v, idx_k, cu_new, q, q_out, positions, slots, out):
        """The rows of an append to `now` but for the sequences `out`; `next` is what follows."""
        c = self.caches
        torch.where(out, self.seq_lens, self.now, out=self.next)
        self.now.masked_fill_(out, 0)
        # (index rows first: they can be written again, a block's scale does not go back)
        fp8_index_insert(idx_k, slots, c.index_scale, c.idx_pages)
        fp8_rope_append(q, k, v, cu_new, self.block_table, self.now, *c.kv(), q_out,
                        phases=self.phases, positions=positions, interleaved=self.interleaved,
                        factor=self.factor)

    def run(self, q, k, v, iq, idx_k, positions=None):
        """One step: q [T, H, 128], k, v [T, Hkv, 128] (fp32 or bf16, before the turn), iq bf16 and
        idx_k fp32 [T, 128].  Returns out, bf16 [T, H, 128].  A step that is refused (an exception)
        leaves the lengths as they were: it can be run again."""
        c, cached = self.caches, (self.block_table, self.now)
        torch.add(self.seq_lens, self.q, out=self.now)
        slots = self._slots(self.row_seq, self.row_back, self.now)
        lost = (slots >= c.num_pages * PAGE_TOKENS).view(-1, self.q).any(1)
        self._write(k, v, idx_k, self.cu_step, q, self.q_out, positions, slots, lost)
        if not self.blocks:
            fp8_paged_decode(self.q_out, self.q, *c.kv(), *cached, self.scale, self.out, self.ws,
                             lse=self.lse)
        else:
            index_block_score_fp8(iq, self.q, c.idx_pages, *cached, c.index_scale, self.scores)
            block_topk(self.scores, self.now, self.q, self.block_idx, first=self.first,
                       last=self.last)
            fp8_block_decode(self.q_out, self.q, *c.kv(), *cached, self.block_idx, self.scale,
                             self.out, self.ws, lse=self.lse)
        self.seq_lens.copy_(self.next)
        return self.out
