"""Chunked prefill through the libecho C ABI: one prompt, blocks of query rows.

A PrefillRunner owns the fixed-size buffers of one prompt (the row-strided
score workspace, per-row histograms and selections, the union of a block's
selections, the GPU cache over the whole prompt) and issues one
echo_prefill_block call per block: the block's recall runs on a copy stream
while the next block is scored.  With attention=True the block's rows then
attend over their selected tokens in the cache (echo_mla_chunk), on the copy
stream after the recall.
"""
from __future__ import annotations

import math

import torch

from . import _lib as L


class PrefillRunner:
    def __init__(self, k8: torch.Tensor, ks: torch.Tensor, k: int, C: int, host_pool: torch.Tensor,
                 block_rows: int, alpha: float = 0.5, attention: bool = False, heads: int = L.MLA_HEADS,
                 mla_scale: float = 1.0 / math.sqrt(192.0), device="cuda"):
        self.n_keys = int(k8.shape[0])
        self.W = self.n_keys                      # row stride: the whole prompt
        self.R = int(block_rows)
        self.k, self.C, self.alpha = int(k), int(C), float(alpha)
        if self.C < self.W:
            raise ValueError("the prompt's cache needs C >= prompt length")
        self.k8, self.ks = k8, ks
        f32 = dict(dtype=torch.float32, device=device)
        i32 = dict(dtype=torch.int32, device=device)
        self.scores = torch.zeros((self.R, self.W), **f32)
        self.hist = torch.zeros((self.R, 256), **i32)
        self.sel_idx = torch.full((self.R, self.k), -1, **i32)
        self.kth = torch.zeros(self.R, **f32)
        self.theta = torch.full((1,), math.inf, **f32)
        self.union_list = torch.full((self.W,), -1, **i32)
        self.union_count = torch.zeros(1, **i32)
        self.union_bits = torch.zeros((self.W + 31) // 32, **i32)
        self.sel_slot = torch.full((self.W,), -1, **i32)
        self.ws = torch.zeros(L.prefill_workspace_size(self.R, self.W), dtype=torch.uint8, device=device)
        self.status = torch.zeros(1, **i32)
        self.stats = torch.zeros(L.STATS_N, **i32)
        self.cache = L.LayerCache(1, self.n_keys, self.C, host_pool, device=device)
        self.copy = torch.cuda.Stream(device=device)
        # sparse MLA attention of the block's rows over their selections: the cache's rows through tok2slot.
        # The selections have two buffers, so that the next block's top-k may run beside this block's attention
        self.attention, self.heads, self.mla_scale = bool(attention), int(heads), float(mla_scale)
        if self.attention:
            if self.cache.row_bytes != 2 * L.MLA_DQK:
                raise ValueError("attention needs 576-dim bf16 cache rows")
            self.pages = L.KVPages.of_cache(self.cache)
            self._sel = [self.sel_idx, torch.full_like(self.sel_idx, -1)]   # taken in turn
            self.tok_off = torch.tensor([0, self.n_keys], dtype=torch.int64, device=device)
            last = self.n_keys - (self.blocks() - 1) * self.R
            self._row_off = {r: torch.tensor([0, r], dtype=torch.int64, device=device) for r in (self.R, last)}
            self.attn_out = torch.zeros((self.R, self.heads, L.MLA_DV), dtype=torch.bfloat16, device=device)
            self.attn_lse = torch.zeros((self.R, self.heads), **f32)
            self.attn_ws = torch.zeros(L.mla_chunk_workspace_size(self.R, self.heads, 1), dtype=torch.uint8,
                                       device=device)

    def blocks(self):
        return (self.n_keys + self.R - 1) // self.R

    def block(self, i: int, q: torch.Tensor, w: torch.Tensor, stream=None, mla_q: torch.Tensor | None = None):
        """Enqueue block i (q [R_i,64,128], w [R_i,64] on the device).

        mla_q: with attention=True, the block's MLA queries [R_i,heads,576] bf16; attn_out and attn_lse
        (first R_i rows) receive the attention of its rows over sel_idx.  It runs on the copy stream,
        after the block's recall: mla_q has to stay as it is until wait_recall, and the results, there
        from then on, are the next call's to overwrite."""
        if self.attention != (mla_q is not None):
            raise ValueError("mla_q goes with attention=True, and only with it")
        row0 = i * self.R
        R = min(self.R, self.n_keys - row0)
        assert q.shape[0] == R and w.shape[0] == R
        if self.attention:
            self._sel.reverse()
            self.sel_idx = self._sel[0]
        L.prefill_block(R, row0, self.n_keys, q, w, self.k8, self.ks, self.k, self.theta, self.alpha,
                        self.scores, self.W, self.hist, self.sel_idx, self.kth, self.union_list,
                        self.union_count, self.union_bits, self.cache, self.sel_slot, self.ws, self.status,
                        stats=self.stats, stream=stream, copy_stream=self.copy)
        if self.attention:
            mla_q.record_stream(self.copy)
            L.mla_chunk(self._row_off[R], mla_q, self.tok_off, self.n_keys, self.pages, self.mla_scale,
                        self.attn_out[:R], self.attn_lse[:R], self.attn_ws, self.status, sel=self.sel_idx[:R],
                        stream=self.copy)
        return row0, R

    def wait_recall(self, stream=None):
        (torch.cuda.current_stream() if stream is None else stream).wait_stream(self.copy)
