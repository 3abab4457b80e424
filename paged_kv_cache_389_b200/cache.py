"""PagedKVCache: one layer's K/V pool on the GPU plus the host block manager.

Orchestration only: the host C++ BlockManager decides slots, tables and copy
pairs; pa_copy_blocks / pa_cache_write / pa_decode / pa_prefill_chunk (for a pool
with a scale per block and kv head pa_copy_blocks_scaled / pa_cache_write_scaled /
pa_decode_scaled) and pa_prefill_packed do all the device work.  Order within a
step follows the pages' data flow (a new token is written back into the cache,
then attended to): copy-on-write copies, then the
cache write, then attention, all on one stream.
"""
from __future__ import annotations

import contextlib
import math

import numpy as np

from . import (BlockManager, pa_cache_write, pa_cache_write_scaled, pa_copy_blocks, pa_copy_blocks_scaled, pa_decode,
               pa_decode_scaled, pa_decode_scaled_workspace_size, pa_decode_workspace_size, pa_prefill_chunk,
               pa_prefill_packed, pa_prefill_packed_workspace_size, BLOCK_SIZE)


def _torch():
    import torch
    return torch


class PagedKVCache:
    def __init__(self, num_blocks: int, num_kv_heads: int, head_dim: int, dtype, device="cuda",
                 free_order=None, fill_nan: bool = True, k_scale: float = 1.0, v_scale: float = 1.0,
                 block_scales: bool = False):
        """dtype torch.float32, torch.bfloat16 or torch.float8_e4m3fn; an fp8 pool stores
        e4m3(x / k_scale) and e4m3(x / v_scale) and takes bf16 queries and K/V.  With
        block_scales, dtype torch.float8_e4m3fn or torch.int8: every (block, kv head) has
        a power-of-two scale of its own that follows the data (nothing to calibrate)."""
        torch = _torch()
        self.num_blocks, self.num_kv_heads, self.head_dim = num_blocks, num_kv_heads, head_dim
        self.dtype, self.device = dtype, torch.device(device)
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self.block_scales = bool(block_scales)
        shape = (num_blocks, num_kv_heads, BLOCK_SIZE, head_dim)
        if dtype == torch.int8 and not block_scales:
            raise ValueError("int8 pools have a scale per block and kv head: block_scales=True")
        if block_scales and dtype not in (torch.int8, torch.float8_e4m3fn):
            raise ValueError("block_scales: torch.float8_e4m3fn or torch.int8 pools")
        # NaN in every slot nothing has written: a stray read poisons the output
        if dtype == torch.float8_e4m3fn:
            code = 0x7F if fill_nan else 0x00          # e4m3 NaN / +0
            self.key_cache = torch.full(shape, code, dtype=torch.uint8, device=self.device).view(dtype)
            self.value_cache = torch.full(shape, code, dtype=torch.uint8, device=self.device).view(dtype)
        elif dtype == torch.int8:
            self.key_cache = torch.zeros(shape, dtype=dtype, device=self.device)
            self.value_cache = torch.zeros(shape, dtype=dtype, device=self.device)
        else:
            fill = float("nan") if fill_nan else 0.0
            self.key_cache = torch.full(shape, fill, dtype=dtype, device=self.device)
            self.value_cache = torch.full(shape, fill, dtype=dtype, device=self.device)
        if block_scales:
            fill = float("nan") if fill_nan else 0.0
            self.key_scales = torch.full(shape[:2], fill, dtype=torch.float32, device=self.device)
            self.value_scales = torch.full(shape[:2], fill, dtype=torch.float32, device=self.device)
        self.manager = BlockManager(num_blocks, BLOCK_SIZE, free_order)
        self.err_flag = torch.zeros(1, dtype=torch.int32, device=self.device)

    # -- allocator passthroughs ------------------------------------------------
    def add_seq(self, seq):
        self.manager.add_seq(seq)

    def fork(self, parent, child):
        self.manager.fork(parent, child)

    def free(self, seq):
        self.manager.free(seq)

    # -- step pieces -----------------------------------------------------------
    def plan_append(self, seqs, counts=None):
        """Allocate slots for ``counts[i]`` new tokens of each seq (default 1), all or
        nothing, in one call to the host manager.  Returns (int64 slots [sum counts],
        int32 copy pairs [P, 2]) as numpy arrays."""
        if self.block_scales and len(set(seqs)) != len(seqs):
            raise ValueError("block_scales: a block's tokens stand next to each other in a step, so no sequence twice")
        return self.manager.append_step(seqs, counts)

    def write(self, k, v, slots, pairs=None, stream=None):
        """Copy-on-write copies (if any), then scatter k/v [T, Hkv, d] into ``slots``."""
        torch = _torch()
        if self.block_scales:
            with self._on(stream):
                if pairs is not None and len(pairs):
                    pairs = torch.as_tensor(pairs, device=self.device)
                    pa_copy_blocks_scaled(self.key_cache, self.value_cache, self.key_scales, self.value_scales, pairs, self.err_flag)
                if len(slots):
                    self._store(k, v, torch.as_tensor(slots, device=self.device))
            return
        if pairs is not None and len(pairs):
            pairs = torch.as_tensor(pairs, device=self.device)
            pa_copy_blocks(self.key_cache, self.value_cache, pairs, self.err_flag, stream)
        if len(slots):
            self._store(k, v, torch.as_tensor(slots, device=self.device), stream)

    def _store(self, k, v, slots, stream=None):
        if self.block_scales:
            pa_cache_write_scaled(k, v, slots, self.key_cache, self.value_cache, self.key_scales, self.value_scales,
                                  self.err_flag, stream)
        else:
            pa_cache_write(k, v, slots, self.key_cache, self.value_cache, self.err_flag, stream, self.k_scale, self.v_scale)

    def append(self, seqs, k, v, counts=None, stream=None):
        slots, pairs = self.plan_append(seqs, counts)
        self.write(k, v, slots, pairs, stream)
        return slots, pairs

    def tables(self, seqs, max_blocks=None):
        """int32 block tables [S, max_blocks] (padded with -1) and lengths, on the device."""
        torch = _torch()
        if max_blocks is None:
            max_blocks = max(1, self.manager.max_seq_blocks(seqs))
        t, lens = self.manager.build_tables(seqs, max_blocks)
        return torch.from_numpy(t).to(self.device), torch.from_numpy(lens).to(self.device), int(lens.max(initial=0))

    def decode(self, q, seqs, scale, out=None, partition_size=0, max_blocks=None, stream=None,
               workspace=None):
        torch = _torch()
        if self.block_scales:    # the context is always split: partition_size says nothing here
            with self._on(stream):
                tables, lens, max_len = self.tables(seqs, max_blocks)
                out = torch.empty_like(q) if out is None else out
                if workspace is None:
                    workspace = self._scratch(pa_decode_scaled_workspace_size(q.shape[1], self.num_kv_heads, q.shape[2]))
                pa_decode_scaled(q, self.key_cache, self.value_cache, self.key_scales, self.value_scales, tables, lens,
                                 max(max_len, 1), scale, out, workspace, self.err_flag)
            return out
        tables, lens, max_len = self.tables(seqs, max_blocks)
        max_len = max(max_len, 1)
        out = torch.empty_like(q) if out is None else out
        if partition_size and workspace is None:
            ws = pa_decode_workspace_size(len(seqs), q.shape[1], q.shape[2], max_len, partition_size)
            workspace = torch.empty(max(ws, 16), dtype=torch.uint8, device=self.device)
        pa_decode(q, self.key_cache, self.value_cache, tables, lens, max_len, scale, out,
                  partition_size, workspace, self.err_flag, stream, self.k_scale, self.v_scale)
        return out

    def _on(self, stream):
        """Makes `stream` (None: leaves it alone) the current one, so that a call's tables, slots
        and scratch are made, copied and given back in its order."""
        return contextlib.nullcontext() if stream is None else _torch().cuda.stream(stream)

    def _scratch(self, nbytes):
        torch = _torch()
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=self.device)

    def prompt(self, q, k, v, seqs, counts, scale, out=None, stream=None):
        """Whole prompts of empty sequences: causal attention over each of them and their
        K/V appended to the cache.  q [T, Hq, d], k/v [T, Hkv, d] bf16, packed: counts[i] rows
        of seqs[i] after those of seqs[i - 1] (their tokens may be strided).  Returns the
        attention's output [T, Hq, d]."""
        torch = _torch()
        seqs, counts = list(seqs), [int(c) for c in counts]
        if len(set(seqs)) != len(seqs) or any(self.manager.num_tokens(s) != 0 for s in seqs):
            raise ValueError("prompt() takes different sequences without tokens; prefill() continues others")
        if len(counts) != len(seqs) or min(counts, default=0) < 0 or sum(counts) != q.shape[0]:
            raise ValueError("counts: one per sequence, adding up to the rows of q")
        if self.dtype == torch.float32:
            raise ValueError("prompt() computes in bf16: a bf16 or 8-bit pool wanted")
        with self._on(stream):
            # What the append or the attention refuse, they refuse before the manager hands out
            # blocks: the append is asked first, without tokens.
            self._store(k[:0], v[:0], torch.empty(0, dtype=torch.int64, device=self.device))
            starts = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(self.device)
            out = torch.empty(q.shape, dtype=q.dtype, device=self.device) if out is None else out
            ws = self._scratch(pa_prefill_packed_workspace_size(q.shape[0], len(counts), q.shape[1], self.num_kv_heads))
            pa_prefill_packed(q, k, v, starts, max(counts, default=0), scale, out, ws, self.err_flag)
            if not self.block_scales:
                k, v = k.contiguous(), v.contiguous()
            slots, pairs = self.plan_append(seqs, counts)
            self.write(k, v, slots, pairs)
        return out

    def prefill(self, q, seqs, chunk_lens, scale, out=None, max_blocks=None, stream=None):
        torch = _torch()
        if self.block_scales:
            raise ValueError("prefill() reads bf16 pools; prompt() fills one with a scale per block and kv head")
        tables, lens, _ = self.tables(seqs, max_blocks)
        out = torch.empty_like(q) if out is None else out
        ch = torch.as_tensor(np.asarray(chunk_lens, np.int32), device=self.device)
        pa_prefill_chunk(q, self.key_cache, self.value_cache, tables, lens, ch, scale, out,
                         self.err_flag, stream)
        return out


def default_scale(head_dim: int) -> float:
    return 1.0 / math.sqrt(head_dim)
