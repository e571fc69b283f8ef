"""Device-side state of one paged low-bit MLA cache, allocated with PyTorch.

PyTorch supplies the memory and the stream; every computation is a call into
the C ABI through ``binding``.
"""

from __future__ import annotations

from typing import Optional, Sequence

import numpy as np

from . import binding


class PagedCache:
    """Page pool, bf16 sink/recent buffers, block table and device error word."""

    def __init__(self, content_bits: int, rope_bits: int, block_table, num_pages: int,
                 device: str = "cuda", rotate: bool = False):
        import torch
        self.torch = torch
        self.layout = binding.layout(content_bits, rope_bits, rotate)
        self.page_bytes = binding.page_bytes(self.layout)
        bt = torch.as_tensor(np.asarray(block_table, dtype=np.int32))
        self.block_table = bt.to(device).contiguous()
        self.num_seqs, self.max_pages = self.block_table.shape
        self.pool = torch.zeros(num_pages, self.page_bytes, dtype=torch.uint8, device=device)
        packed = content_bits != 16
        self.sink = (torch.zeros(self.num_seqs, 4, 576, dtype=torch.bfloat16, device=device)
                     if packed else None)
        self.recent = (torch.zeros(self.num_seqs, 128, 576, dtype=torch.bfloat16, device=device)
                       if packed else None)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.device = device
        self._ws = None
        self._sms = None
        self.seq_lens = None  # the device state of assign: see empty()

    @classmethod
    def empty(cls, content_bits: int, rope_bits: int, num_seqs: int, max_pages: int, num_pages: int,
              max_tokens: int, device: str = "cuda", rotate: bool = False) -> "PagedCache":
        """A cache of ``num_seqs`` empty sequences whose pages are given out by
        ``assign``: at most ``max_pages`` a sequence, ``max_tokens`` new tokens a
        step.  Its lengths, tables and free pages live on the device."""
        cache = cls(content_bits, rope_bits, np.full((num_seqs, max_pages), -1, np.int32), num_pages,
                    device, rotate)
        torch = cache.torch
        i32 = dict(dtype=torch.int32, device=device)
        cache.seq_lens = torch.zeros(num_seqs, **i32)
        cache.free_pages = torch.arange(num_pages, **i32)
        cache.free_count = torch.full((1,), num_pages, **i32)
        cache.token_start = torch.zeros(num_seqs + 1, **i32)
        cache.seq_idx = torch.full((max_tokens,), -1, **i32)
        cache.pos = torch.full((max_tokens,), -1, **i32)
        cache.slots = torch.full((max_tokens,), -1, dtype=torch.int64, device=device)
        return cache

    def assign(self, new_lens, release=None, stream=None):
        """Pages and slots for ``new_lens[s]`` tokens of every sequence (int32,
        device), after ending the sequences with a non-zero ``release[s]``.
        Updates seq_lens, block_table, free_pages and free_count, and fills
        seq_idx, pos, slots and token_start."""
        self._needs_state("assign")
        binding.assign(new_lens, self.seq_lens, self.block_table, self.free_pages, self.free_count,
                       self.seq_idx, self.pos, self.err, slots=self.slots, token_start=self.token_start,
                       release=release, stream=stream)

    def _needs_state(self, what: str):
        if self.seq_lens is None:
            raise ValueError(f"{what} needs a cache made by PagedCache.empty")

    def append(self, kv, weight, rope, pos=None, seq_idx=None, seq_lens_after=None, eps: float = 1e-6,
               ckv_out=None, krope_out=None, stream=None):
        """Norm, rotate and pack the rows of a projection's output ([n][576]
        bf16).  Without ``pos`` they are the tokens of the last assign (n is at
        most max_tokens, the rows behind the last token are padding)."""
        if pos is None:
            self._needs_state("append without positions")
            if seq_idx is not None or seq_lens_after is not None:
                raise ValueError("append takes seq_idx and seq_lens_after with pos only")
            n = kv.shape[0]
            pos, seq_idx, seq_lens_after = self.pos, self.seq_idx, self.seq_lens
            if n != pos.shape[0]:
                pos, seq_idx = pos[:n], seq_idx[:n]
        binding.norm_rope_write(self.layout, kv, weight, rope, pos, self.block_table, self.pool, self.sink,
                                self.recent, self.err, eps=eps, seq_idx=seq_idx,
                                seq_lens_after=seq_lens_after, ckv_out=ckv_out, krope_out=krope_out,
                                stream=stream)

    def read(self, seq_idx, pos, seq_lens=None, out=None, stream=None):
        """Cached tokens as values, [n][576] (bf16 unless ``out`` is float32):
        as decode sees them in sequences of ``seq_lens``, or (None) their packed
        copies.  The rows of padding (``seq_idx < 0``) and of tokens with an error
        are zeros, or in a given ``out`` stay as they were."""
        new = out is None
        if new:
            out = binding.new_output((pos.shape[0], 576), self.torch.bfloat16, self.device, stream)
        return binding.read(self.layout, seq_idx, pos, self.block_table, self.pool, self.sink, self.recent,
                            out, self.err, seq_lens=seq_lens, clear_skipped=new, stream=stream)

    def decode_window(self, q, seq_lens, softmax_scale: float, window: int, sinks: int = 0, out=None,
                      lse=None, workspace=None, stream=None):
        """Attention of the last n tokens of every sequence (q [B][n][H][576] or
        [B][H][576]) over a sliding window and the first ``sinks`` tokens.  The
        workspace, when not given, is this call's own: captured graphs and
        calls on other streams do not share it."""
        torch = self.torch
        if out is None:
            out = binding.new_output((*q.shape[:-1], 512), torch.float32, self.device, stream)
        if workspace is None:
            n = q.shape[1] if q.dim() == 4 else 1
            if self._sms is None:  # the call plans for the cache's device, whichever is current here
                self._sms = torch.cuda.get_device_properties(self.pool.device).multi_processor_count
            _, nbytes = binding.window_plan(self.layout, self.num_seqs, q.shape[-2], n, window, sinks,
                                            self.max_pages, num_sms=self._sms)
            workspace = binding.new_output((nbytes,), torch.uint8, self.device, stream)
        return binding.decode_window(self.layout, q, self.pool, self.block_table, seq_lens, self.sink,
                                     self.recent, out, workspace, self.err, softmax_scale, window,
                                     sinks=sinks, lse=lse, stream=stream)

    def write(self, ckv, krope, pos, seq_idx=None, seq_lens_after=None, stream=None):
        binding.write(self.layout, ckv, krope, pos, self.block_table, self.pool, self.sink,
                      self.recent, self.err, seq_idx=seq_idx, seq_lens_after=seq_lens_after,
                      stream=stream)

    def workspace(self, heads: int, seq_lens_host: Sequence[int]):
        _, _, nbytes = binding.decode_plan(self.layout, heads, seq_lens_host)
        nbytes = max(int(nbytes), 16)
        if self._ws is None or self._ws.numel() < nbytes:
            self._ws = self.torch.empty(nbytes, dtype=self.torch.uint8, device=self.device)
        return self._ws

    def decode(self, q, seq_lens, seq_lens_host, softmax_scale: float, out=None, lse=None,
               workspace=None, stream=None):
        torch = self.torch
        B, H, _ = q.shape
        if out is None:
            out = torch.empty(B, H, 512, dtype=torch.float32, device=self.device)
        if workspace is None:
            workspace = self.workspace(H, seq_lens_host)
        binding.decode(self.layout, q, self.pool, self.block_table, seq_lens, seq_lens_host,
                       self.sink, self.recent, out, workspace, self.err, softmax_scale, lse=lse,
                       stream=stream)
        return out

    def write_decode(self, ckv_new, krope_new, q, seq_lens, seq_lens_host, softmax_scale: float,
                     out=None, lse=None, workspace=None, stream=None):
        """Append one token per sequence (at position seq_lens[s] - 1) and decode."""
        torch = self.torch
        B, H, _ = q.shape
        if out is None:
            out = torch.empty(B, H, 512, dtype=torch.float32, device=self.device)
        if workspace is None:
            workspace = self.workspace(H, seq_lens_host)
        binding.write_decode(self.layout, q, ckv_new, krope_new, self.pool, self.block_table,
                             seq_lens, seq_lens_host, self.sink, self.recent, out, workspace,
                             self.err, softmax_scale, lse=lse, stream=stream)
        return out

    def decode_multi(self, q, seq_lens, seq_lens_host, softmax_scale: float, out=None, lse=None,
                     workspace=None, stream=None):
        """n causal queries per sequence (q [B][n][H][576]) over the cache."""
        torch = self.torch
        B, n, H, _ = q.shape
        if out is None:
            out = torch.empty(B, n, H, 512, dtype=torch.float32, device=self.device)
        if workspace is None:
            workspace = self.workspace(n * H, seq_lens_host)
        binding.decode_multi(self.layout, q, self.pool, self.block_table, seq_lens, seq_lens_host,
                             self.sink, self.recent, out, workspace, self.err, softmax_scale,
                             lse=lse, stream=stream)
        return out

    def error(self) -> int:
        return binding.read_error(self.err)

    def clear_error(self):
        self.err.zero_()
