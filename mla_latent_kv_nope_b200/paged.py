"""A paged latent cache and its bookkeeping on the device.

``PagedCache`` owns what a server keeps per layer stack of a paged cache: the
pool of pages (bf16 or fp32 rows, or 8-bit rows with one scale per page), the
free list, the block tables and the lengths.  A serving step is

    cache.plan(new_lens)                   # pages, positions and slots of the new tokens
    cache.write(x)                         # their latent rows, x = W^DKV h for all of them
    out = step(q_nope, q_pe, cache.last_positions(), cache.pool, cache.seqlens,
               block_table=cache.block_table, page_scales=cache.page_scales)

and ``cache.release(mask)`` ends requests.  Everything stays on the device and
in buffers that never move, so a step can be captured into a CUDA graph and
replayed with other contents of ``new_lens`` and ``x``.  The operators are the
library's kernels; this class keeps buffers and their order.
"""
from __future__ import annotations

import torch

from . import binding as b


class PagedCache:
    """dims: B requests at most, cache_capacity tokens of each; num_pages pages of 64
    rows; max_tokens new tokens in one step.  ``fp8`` holds 8-bit rows.  ``table`` (see
    rope_table) rotates the rotary keys; None stores them as they come."""

    def __init__(self, dims: b.Dims, num_pages: int, max_tokens: int, fp8=False, gamma=None,
                 table=None, eps=1e-6, device="cuda"):
        self.dims, self.num_pages, self.gamma, self.table, self.eps = dims, num_pages, gamma, table, eps
        B, blocks = dims.B, (dims.cache_capacity + b.PAGE_ROWS - 1) // b.PAGE_ROWS
        i32 = dict(dtype=torch.int32, device=device)
        if fp8:
            self.pool = torch.zeros(num_pages, b.PAGE_ROWS, dims.d_c + 2 * dims.d_r,
                                    dtype=torch.uint8, device=device)
            self.page_scales = torch.ones(num_pages, dtype=torch.float32, device=device)
        else:
            self.pool = torch.zeros(num_pages, b.PAGE_ROWS, dims.R, dtype=dims.torch_dtype,
                                    device=device)
            self.page_scales = None
        self.block_table = torch.full((B, blocks), -1, **i32)
        self.seqlens = torch.zeros(B, **i32)
        self.free_pages = torch.arange(num_pages - 1, -1, -1, **i32)   # page 0 is taken first
        self.free_count = torch.full((1,), num_pages, **i32)
        self.query_start = torch.zeros(B + 1, **i32)
        self._step_tokens = self.query_start[B:]     # [1]: the planned step's tokens
        self.positions = torch.full((max_tokens,), -1, **i32)
        self.slots = torch.full((max_tokens,), -1, dtype=torch.int64, device=device)
        self.token_request = torch.full((max_tokens,), -1, **i32)
        self._open = False       # a step is planned
        self._planned = None     # rows that its write must have, if they were stated
        self._last = torch.zeros(B, **i32)
        self._ws = torch.zeros(b.plan_pages_workspace_bytes(), dtype=torch.uint8, device=device)

    def plan(self, new_lens, tokens=None) -> None:
        """plan_pages in place: request r gets new_lens[r] more tokens (int32 [B]), at most
        ``tokens`` in all (max_tokens if None): the rows that write() will be given.  A
        step of more is not begun and records MLA_ERR_BOUNDS."""
        self._open = False       # until the plan is made
        T = self.positions.shape[0] if tokens is None else tokens
        if not 0 <= T <= self.positions.shape[0]:
            raise ValueError(f"tokens must be in [0, {self.positions.shape[0]}], got {T}")
        b.plan_pages(self.seqlens, new_lens, self.block_table, self.free_pages, self.free_count,
                     self.num_pages, self.query_start, self.positions[:T], self.slots[:T],
                     self.seqlens, self.free_count, self._ws, token_request=self.token_request[:T],
                     capacity=self.dims.cache_capacity)
        self._open, self._planned = True, tokens

    def write(self, x) -> None:
        """The planned tokens' rows: x [T, d_c + d_r], requests in order; T = plan's
        ``tokens``.  Without it T is at least 1 and not less than the step's tokens, which
        only the device knows: fewer rows record MLA_ERR_BOUNDS.  Rows behind the last
        token are not stored."""
        if not self._open:
            raise ValueError("no step is planned")
        if self._planned is not None and x.shape[0] != self._planned:
            raise ValueError(f"x has {x.shape[0]} rows, the step was planned for {self._planned}")
        if self._planned is None and x.shape[0] == 0:
            raise ValueError("no rows: plan an empty step with tokens=0")
        if self.page_scales is not None:
            b.cache_write_fp8_paged(self.dims, x, self.gamma, self.query_start, self.seqlens,
                                    self.block_table, self.pool, self.page_scales, self.table,
                                    self.eps)
        else:
            T = x.shape[0]
            b.cache_write_paged(self.dims, x, self.gamma, self.positions[:T], self.slots[:T],
                                self.pool, self.table, self.eps, None,
                                self._step_tokens if self._planned is None else None)

    def last_positions(self):
        """Position of each request's last token (-1 without one): the query's in a decode step."""
        return torch.sub(self.seqlens, 1, out=self._last)

    def release(self, mask) -> None:
        """Return the pages of the requests with mask[r] != 0 (int32 [B])."""
        b.release_pages(self.seqlens, mask, self.block_table, self.free_pages, self.free_count,
                        self.num_pages)
