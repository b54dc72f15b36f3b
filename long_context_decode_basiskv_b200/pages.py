"""The pool of physical pages behind a batch's block table, kept on the device.

``PagePool`` owns the free list and steps a batch's lengths and block table in
place with the library's page calls, so that a decode step captured in a CUDA
graph allocates its own pages: ``extend`` before the append of new tokens,
``release`` when requests end.  A released request holds no token, and
basiskv_append takes a length below its new tokens for a fault: it leaves the
batch, or gets tokens from ``extend``, before the next append.

The pool's tensors are made on the current stream.  ``extend`` and ``release``
run on ``stream`` (default: the current one); a caller that gives one orders it
behind the pool's making, and keeps ``add_len`` or ``release`` from being
written over or freed before the call has run.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import binding as bk


class PagePool:
    def __init__(self, cfg: bk.Config, num_phys_pages: int, batch: int, max_pages: int, device="cuda"):
        self.cfg = cfg
        dev = torch.device(device)
        # popped from the back: pages 0, 1, 2 ... in this order
        self.free_pages = torch.arange(num_phys_pages - 1, -1, -1, dtype=torch.int32, device=dev)
        self.free_count = torch.full((1,), num_phys_pages, dtype=torch.int32, device=dev)
        self.block_table = torch.full((batch, max_pages), -1, dtype=torch.int32, device=dev)
        self.seq_len = torch.zeros(batch, dtype=torch.int32, device=dev)

    def extend(self, add_len: torch.Tensor, err: torch.Tensor, slots: Optional[torch.Tensor] = None, stream=None):
        """Room for add_len[b] more tokens of every request; seq_len counts them afterwards."""
        bk.assign_pages(self.cfg, self.block_table, self.seq_len, add_len, self.free_pages, self.free_count,
                        self.seq_len, self.free_count, slots, err, stream)

    def release(self, release: torch.Tensor, err: torch.Tensor, stream=None):
        """The pages of every request with release[b] != 0 back to the pool; its length is 0 then."""
        bk.release_pages(self.cfg, self.block_table, self.seq_len, release, self.free_pages, self.free_count,
                         self.seq_len, self.free_count, err, stream)
