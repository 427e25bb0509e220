"""PageTable: the pages of a paged cache, shared by the layers of a model.

The block table, a reference count per page and the sequences' lengths live on
the device; every operation runs in libuaa on the current stream and can be
captured into a graph. Build the layers on the table (`DecodeLayer(...,
page_size=..., block_table=pages.block_table, n_pages=...)`), then between steps:

    pages.fork(parents)      # beams, samples: row b continues row parents[b]; -1 ends it
    pages.reserve(q_len)     # pages of their own for the next q_len tokens
    pages.copy_layer(layer)  # the copies that this asked for, in every layer's pools
    layer.step(...)
    pages.trim(window, first_tokens)   # pages that no later token sees
    pages.compact(); pages.copy_layer(layer)   # held pages to the front of the pool

A layer's `seq_lens` is its own (a step advances it); one layer may be built on
the table's (`cache=dict(seq_lens=pages.seq_lens)`), the others follow with
`layer.seq_lens.copy_(pages.seq_lens)` after a fork.

A row that ended has length 0 and starts over with the next tokens: reserve gives it
a page like any other. One that is to stay idle takes a negative length
(`pages.seq_lens.masked_fill_(parents < 0, -1)`): it asks for no page, a step neither
appends to it nor reads it, and its output rows are zero.
"""
from __future__ import annotations

import torch

from . import binding as B


class PageTable:
    """block_table: [batch][pages_per_seq] int32 (-1: no page), used in place when it
    is on the device, int32 and contiguous. page_refs (default: counted from the
    table) and seq_lens (default: zeros) likewise."""

    def __init__(self, block_table, page_size: int, n_pages: int, page_refs=None, seq_lens=None, device="cuda"):
        if not torch.cuda.is_available():
            raise RuntimeError("PageTable needs a CUDA device; libuaa has no CPU implementation")
        dev = torch.device(device)
        self.device = dev = dev if dev.index is not None else torch.device("cuda", torch.cuda.current_device())
        to = lambda t: torch.as_tensor(t, dtype=torch.int32).to(dev).contiguous()
        self._index = dev.index
        self.block_table = to(block_table)
        if self.block_table.dim() != 2:
            raise ValueError(f"block_table has {self.block_table.dim()} dimensions, not 2")
        self.batch, self.pages_per_seq = (int(x) for x in self.block_table.shape)
        self.page_size, self.n_pages = int(page_size), int(n_pages)
        if page_refs is None:
            e = self.block_table.reshape(-1)
            if e.numel() and (int(e.max()) >= self.n_pages or int(e.min()) < -1):
                raise ValueError(f"block_table has entries outside [-1, {self.n_pages})")
            page_refs = torch.bincount(e[e >= 0].long(), minlength=self.n_pages)
        self.page_refs = to(page_refs)
        self.seq_lens = torch.zeros(self.batch, dtype=torch.int32, device=dev) if seq_lens is None else to(seq_lens)
        if self.page_refs.shape != (self.n_pages,) or self.seq_lens.shape != (self.batch,):
            raise ValueError("page_refs is not [n_pages], or seq_lens not [batch]")
        self.moves = torch.full((self.n_pages, 2), -1, dtype=torch.int32, device=dev)
        self.counts = torch.zeros(4, dtype=torch.int32, device=dev)
        nbytes = B.uaa_pages_workspace_size(self.batch, self.pages_per_seq, self.n_pages)
        if nbytes == 0:
            raise B.UaaError(B.UAA_ERR_UNSUPPORTED, B.last_error())
        self.ws_tensor = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
        self.ws = B.UaaWorkspace(self.ws_tensor.data_ptr(), nbytes)
        a = self.args = B.UaaPageArgs()
        a.batch, a.page_size, a.pages_per_seq, a.n_pages = (self.batch, self.page_size, self.pages_per_seq,
                                                           self.n_pages)
        a.block_table, a.seq_lens, a.page_refs = (B.ptr(self.block_table), B.ptr(self.seq_lens),
                                                  B.ptr(self.page_refs))
        a.moves, a.counts = B.ptr(self.moves), B.ptr(self.counts)

    def _s(self, stream):
        return B.call_stream(stream, self._index)

    def fork(self, parents, stream=None):
        """Row b becomes a copy of row parents[b] (int32 [batch] on the device; -1: it ends)."""
        if (parents.dtype is not torch.int32 or parents.shape != self.seq_lens.shape
                or parents.get_device() != self._index or not parents.is_contiguous()):
            raise ValueError("parents is not a contiguous int32 tensor [batch] on the device")
        B.uaa_pages_fork(self.args, B.ptr(parents), self.ws, self._s(stream))

    def trim(self, window: int, first_tokens: int = 0, stream=None):
        """Frees the pages behind the window and past the first tokens."""
        B.uaa_pages_trim(self.args, int(window), int(first_tokens), self.ws, self._s(stream))

    def reserve(self, q_len: int = 1, stream=None):
        """Pages of their own for every sequence's next q_len tokens; copy() must follow."""
        B.uaa_pages_reserve(self.args, int(q_len), self.ws, self._s(stream))

    def compact(self, stream=None):
        """Held pages to the front of the pool; copy() must follow."""
        B.uaa_pages_compact(self.args, self.ws, self._s(stream))

    def copy(self, *pools, stream=None):
        """The copies of the last reserve() or compact() in pools [n_pages][...] (up to eight)."""
        n, ptrs, sizes = self.n_pages, [], []
        for t in pools:
            if t.size(0) != n or not t.is_contiguous() or t.get_device() != self._index:
                raise ValueError(f"a pool is {tuple(t.shape)} on {t.device}, not a contiguous [{n}][...] tensor on "
                                 "the device")
            ptrs.append(t.data_ptr())
            sizes.append(t.nbytes // n)
        B.uaa_pages_copy(self.args, ptrs, sizes, self.ws, self._s(stream))

    def copy_layer(self, layer, stream=None):
        """copy() for a DecodeLayer's caches and their scales."""
        self.copy(*(t for t in (layer.k_cache, layer.v_cache, layer.k_scale, layer.v_scale) if t is not None),
                  stream=stream)

    def held(self) -> int:
        """Pages that are not free (waits for the device)."""
        return int((self.page_refs > 0).sum())

    def device_status(self, stream=None) -> int:
        """The page operators' flags (B.UAA_DEVFLAG_PAGE, _POOL); clears them."""
        return B.uaa_device_status(self.ws, self._s(stream))
