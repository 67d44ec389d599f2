"""A key/value cache in pages, held in 4 bits: the public functions.

Their checks, outputs and argument marshalling are in csrc/calls.cpp (the module _calls); every computation runs in the
CUDA kernels behind include/raattn.h, which describes the layout, on torch's current stream of the pool's device.

    ra_page_pool(pages, ...)                        an empty pool
    ra_page_write(k, v, pool, table, ...)           keys and values quantised into their sequences' pages
    ra_page_read(pool, table, ...)                  what slots hold, dense
    ra_attention_decode_paged(q, pool, table, ...)  one query token per sequence
    ra_page_fork(table, length, uses, parent)       rows of the table replaced: fork, reorder, free
    ra_page_reserve(pool, table, ...)               free pages for the next tokens, shared ones copied
    ra_page_compact(pool, table, uses, out)         the pages in use moved together into another pool
    RaPagedCache                                    one layer's cache, with its table, lengths and positions
"""
from __future__ import annotations

import torch

from . import _dtype_code
from .serving import _native, ra_qk_norm_rope


def ra_page_pool(pages, num_kv_heads, head_dim, page_size=64, device="cuda"):
    """Zeroed pages for keys and values of num_kv_heads heads: uint8 [pages, num_kv_heads, 2, page_size, row],
    row = head_dim / 2 + head_dim / 16 bytes, for head_dim 64 or 128 and page_size 16, 32, 64, 128 or 256."""
    if head_dim not in (64, 128):
        raise ValueError("head_dim must be 64 or 128")
    if page_size not in (16, 32, 64, 128, 256):
        raise ValueError("page_size must be 16, 32, 64, 128 or 256")
    if min(pages, num_kv_heads) < 1:
        raise ValueError("pages and num_kv_heads must be at least 1")
    return torch.zeros(pages, num_kv_heads, 2, page_size, head_dim // 2 + head_dim // 16, dtype=torch.uint8, device=device)


def ra_page_write(k, v, pool, table, start=None, *, count=None, held=False):
    """k, v [B, num_kv_heads, N, head_dim] (any strides) quantised into the pool: token n of sequence b to slot
    start[b] + n (int32 [B]; None: n), which lies in page table[b, slot // page_size] (int32 [B, M]).

    Every 64 dimensions of a row are held as 16 equally spaced values from their minimum on: the held value is at most half a step,
    1/30 of the span between minimum and maximum, away.  count: optional int32 [B], how many of the tokens of each sequence are
    stored; slots outside the row and pages outside the pool are not.  held: return (k, v) as the cache holds them, of
    k's dtype and shape.  No autograd."""
    return _native().page_write(k, v, pool, table, start, count, held)


def ra_page_read(pool, table, length, tokens, *, start=None, dtype=torch.bfloat16):
    """(k, v), each [B, num_kv_heads, tokens, head_dim] of dtype (bfloat16 or float32): what slots start[b] ..
    start[b] + tokens - 1 (start int32 [B]; None: 0) hold.  Zeros from length[b] (int32 [B]; None: no limit) on, and
    where there is no page."""
    return _native().page_read(pool, table, length, tokens, start, _dtype_code(dtype))


def ra_attention_decode_paged(q, pool, table, length, *, scale=None):
    """ra_attention of one query token per sequence: o [B, H, head_dim] for q [B, H, head_dim] (bfloat16 or float32) over the
    first length[b] (int32 [B]) slots of its pages, as the cache holds them.

    H is a multiple of num_kv_heads; consecutive query heads share a key head.  A sequence without any key
    gives zeros; slots without a page count as keys and values of zeros.  No autograd."""
    return _native().attention_decode_paged(q, pool, table, length, scale)


def ra_page_fork(table, length, uses, parent):
    """Rows of the page table replaced, in place: row b of table (int32 [B, M]) and length[b] become what row parent[b]
    (int32 [B]) and its length were; parent[b] outside 0 .. B - 1 empties the row.  uses (int32 [pages], in how many
    places of the table a page stands) follow.  Pages are shared afterwards: ra_page_reserve comes before the next write."""
    return _native().page_fork(table, length, uses, parent)


def ra_page_reserve(pool, table, length, uses, tokens, *, count=None):
    """Pages for the next `tokens` tokens of every sequence, or count[b] of them (int32 [B]), in place: of the pages that
    slots length[b] on touch, those that are missing or have other users are replaced by free ones (lowest first, in the
    order of the sequences), and what a shared one holds of the sequence is copied.

    Returns int32 [B], how many of the tokens have room, which is what ra_page_write takes as count: fewer than asked
    where the pages run out or the row ends."""
    return _native().page_reserve(pool, table, length, uses, tokens, count)


def ra_page_compact(pool, table, uses, out):
    """The pages in use moved together: in their order to the first pages of `out`, another pool of any number of pages.
    Returns (table, uses, live): the renumbered table, the uses of out's pages, and int32 [1], how many pages are
    in use; where out has fewer, the last ones are lost and the table has -1 for them."""
    return _native().page_compact(pool, table, uses, out)


class RaPagedCache:
    """One attention layer's key/value cache in pages of 4-bit entries: `batch` sequences of up to `capacity` entries
    that take pages from one pool as they grow, and share them after fork.

    pool, table [B, M], uses [pages]: see ra_page_pool, ra_page_write, ra_page_fork; length int32 [B] (entries
    held) and position int32 [B] (position of the next token), all on the device.  pages: pages of the pool, or enough for
    every sequence's capacity.  dtype: of the keys and values that are given and read.

    A pool that is smaller than batch times the longest sequence's pages (and batch / 2 more after a fork) costs a read-back of the
    counts at every append, which a capture refuses.

    `bound` is the host's count of the entries of the longest sequence, or more.  A captured graph of append and
    attend advances length and position when it is replayed, but not `bound`: whoever replays it sees to it that there is
    room (tokens without a page are not stored, and not counted), and calls recount before append again.  compact
    changes which tensors the cache uses, so graphs of it are captured anew afterwards."""

    def __init__(self, batch, num_kv_heads, capacity, head_dim, *, page_size=64, pages=None, device="cuda",
                 dtype=torch.bfloat16):
        batch, capacity = int(batch), int(capacity)
        if min(batch, capacity) < 1:
            raise ValueError("batch and capacity must be at least 1")
        _dtype_code(dtype)
        row = -(-capacity // page_size) if page_size else 1   # a size of 0 is refused with the others
        self.pool = ra_page_pool(int(pages) if pages is not None else batch * row, int(num_kv_heads), head_dim, page_size,
                                 device=device)
        self.table = torch.full((batch, row), -1, device=device, dtype=torch.int32)
        self.uses = torch.zeros(self.pool.shape[0], device=device, dtype=torch.int32)
        self.length = torch.zeros(batch, device=device, dtype=torch.int32)
        self.position = torch.zeros_like(self.length)
        self.dtype = dtype
        self.bound = 0            # no sequence holds more entries than this
        self.shared = False       # whether pages may have several users
        self.captured = False     # whether an append is part of a graph, whose replays `bound` does not count

    @property
    def pages(self):
        return self.pool.shape[0]

    @property
    def page_size(self):
        return self.pool.shape[3]

    @property
    def capacity(self):
        return self.table.shape[1] * self.page_size

    @property
    def head_dim(self):
        return self.pool.shape[4] // 36 * 64

    @property
    def num_kv_heads(self):
        return self.pool.shape[1]

    def _wanted(self, tokens, count):
        """Pages that reserve would take, counted on the device."""
        n = self.length.new_full(self.length.shape, tokens) if count is None else count.clamp(0, tokens)
        touched = -(-(tokens - 1) // self.page_size) + 1
        at = (self.length // self.page_size).unsqueeze(1) + torch.arange(touched, device=n.device, dtype=torch.int32)
        there = (at * self.page_size < (self.length + n).unsqueeze(1)) & (n > 0).unsqueeze(1) & (at < self.table.shape[1])
        page = self.table.gather(1, at.clamp(max=self.table.shape[1] - 1).long())
        return (there & ((page < 0) | (self.uses[page.clamp(min=0).long()] > 1))).sum()

    def require_room(self, tokens, count=None):
        """Raises unless every sequence has room for `tokens` more entries, or count[b] of them, and the pool has
        the pages.  Where the host's counts leave a doubt, the device's are read back, which waits for it (not while a
        graph is captured)."""
        size = self.page_size
        # each place of the table a page of its own, and those that their sharers leave
        most = self.table.shape[0] * -(-min(self.bound + tokens, self.capacity) // size) + (self.table.shape[0] // 2 if self.shared else 0)
        if self.bound + tokens <= self.capacity and most <= self.pages:
            return
        if self.length.is_cuda and torch.cuda.is_current_stream_capturing():
            raise ValueError("whether the cache has room is not known while a graph is captured")
        held = self.length.clamp(0, self.capacity)
        after = held + (tokens if count is None else count.clamp(0, tokens))
        self.bound, longest, wanted, free = (int(n) for n in torch.stack(
            [held.max(), after.max(), self._wanted(tokens, count), (self.uses == 0).sum()]))
        if longest > self.capacity:
            raise ValueError(f"the cache holds up to {self.bound} of {self.capacity} entries: no room for {tokens} more")
        if wanted > free:
            raise ValueError(f"the pool has {free} free pages of {self.pages}: {wanted} are needed")

    def append(self, qkv, num_heads, *, count=None, held=False, **how):
        """ra_qk_norm_rope of new tokens, their keys and values quantised into this cache's next slots, which advance;
        returns q, or with held (q, k, v) with k and v as the cache holds them."""
        tokens = qkv.shape[1]
        self.require_room(tokens, count)
        with torch.no_grad():
            q, k, v = ra_qk_norm_rope(qkv, num_heads, self.num_kv_heads, **how)
        if k.shape != (self.table.shape[0], self.num_kv_heads, tokens, self.head_dim) or k.device != self.pool.device:
            raise ValueError("qkv must have the cache's batch size, head dimension and device")   # before any page is taken
        granted = ra_page_reserve(self.pool, self.table, self.length, self.uses, tokens, count=count)
        kept = ra_page_write(k, v, self.pool, self.table, self.length, count=granted, held=held)
        self.length.add_(granted)
        self.position.add_(granted)
        self.bound = min(self.bound + tokens, self.capacity)
        if self.length.is_cuda and torch.cuda.is_current_stream_capturing():
            self.captured = True
        return (q, *kept) if held else q

    def recount(self):
        """Reads the length of the longest sequence back into `bound`, and returns it."""
        self.bound = int(self.length.clamp(0, self.capacity).max())
        return self.bound

    def attend(self, q, scale=None):
        """ra_attention_decode_paged of q [B, H, head_dim] against everything this cache holds."""
        return ra_attention_decode_paged(q, self.pool, self.table, self.length, scale=scale)

    def read(self, tokens, start=None):
        """(k, v) [B, num_kv_heads, tokens, head_dim] of the cache's dtype: ra_page_read."""
        return ra_page_read(self.pool, self.table, self.length, tokens, start=start, dtype=self.dtype)

    def fork(self, parent):
        """Sequence b goes on from what sequence parent[b] (int32 [B]) holds; outside 0 .. B - 1: from nothing."""
        ra_page_fork(self.table, self.length, self.uses, parent)
        there = (parent >= 0) & (parent < parent.numel())
        self.position.copy_(torch.where(there, self.position[parent.clamp(0, parent.numel() - 1).long()], 0))
        self.shared = True

    def free(self, sequences):
        """Empties these sequences (integers) and gives their pages back; reads the lengths of the others back."""
        parent = torch.arange(self.length.numel(), dtype=torch.int32)
        parent[list(sequences)] = -1
        ra_page_fork(self.table, self.length, self.uses, parent.to(self.length.device))
        self.position.mul_((parent >= 0).to(self.position.device))
        self.recount()

    def compact(self, pages=None):
        """Moves the cache into a pool of `pages` pages (those in use when not given; their number is read back).

        The default leaves no page free: an append that crosses a page's border, or meets a page with several users, is refused until
        the cache has moved into a larger pool."""
        used = int((self.uses > 0).sum())
        pages = max(used, 1) if pages is None else int(pages)
        if pages < max(used, 1):
            raise ValueError(f"{used} pages are in use")
        out = ra_page_pool(pages, self.num_kv_heads, self.head_dim, self.page_size, device=self.pool.device)
        self.table, self.uses, _ = ra_page_compact(self.pool, self.table, self.uses, out)
        self.pool = out
