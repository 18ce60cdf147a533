"""Python front end of decoding with trees of drafts: the tree, pages shared among sequences, and
tokens from logits (include/engram_attention.h).

Argument marshalling only, as in attention.py: every step runs in the library's CUDA kernels on the
current stream.  A step with trees of drafts:

    pairs, missing = pool.reserve(fed, fed + n)          # pages for the new tokens; copy on write
    if int(missing): ...                                 # nothing has changed: free pages, or extend fewer rows
    cache.copy_pages(pairs)                              # in every layer's cache
    tree = DraftTree(plan, batch, parent, max_nodes=64)
    q, k = plan.qk_norm_rope(q, k, tree.positions, rope) # in every layer
    cache.append(batch, k, v)
    out, lse = cache.attend_tree(tree, q)
    sampled = sample_tokens(logits, u, top_p=0.9)        # after every new token
    path, count, emitted, fed = tree.accept(tokens, sampled)
    cache.compact(batch, path, count)                    # in every layer's cache

Appending after a reserve whose ``missing`` is not 0 would write into pages that other rows share.
"""
from __future__ import annotations

import struct
from typing import Dict, Optional, Tuple, Union

import torch

from . import _lib
from . import attention as _a
from .attention import _INT_MAX, AttentionPlan, SequenceBatch, _off_device, _ptr

_MAX_WORDS = 8              # of a row of a tree's mask (32 tokens each)
_MAX_ROWS = 65536           # of a table that reserve extends, and that a call of free or fork names

_pack_tree = struct.Struct("@PPii").pack
_pack_pool = struct.Struct("@PPiiq").pack
_pack_settings = struct.Struct("@PPPPfiff").pack

_F32, _I32 = torch.float32, torch.int32


def _output(t: Optional[torch.Tensor], name: str, shape: tuple, like: torch.Tensor) -> Tuple[torch.Tensor, int]:
    """An int32 output and its address: the caller's, checked, or a new one beside `like`."""
    if t is None:
        t = torch.empty(shape, dtype=_I32, device=like.device)
        return t, t.data_ptr()
    return t, _ptr(t, name, _I32, shape, like.get_device())


def _rows_of(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dim() != 1:
        raise ValueError(f"{name}: expected int32 [n]")
    if t.shape[0] > _MAX_ROWS:
        raise ValueError(f"{name}: {t.shape[0]} rows, at most {_MAX_ROWS} a call")
    return t.shape[0]


def _plan_handle(plan: AttentionPlan):
    if not plan._h:
        raise ValueError("plan: it is closed")
    return plan._h


class DraftTree:
    """The new tokens of a batch as trees (engram_tree_build, on the current stream): ``parent`` int32
    [tokens] names the new token of its sequence that each follows, -1 the cached text.  A token's
    parent comes before it.

    ``max_nodes``: the most new tokens of a sequence, at most 256.  ``window`` as in ``attend``.
    ``positions`` int32 [tokens] then holds each token's place in the text (for the rotation), ``mask``
    int32 [tokens, words] the new tokens that it sees, bit by bit.  They are allocated unless given.
    Rows of no sequence (past ``start[B]``) are not written: give zeroed ``positions`` where a batch is
    padded with such rows and its queries are rotated."""

    def __init__(self, plan: AttentionPlan, batch: SequenceBatch, parent: torch.Tensor, *, max_nodes: int = 64,
                 window: int = 0, mask: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None):
        if not isinstance(parent, torch.Tensor) or parent.dim() != 1:
            raise ValueError("parent: expected int32 [tokens]")
        words = (int(max_nodes) + 31) // 32
        if not 1 <= words <= _MAX_WORDS:
            raise ValueError(f"max_nodes: {max_nodes}, expected 1 to {32 * _MAX_WORDS}")
        if window < 0:
            raise ValueError("window: must not be negative")
        h, dev, T = _plan_handle(plan), plan.device, parent.shape[0]
        parent_ptr = _ptr(parent, "parent", _I32, (T,), dev)
        mask, mask_ptr = _output(mask, "mask", (T, words), parent)
        positions, at_ptr = _output(positions, "positions", (T,), parent)
        self.plan, self.batch, self.parent, self.mask, self.positions = plan, batch, parent, mask, positions
        self.tokens, self.window = T, min(int(window), _INT_MAX)
        self._packed = _pack_tree(mask_ptr, at_ptr, words, self.window)
        _lib.check(plan._lib.engram_tree_build(h, batch._struct(T, dev), parent_ptr, self._packed,
                                               _a._current_stream(dev)), "engram_tree_build")

    def _struct(self, device: int) -> bytes:
        if self.plan.device != device:
            raise _off_device(self.mask, "tree", device)
        return self._packed

    def accept(self, tokens: torch.Tensor, sampled: torch.Tensor, *, width: int = 16,
               path: Optional[torch.Tensor] = None, count: Optional[torch.Tensor] = None,
               emitted: Optional[torch.Tensor] = None, length: Optional[torch.Tensor] = None
               ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
        """The path that the sampled tokens take (engram_tree_accept): from new token 0, to the child
        whose token was drawn, at most ``width`` tokens.  ``tokens`` and ``sampled`` int32 [tokens]: the
        new tokens, and what was drawn after each.  Returns int32 (path [B, width], count [B], emitted
        [B, width]: what was drawn after each of the path, length [B]: tokens in the cache once
        ``compact`` has moved the path together)."""
        plan, T, B = self.plan, self.tokens, self.batch.B
        h, dev, width = _plan_handle(plan), plan.device, int(width)
        if not 1 <= width <= 32 * _MAX_WORDS:
            raise ValueError(f"width: {width}, expected 1 to {32 * _MAX_WORDS}")
        parent = self.parent
        path, path_ptr = _output(path, "path", (B, width), parent)
        count, count_ptr = _output(count, "count", (B,), parent)
        emitted, emitted_ptr = _output(emitted, "emitted", (B, width), parent)
        length, length_ptr = _output(length, "length", (B,), parent)
        _lib.check(plan._lib.engram_tree_accept(
            h, self.batch._struct(T, dev), parent.data_ptr(), _ptr(tokens, "tokens", _I32, (T,), dev),
            _ptr(sampled, "sampled", _I32, (T,), dev), width, path_ptr, count_ptr, emitted_ptr, length_ptr,
            _a._current_stream(dev)), "engram_tree_accept")
        return path, count, emitted, length


class PagePool:
    """Pages shared among the rows of a page table: ``table`` int32 [rows, table_pages] (below 0: no
    page) and ``ref`` int32 [pages], how many entries name each page; both are the caller's and updated
    in place.  The table's rows serve SequenceBatch, one table all layers' caches.  ``reserve`` takes
    tables of up to 65536 rows, ``free`` and ``fork`` up to 65536 rows a call.  Calls on one pool
    run one after another, whatever their streams: they update the same two tensors, which like the
    plan have to outlive what is queued or captured on them (the pool itself may go)."""

    def __init__(self, plan: AttentionPlan, table: torch.Tensor, ref: torch.Tensor):
        if not isinstance(table, torch.Tensor) or table.dim() != 2:
            raise ValueError("table: expected int32 [rows, table_pages]")
        if not isinstance(ref, torch.Tensor) or ref.dim() != 1:
            raise ValueError("ref: expected int32 [pages]")
        dev = plan.device
        if table.shape[0] > _INT_MAX or table.shape[1] > _INT_MAX:
            raise ValueError("table: more rows or pages than 31 bits count")
        self.plan, self.table, self.ref = plan, table, ref
        self._packed = _pack_pool(_ptr(table, "table", _I32, table.shape, dev), _ptr(ref, "ref", _I32, ref.shape, dev),
                                  table.shape[0], table.shape[1], ref.shape[0])
        n = _lib.ctypes.c_size_t()
        _lib.check(plan._lib.engram_pool_workspace_bytes(self._packed, _lib.ctypes.byref(n)),
                   "engram_pool_workspace_bytes")
        self.workspace_bytes = n.value

    @classmethod
    def empty(cls, plan: AttentionPlan, rows: int, table_pages: int, pages: int) -> "PagePool":
        """A pool of `pages` unused pages and `rows` rows without pages."""
        device = torch.device("cuda", plan.device)
        return cls(plan, torch.full((rows, table_pages), -1, dtype=_I32, device=device),
                   torch.zeros(pages, dtype=_I32, device=device))

    _workspaces: Optional[Dict[int, torch.Tensor]] = None      # of each stream, from its first call on

    def _workspace_on(self, stream: int) -> torch.Tensor:
        """Memory for a call on a stream, which is the current one: allocated there, so that once the
        pool is gone it is used again only behind what is queued.  A call under capture gets memory of its
        graph, which stays that graph's.  (Allocated with each call it took 2 to 4 us of the host's time.)"""
        kept = self._workspaces
        if kept is None:
            kept = self._workspaces = {}
        captured = _a._capturing()
        ws = None if captured else kept.get(stream)
        if ws is None:
            ws = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=self.table.device)
            if not captured:
                kept[stream] = ws
        return ws

    def free(self, rows: torch.Tensor, keep: torch.Tensor) -> None:
        """Rows int32 [n] keep the pages of their first ``keep`` int32 [n] tokens (engram_pool_free)."""
        dev, n = self.plan.device, _rows_of(rows, "rows")
        _lib.check(self.plan._lib.engram_pool_free(
            _plan_handle(self.plan), self._packed, _ptr(rows, "rows", _I32, (n,), dev), _ptr(keep, "keep", _I32, (n,), dev), n,
            _a._current_stream(dev)), "engram_pool_free")

    def fork(self, src: torch.Tensor, dst: torch.Tensor, length: torch.Tensor) -> None:
        """Rows ``dst`` int32 [n], which have no pages, share those of the first ``length`` int32 [n]
        tokens of rows ``src`` int32 [n] (engram_pool_fork)."""
        dev, n = self.plan.device, _rows_of(src, "src")
        _lib.check(self.plan._lib.engram_pool_fork(
            _plan_handle(self.plan), self._packed, _ptr(src, "src", _I32, (n,), dev), _ptr(dst, "dst", _I32, (n,), dev),
            _ptr(length, "length", _I32, (n,), dev), n, _a._current_stream(dev)), "engram_pool_fork")

    def reserve(self, before: torch.Tensor, after: torch.Tensor, *, pairs: Optional[torch.Tensor] = None,
                missing: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Pages for tokens ``before[r]`` .. ``after[r]`` - 1 of every row r (int32 [rows]) that are each
        that row's alone (engram_pool_reserve).  Returns (pairs int32 [rows, 2] for
        ``PagedCache.copy_pages``, missing int32 [1]: pages that were too few; then nothing changed, and
        the tokens must not be appended: rows may still share the pages that they would be written to)."""
        dev, n = self.plan.device, self.table.shape[0]
        if n > _MAX_ROWS:
            raise ValueError(f"table: {n} rows, reserve extends tables of at most {_MAX_ROWS}")
        pairs, pairs_ptr = _output(pairs, "pairs", (n, 2), self.table)
        missing, missing_ptr = _output(missing, "missing", (1,), self.table)
        stream = _a._current_stream(dev)
        workspace = self._workspace_on(stream)
        _lib.check(self.plan._lib.engram_pool_reserve(
            _plan_handle(self.plan), self._packed, _ptr(before, "before", _I32, (n,), dev), _ptr(after, "after", _I32, (n,), dev),
            pairs_ptr, missing_ptr, workspace.data_ptr(), self.workspace_bytes, stream), "engram_pool_reserve")
        return pairs, missing


def sample_tokens(logits: torch.Tensor, u: torch.Tensor, *, temperature: Union[float, torch.Tensor] = 1.0,
                  top_k: Union[int, torch.Tensor] = 0, top_p: Union[float, torch.Tensor] = 1.0,
                  min_p: Union[float, torch.Tensor] = 0.0, tokens: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of each row of logits [R, V] (float32 or bfloat16; rows may be apart, their elements
    not), drawn with the random numbers u float32 [R] (engram_sample_tokens).  Each setting is a number
    for all rows or a tensor [R] (top_k int32, the others float32): ``temperature`` (0: greedy),
    ``top_k`` (0: off), ``top_p`` (1: off), ``min_p`` (0: off).  Returns int32 [R]."""
    if not isinstance(logits, torch.Tensor) or logits.dtype not in (_F32, torch.bfloat16) or logits.dim() != 2:
        raise ValueError("logits: expected float32 or bfloat16 [R, V]")
    if not isinstance(u, torch.Tensor):
        raise TypeError("u: expected a torch.Tensor")
    if _a._grad_mode() and (logits.requires_grad or u.requires_grad):
        _a._forward_only(logits=logits, u=u)
    R, V = logits.shape
    dev = logits.get_device()
    if dev < 0:
        raise ValueError("logits: must be a CUDA tensor")
    if dev != _a._current_device():                   # which the launch goes to
        raise _off_device(logits, "logits", _a._current_device())
    s0, s1 = logits.stride()
    if s1 != 1 and V > 1 and R:
        raise ValueError("logits: the last dimension must be dense")
    if s0 < V:
        if R > 1:
            raise ValueError("logits: rows must not overlap")
        s0 = V
    ptrs, values = [], []
    for name, x, dtype in (("temperature", temperature, _F32), ("top_k", top_k, _I32), ("top_p", top_p, _F32),
                           ("min_p", min_p, _F32)):
        if isinstance(x, torch.Tensor):
            if x.requires_grad and _a._grad_mode():
                _a._forward_only(**{name: x})
            ptrs.append(_ptr(x, name, dtype, (R,), dev))
            values.append(0)
        else:
            ptrs.append(0)
            try:
                values.append(min(max(int(x), -1), _INT_MAX) if dtype is _I32 else float(x))
            except (TypeError, ValueError, OverflowError):
                raise ValueError(f"{name}: {x!r}, expected a number or a tensor of one for each row") from None
    tokens, tokens_ptr = _output(tokens, "tokens", (R,), logits)
    _lib.check(_lib._lib().engram_sample_tokens(
        logits.data_ptr(), _lib.F32 if logits.dtype is _F32 else _lib.BF16, s0, _ptr(u, "u", _F32, (R,), dev),
        _pack_settings(*ptrs, *values), R, V, tokens_ptr, _a._current_stream(dev)),
        "engram_sample_tokens")
    return tokens
