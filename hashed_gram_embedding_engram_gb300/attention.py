"""Python front end of the attention sub-block's C ABI (include/engram_attention.h).

Argument marshalling only, as in engram.py: every step runs in the library's
CUDA kernels on the current stream, tensors are passed by pointer.  Outputs are
allocated unless given.  The operators are forward only: in grad mode an input
that requires a gradient is refused.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional, Tuple

import torch

from . import _lib
from .engram import _ACT_DTYPES, _dev, _stream

_ROPE_STYLES = {"halves": 0, "adjacent": 1}
_COUNTER_BYTES = 16384      # of a workspace, zero when it is new (engram_attn_workspace_bytes)

_INT_MAX = 2 ** 31 - 1      # ctypes cuts larger whole numbers to their low 32 bits

# engram_heads_view_t and engram_sequences_t as bytes of the call's own: a step's calls take a few
# microseconds on the device, so the front end must not take longer (a ctypes structure costs three times this)
_pack_view = struct.Struct("@Pqq").pack
_pack_sequences = struct.Struct("@PPPiiqi4x").pack
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)
_grad_mode = torch.is_grad_enabled
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _current_stream(device: int) -> int:
    if _raw_stream is not None:
        return _raw_stream(device)
    return torch.cuda.current_stream(device).cuda_stream


def _off_device(t: torch.Tensor, name: str, device: int) -> ValueError:
    where = f"cuda:{t.get_device()}" if t.is_cuda else str(t.device)
    return ValueError(f"{name}: must be a CUDA tensor on cuda:{device}, is on {where}")


def _ptr(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device: int) -> int:
    """_dev with its checks in one test where all hold, on the device that the call runs on."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:      # no tensor
        pass
    _dev(t, name, dtype, shape)
    raise _off_device(t, name, device)


def _forward_only(**tensors: Optional[torch.Tensor]) -> None:
    """In grad mode: the operators record nothing for a backward pass, so an input that asks for a
    gradient would silently get none.  (The calls look first by themselves: a loop costs a microsecond.)"""
    for name, t in tensors.items():
        if t is not None and t.requires_grad:
            raise ValueError(f"{name}: requires a gradient, which this operator does not compute; "
                             "detach it, or call under torch.no_grad()")


def _view(t: torch.Tensor, name: str, dtype: torch.dtype, heads: int, head_dim: int, device: int,
          tokens: Optional[int] = None) -> bytes:
    """A [tokens, heads, head_dim] device tensor whose last dimension is dense."""
    try:
        at, shape = t.get_device(), t.shape
    except AttributeError:
        raise TypeError(f"{name}: expected a torch.Tensor") from None
    if at != device:
        raise _off_device(t, name, device)
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if len(shape) != 3 or shape[1] != heads or shape[2] != head_dim or (tokens is not None and shape[0] != tokens):
        raise ValueError(f"{name}: shape {tuple(shape)}, expected "
                         f"({'tokens' if tokens is None else tokens}, {heads}, {head_dim})")
    s0, s1, s2 = t.stride()
    if s2 != 1 and shape[0]:
        raise ValueError(f"{name}: the last dimension must be dense")
    # the stride of a dimension of one element is never used and may be anything
    return _pack_view(t.data_ptr(), s0 if shape[0] > 1 else 0, s1 if heads > 1 else 0)


def _norm_weight(g: Optional[torch.Tensor], name: str, head_dim: int, device: int) -> int:
    return 0 if g is None else _ptr(g, name, torch.float32, (head_dim,), device)


class AttentionPlan:
    """A validated attention shape bound to the current CUDA device: its calls are made with that
    device current, on its tensors.

    ``rotary_dim`` elements of each head are rotated (default: all); ``rope_style``
    pairs element i with i + rotary_dim/2 ("halves") or 2i with 2i+1 ("adjacent").
    ``scale`` multiplies q.k (default 1/sqrt(head_dim))."""

    def __init__(self, *, heads: int, heads_kv: int, head_dim: int, page: int = 64, dtype: str = "bf16",
                 rotary_dim: Optional[int] = None, rope_style: str = "halves", eps: float = 1e-6,
                 scale: Optional[float] = None):
        if rope_style not in _ROPE_STYLES:
            raise ValueError(f"rope_style: {rope_style!r}, expected one of {sorted(_ROPE_STYLES)}")
        if dtype not in _ACT_DTYPES:
            raise ValueError(f"dtype: {dtype!r}, expected one of {sorted(_ACT_DTYPES)}")
        if scale is not None and not ctypes.c_float(scale).value > 0:     # 0 would mean the default
            raise ValueError("scale: must be positive as a float32")
        self.heads, self.heads_kv, self.head_dim, self.page = heads, heads_kv, head_dim, page
        self.dtype, self.rope_style, self.eps, self.scale = dtype, rope_style, eps, scale
        self.rotary_dim = head_dim if rotary_dim is None else rotary_dim
        self.torch_dtype = _ACT_DTYPES[dtype][1]
        cfg = _lib.AttnConfig(heads, heads_kv, head_dim, page, _ACT_DTYPES[dtype][0], self.rotary_dim,
                              _ROPE_STYLES[rope_style], eps, 0.0 if scale is None else scale)
        self._lib = _lib._lib()
        self._h = ctypes.c_void_p()
        self._workspaces = {}
        self.device = torch.cuda.current_device()   # also makes sure a context exists
        _lib.check(self._lib.engram_attn_plan_create(ctypes.byref(cfg), ctypes.byref(self._h)),
                   "engram_attn_plan_create")
        n = ctypes.c_size_t()
        _lib.check(self._lib.engram_attn_workspace_bytes(self._h, ctypes.byref(n)), "engram_attn_workspace_bytes")
        self.workspace_bytes = n.value

    def new_workspace(self, device=None) -> torch.Tensor:
        """A workspace for attention calls; calls that may run at the same time need one each."""
        device = torch.device("cuda", self.device) if device is None else device
        ws = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device)
        ws[:_COUNTER_BYTES].zero_()
        return ws

    def _workspace(self, stream: int) -> torch.Tensor:
        """The plan's own workspace of a stream (calls on one stream run one after another).  A call
        under capture gets one of its own, in the graph's memory and zeroed by every replay: replays
        may run beside the stream's calls, and nothing of the capture has run yet when they do."""
        if _capturing():
            return self.new_workspace()
        ws = self._workspaces.get(stream)
        if ws is None:
            ws = self._workspaces[stream] = self.new_workspace()
        return ws

    def close(self) -> None:
        if getattr(self, "_h", None) and self._h.value:
            self._lib.engram_attn_plan_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def get_error(self) -> Tuple[int, int]:
        """(status, error bits) after synchronising the current stream; clears the bits."""
        flags = ctypes.c_uint32()
        st = self._lib.engram_attn_get_error(self._h, _stream(), ctypes.byref(flags))
        return st, flags.value

    def rope_table(self, length: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
        """float32 [length, rotary_dim]: cosines, then sines, of position / theta^(2i/rotary_dim)."""
        r = self.rotary_dim
        inv = float(theta) ** (-torch.arange(0, r, 2, dtype=torch.float64, device=device) / r)
        angle = torch.arange(length, dtype=torch.float64, device=device)[:, None] * inv
        return torch.cat((angle.cos(), angle.sin()), 1).float().contiguous()

    def _rope(self, rope: Optional[torch.Tensor]) -> Tuple[int, int]:
        if rope is None:
            return 0, 0
        if not isinstance(rope, torch.Tensor) or rope.dim() != 2 or rope.shape[1] != self.rotary_dim:
            raise ValueError(f"rope: expected a tensor of shape (length, {self.rotary_dim})")
        return _ptr(rope, "rope", torch.float32, rope.shape, self.device), rope.shape[0]

    def qk_norm_rope(self, q: torch.Tensor, k: Optional[torch.Tensor] = None,
                     positions: Optional[torch.Tensor] = None, rope: Optional[torch.Tensor] = None, *,
                     g_q: Optional[torch.Tensor] = None, g_k: Optional[torch.Tensor] = None,
                     q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None
                     ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """Per-head norm (where a weight is given) and rotation of q [T, heads, D] and k
        [T, heads_kv, D] in one launch (engram_qk_norm_rope): dense outputs (q, k)."""
        if _grad_mode() and (q.requires_grad or k is not None and k.requires_grad
                             or rope is not None and rope.requires_grad or g_q is not None and g_q.requires_grad
                             or g_k is not None and g_k.requires_grad):
            _forward_only(q=q, k=k, rope=rope, g_q=g_q, g_k=g_k)
        D, dt, dev = self.head_dim, self.torch_dtype, self.device
        T = q.shape[0]
        vq = _view(q, "q", dt, self.heads, D, dev)
        if q_out is None:
            q_out = torch.empty(T, self.heads, D, dtype=dt, device=q.device)
        vk, k_ptr = None, 0
        if k is not None:
            vk = _view(k, "k", dt, self.heads_kv, D, dev, T)
            if k_out is None:
                k_out = torch.empty(T, self.heads_kv, D, dtype=dt, device=q.device)
            k_ptr = _ptr(k_out, "k_out", dt, (T, self.heads_kv, D), dev)
        rope_ptr, rope_len = self._rope(rope)
        pos = 0 if positions is None else _ptr(positions, "positions", torch.int32, (T,), dev)
        _lib.check(self._lib.engram_qk_norm_rope(
            self._h, vq, vk, T, pos, rope_ptr, rope_len, _norm_weight(g_q, "g_q", D, dev),
            _norm_weight(g_k, "g_k", D, dev), _ptr(q_out, "q_out", dt, (T, self.heads, D), dev), k_ptr,
            _current_stream(dev)), "engram_qk_norm_rope")
        return q_out, k_out


class SequenceBatch:
    """The sequences of a step (engram_sequences_t): ``start`` int32 [B+1] rows of the packed
    new tokens, ``length`` int32 [B] tokens in the cache once they are appended, ``table``
    int32 [B, pages] page ids.  ``max_new``: the most new tokens of a sequence, a launch hint
    (0: unknown).  The tensors are read when a call runs; they are those given here."""

    def __init__(self, start: torch.Tensor, length: torch.Tensor, table: torch.Tensor, max_new: int = 0):
        if length.dim() != 1 or table.dim() != 2:
            raise ValueError("length: expected [B]; table: expected [B, pages]")
        B = length.shape[0]
        self.start, self.length, self.table, self.max_new = start, length, table, int(max_new)
        self._fixed = (_dev(start, "start", torch.int32, (B + 1,)), _dev(length, "length", torch.int32, (B,)),
                       _dev(table, "table", torch.int32, (B, table.shape[1])), B, table.shape[1])
        self.device = start.get_device()
        for t, name in ((length, "length"), (table, "table")):
            if t.get_device() != self.device:
                raise _off_device(t, name, self.device)

    def _struct(self, tokens: int, device: int) -> bytes:
        if self.device != device:
            raise _off_device(self.start, "batch", device)
        return _pack_sequences(*self._fixed, tokens, self.max_new)


class PagedCache:
    """One layer's keys and values in pages: ``k`` and ``v`` [pages, heads_kv, page, head_dim]
    in the plan's type, owned by the caller, updated in place."""

    def __init__(self, plan: AttentionPlan, k: torch.Tensor, v: torch.Tensor):
        shape = (k.shape[0], plan.heads_kv, plan.page, plan.head_dim)
        self.plan, self.k, self.v = plan, k, v
        self._lib = plan._lib
        self._h = ctypes.c_void_p()
        _lib.check(self._lib.engram_kv_cache_create(plan._h, _ptr(k, "k", plan.torch_dtype, shape, plan.device),
                                                    _ptr(v, "v", plan.torch_dtype, shape, plan.device), k.shape[0],
                                                    ctypes.byref(self._h)), "engram_kv_cache_create")

    @classmethod
    def empty(cls, plan: AttentionPlan, pages: int, device=None) -> "PagedCache":
        shape = (pages, plan.heads_kv, plan.page, plan.head_dim)
        device = torch.device("cuda", plan.device) if device is None else device
        return cls(plan, torch.empty(shape, dtype=plan.torch_dtype, device=device),
                   torch.empty(shape, dtype=plan.torch_dtype, device=device))

    def close(self) -> None:
        if getattr(self, "_h", None) and self._h.value:
            self._lib.engram_kv_cache_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def append(self, batch: SequenceBatch, k: torch.Tensor, v: torch.Tensor, rope: Optional[torch.Tensor] = None, *,
               g_k: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
               g_q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
        """Append the new tokens' k (normed where g_k is given, rotated where rope is) and v
        [tokens, heads_kv, D]; with q, also its norm and rotation in the same launch
        (engram_kv_append).  Returns the queries, or None."""
        p = self.plan
        if not p._h:
            raise ValueError("cache: its plan is closed")
        if _grad_mode() and (k.requires_grad or v.requires_grad or q is not None and q.requires_grad
                             or rope is not None and rope.requires_grad or g_q is not None and g_q.requires_grad
                             or g_k is not None and g_k.requires_grad):
            _forward_only(k=k, v=v, rope=rope, g_k=g_k, q=q, g_q=g_q)
        D, dt, dev, T = p.head_dim, p.torch_dtype, p.device, k.shape[0]
        vk, vv = _view(k, "k", dt, p.heads_kv, D, dev), _view(v, "v", dt, p.heads_kv, D, dev, T)
        vq, q_ptr = None, 0
        if q is not None:
            vq = _view(q, "q", dt, p.heads, D, dev, T)
            if q_out is None:
                q_out = torch.empty(T, p.heads, D, dtype=dt, device=q.device)
            q_ptr = _ptr(q_out, "q_out", dt, (T, p.heads, D), dev)
        rope_ptr, rope_len = p._rope(rope)
        _lib.check(self._lib.engram_kv_append(
            self._h, batch._struct(T, dev), vk, vv, rope_ptr, rope_len, _norm_weight(g_k, "g_k", D, dev), vq,
            _norm_weight(g_q, "g_q", D, dev), q_ptr, _current_stream(dev)), "engram_kv_append")
        return q_out if q is not None else None

    def attend(self, batch: SequenceBatch, q: torch.Tensor, *, causal: bool = True, window: int = 0,
               out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Attention of the queries [tokens, heads, D] over the cache (engram_paged_attention):
        (out, lse float32 [tokens, heads]).  ``window``: keys that a query sees, its own the last
        (0: all).  Without a ``workspace`` the plan keeps one per stream."""
        p = self.plan
        if not p._h:
            raise ValueError("cache: its plan is closed")
        if _grad_mode() and q.requires_grad:
            _forward_only(q=q)
        D, dt, dev, T = p.head_dim, p.torch_dtype, p.device, q.shape[0]
        vq = _view(q, "q", dt, p.heads, D, dev)
        if out is None:
            out = torch.empty(T, p.heads, D, dtype=dt, device=q.device)
        if lse is None:
            lse = torch.empty(T, p.heads, dtype=torch.float32, device=q.device)
        s = _current_stream(dev)
        if workspace is None:
            ws = p._workspace(s)
            ws_ptr, ws_bytes = ws.data_ptr(), p.workspace_bytes
        else:
            ws_ptr, ws_bytes = _ptr(workspace, "workspace", torch.uint8, workspace.shape, dev), workspace.numel()
        _lib.check(self._lib.engram_paged_attention(
            self._h, batch._struct(T, dev), vq, int(causal), min(int(window), _INT_MAX), _ptr(out, "out", dt, (T, p.heads, D), dev),
            _ptr(lse, "lse", torch.float32, (T, p.heads), dev), ws_ptr, ws_bytes, s), "engram_paged_attention")
        return out, lse


def verify_drafts(target: torch.Tensor, drafts: torch.Tensor, u: torch.Tensor, *,
                  draft_probs: Optional[torch.Tensor] = None, n_drafts: Optional[torch.Tensor] = None,
                  tokens: Optional[torch.Tensor] = None, accepted: Optional[torch.Tensor] = None
                  ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Check drafted tokens int32 [B, S] against the target's probabilities [B, S+1, V] with the
    random numbers u [B, S+1] (engram_verify_drafts).  ``draft_probs`` [B, S, V], or None where
    each draft is certain; ``n_drafts`` int32 [B], or None for S each.  Returns (tokens int32
    [B, S+1], accepted int32 [B])."""
    if not isinstance(target, torch.Tensor) or target.dtype not in (torch.float32, torch.bfloat16) or target.dim() != 3:
        raise ValueError("target: expected float32 or bfloat16 [B, S+1, V]")
    if _grad_mode() and (target.requires_grad or u.requires_grad
                         or draft_probs is not None and draft_probs.requires_grad):
        _forward_only(target=target, draft_probs=draft_probs, u=u)
    B, S1, V = target.shape
    S, dev = S1 - 1, target.get_device()
    if dev < 0:
        raise ValueError("target: must be a CUDA tensor")
    if dev != _current_device():                      # which the launch goes to
        raise _off_device(target, "target", _current_device())
    if tokens is None:
        tokens = torch.empty(B, S1, dtype=torch.int32, device=target.device)
    if accepted is None:
        accepted = torch.empty(B, dtype=torch.int32, device=target.device)
    i32 = torch.int32
    _lib.check(_lib._lib().engram_verify_drafts(
        _ptr(target, "target", target.dtype, target.shape, dev),
        0 if draft_probs is None else _ptr(draft_probs, "draft_probs", target.dtype, (B, S, V), dev),
        _lib.F32 if target.dtype is torch.float32 else _lib.BF16, _ptr(drafts, "drafts", i32, (B, S), dev),
        0 if n_drafts is None else _ptr(n_drafts, "n_drafts", i32, (B,), dev), _ptr(u, "u", torch.float32, (B, S1), dev),
        B, S, V, _ptr(tokens, "tokens", i32, (B, S1), dev), _ptr(accepted, "accepted", i32, (B,), dev),
        _current_stream(dev)), "engram_verify_drafts")
    return tokens, accepted
