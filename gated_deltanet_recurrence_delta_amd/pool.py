"""A pool of recurrent states for serving (``include/gdn_pool.h``): the
token-by-token forms on states in slots, and the moving of slots."""
from __future__ import annotations

import math
from array import array

from . import GdnError, load
from .linear import _call, _decays, _like, _placed, _ptr, _raw_stream, _sizes

__all__ = ["gdn_fwd_recurrent_pool", "gdn_linear_fwd_recurrent_pool", "gdn_state_move", "fwd_recurrent_pool",
           "linear_fwd_recurrent_pool", "state_move", "StatePool"]


def gdn_fwd_recurrent_pool(q, k, v, g, beta, pool, slots, cu_seqlens, out, nslots, B, T, H, dk, dv, stream,
                           dtype) -> int:
    """Raw C call of the delta rule on a pool of states (0 = NULL).  Returns the status."""
    return load().gdn_fwd_recurrent_pool(q, k, v, g, beta, pool, slots, cu_seqlens, out, int(nslots), int(B), int(T),
                                         int(H), int(dk), int(dv), stream, int(dtype))


def gdn_linear_fwd_recurrent_pool(q, k, v, g, pool, slots, cu_seqlens, out, nslots, B, T, H, dk, dv, stream,
                                  dtype) -> int:
    """Raw C call of linear attention on a pool of states (0 = NULL).  Returns the status."""
    return load().gdn_linear_fwd_recurrent_pool(q, k, v, g, pool, slots, cu_seqlens, out, int(nslots), int(B), int(T),
                                                int(H), int(dk), int(dv), stream, int(dtype))


def gdn_state_move(pool, outer, slots, slot_bytes, src, dst, n, stream) -> int:
    """Raw C call of the slot moves; ``src`` and ``dst`` are host int32 arrays (their addresses, or ctypes arrays).  Returns the status."""
    return load().gdn_state_move(pool, int(outer), int(slots), int(slot_bytes), src, dst, int(n), stream)


def _pooled(q, k, v, pool, slots, cu_seqlens, out, stream, more):
    """Checked sizes, output and stream of a call on a pool."""
    import torch

    dtype, B, T, H, dk, dv = _sizes(q, k, v, cu_seqlens)
    if pool.dim() != 4:
        raise ValueError("pool must be (slots, H, dk, dv)")
    _like("pool", pool, (pool.shape[0], H, dk, dv), torch.float32)
    _like("slots", slots, (B,), torch.int32)
    dev = q.device
    _placed(dev, (q, k, v, pool, slots, cu_seqlens, out, *more))
    if out is None:
        out = torch.empty_like(v)
    else:
        _like("out", out, v.shape, v.dtype)
    return (pool.shape[0], B, T, H, dk, dv, _raw_stream(dev, stream), dtype), out


def fwd_recurrent_pool(q, k, v, g, beta, pool, slots, cu_seqlens=None, out=None, stream=None):
    """``fwd_recurrent`` (the gated delta rule, token by token) on states in a pool.

    pool: (slots, H, dk, dv) float32, updated in place; slots: (B,) int32 on
    the GPU, each sequence's own slot.  A sequence whose slot is outside the
    pool (-1 for a padding row) or an earlier sequence's changes no state and
    gets zeros.  Other arguments as for ``fwd_recurrent``.  Returns out.
    """
    import torch

    for name, t in (("g", g), ("beta", beta)):
        _like(name, t, q.shape[:-1], torch.float32)
    sizes, out = _pooled(q, k, v, pool, slots, cu_seqlens, out, stream, (g, beta))
    _call("gdn_fwd_recurrent_pool", q.device, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
          pool.data_ptr(), slots.data_ptr(), _ptr(cu_seqlens), out.data_ptr(), *sizes)
    return out


def linear_fwd_recurrent_pool(q, k, v, g, pool, slots, cu_seqlens=None, out=None, stream=None):
    """``linear_fwd_recurrent`` on states in a pool; pool and slots as for
    ``fwd_recurrent_pool``, g: (H,) float32.  Returns out."""
    _decays(g, q.shape[-2])
    sizes, out = _pooled(q, k, v, pool, slots, cu_seqlens, out, stream, (g,))
    _call("gdn_linear_fwd_recurrent_pool", q.device, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
          pool.data_ptr(), slots.data_ptr(), _ptr(cu_seqlens), out.data_ptr(), *sizes)
    return out


def _host_ints(name, x):
    """An int32 array from a list, a range, a NumPy array or a CPU tensor."""
    if type(x) is not list:
        if getattr(x, "is_cuda", False):
            raise TypeError(f"{name} must be on the host: the slots' owner knows them there")
        x = x.tolist() if hasattr(x, "tolist") else list(x)
    try:
        return array("i", x)
    except OverflowError:
        raise ValueError(f"{name} holds a number that is no slot") from None
    except TypeError:
        raise TypeError(f"{name} must be a sequence of ints") from None


def _check_moves(src, dst, slots):
    if len(src) != len(dst):
        raise ValueError(f"src and dst must have one length, got {len(src)} and {len(dst)}")
    if src and (min(src) < -1 or max(src) >= slots or min(dst) < 0 or max(dst) >= slots):
        raise ValueError(f"slots must lie in [0, {slots}) (src: or be -1)")
    if len(set(dst)) != len(dst):
        raise ValueError("a target may be written once only")


def state_move(pool, src, dst, dim=0, stream=None):
    """pool.select(dim, dst[i]) <- pool.select(dim, src[i]) for all i at once.

    Every source is read as it was before the call: one source may go to many
    targets (a fork), targets may be sources (a reordering), src[i] == -1
    clears a target.  ``pool``: a contiguous GPU tensor of any dtype whose
    slots, along ``dim``, are multiples of 16 bytes; ``src``, ``dst``: ints on
    the host, no target twice.  In place, on the current stream (or
    ``stream``); returns pool.
    """
    src, dst = _host_ints("src", src), _host_ints("dst", dst)
    shape = pool.shape
    if not -len(shape) <= dim < len(shape):
        raise ValueError(f"pool has no dimension {dim}")
    dim %= len(shape)
    slots, n, dev = shape[dim], len(src), pool.device
    if n != len(dst) or n > slots or pool.numel() == 0:
        _check_moves(src, dst, slots)
    _placed(dev, (pool,))
    if n == 0 or pool.numel() == 0:
        return pool
    try:
        _call("gdn_state_move", dev, pool.data_ptr(), math.prod(shape[:dim]), slots,
              math.prod(shape[dim + 1:]) * pool.element_size(), src.buffer_info()[0], dst.buffer_info()[0], n,
              _raw_stream(dev, stream))
    except GdnError:
        _check_moves(src, dst, slots)  # says which of the arguments it was
        raise
    return pool


class StatePool:
    """Slots of recurrent states and who holds them.

    ``states``: (slots, H, dk, dv) float32, or (layers, slots, H, dk, dv) with
    ``layers``; ``states[l]`` is what ``fwd_recurrent_pool`` and
    ``linear_fwd_recurrent_pool`` take for layer l.  The bookkeeping is the
    host's; copies run on the stream that is current at each call.
    """

    def __init__(self, slots, H, dk, dv, layers=None, device="cuda"):
        import torch

        shape = (slots, H, dk, dv) if layers is None else (layers, slots, H, dk, dv)
        self.states = torch.zeros(shape, dtype=torch.float32, device=device)
        self._dim = 0 if layers is None else 1
        self._free = list(range(slots))[::-1]  # the lowest slot is handed out first
        self._live = set()

    @property
    def live(self):
        """The slots in use, ascending."""
        return sorted(self._live)

    @property
    def free_slots(self):
        return len(self._free)

    def _check(self, slots):
        slots = _host_ints("slots", slots).tolist()
        for s in slots:
            if s not in self._live:
                raise ValueError(f"slot {s} is not in use")
        if len(set(slots)) != len(slots):
            raise ValueError("a slot is named twice")
        return slots

    def _take(self, n, src):
        """n free slots with the state of slot ``src`` (-1: zeros), in use once their states are queued."""
        if not 0 <= n <= len(self._free):
            raise ValueError(f"{n} slots are wanted, {len(self._free)} are free")
        got = self._free[len(self._free) - n:][::-1]
        self._move([src] * n, got)
        del self._free[len(self._free) - n:]
        self._live.update(got)
        return got

    def _move(self, src, dst):
        if self.states.numel():
            state_move(self.states, src, dst, dim=self._dim)

    def alloc(self, n=1):
        """n slots with zero states."""
        return self._take(n, -1)

    def fork(self, slot, n=1):
        """n new slots that hold copies of ``slot``'s state."""
        self._check([slot])
        return self._take(n, slot)

    def copy(self, src, dst):
        """State of src[i] into dst[i], all at once; slots in use."""
        src, dst = _host_ints("src", src).tolist(), self._check(dst)
        self._check(set(src))
        if len(src) != len(dst):
            raise ValueError("src and dst must have one length")
        self._move(src, dst)

    def free(self, slots):
        """Hands slots back; their states are left as they are."""
        slots = self._check(slots)
        self._live.difference_update(slots)
        self._free = sorted(self._free + slots, reverse=True)

    def compact(self):
        """Moves the states in use to slots 0 .. n - 1, as few as that takes;
        returns {old slot: new slot} of the moved ones."""
        n = len(self._live)
        src = sorted(s for s in self._live if s >= n)
        dst = sorted(set(range(n)) - self._live)
        self._move(src, dst)
        self._live = set(range(n))
        self._free = list(range(n, self.states.shape[self._dim]))[::-1]
        return dict(zip(src, dst))
