"""The selective state space scan (``include/gdn_ssm.h``):

h_t = exp(s_t A) h_{t-1} + s_t x_t b_t,  y_t = c_t . h_t + D x_t,
out_t = y_t SiLU(z_t),  s_t = softplus(dt_t + dt_bias),  A = -exp(A_log),

per channel, for prompts, for training and on a pool of states.  Argument
checks and marshalling only, as in the package's other entry points.
"""
from __future__ import annotations

import functools

from . import load
from .conv import _batch, _flat, _optional, _pool_of, _storage
from .linear import _call, _like, _placed, _ptr, _raw_stream, _scratch

__all__ = ["gdn_ssm_fwd", "gdn_ssm_bwd", "gdn_ssm_workspace_size", "gdn_ssm_fwd_recurrent_pool", "ssm_fwd", "ssm_bwd",
           "ssm_fwd_recurrent_pool", "selective_scan"]

GDN_SSM_SOFTPLUS = 1


def gdn_ssm_fwd(x, dt, b, c, A_log, Dskip, z, dt_bias, h0, cu_seqlens, out, hT, B, T, D, G, N, stream, dtype, flags,
                workspace, workspace_bytes) -> int:
    """Raw C call with integer pointers (0 = NULL).  Returns the status."""
    return load().gdn_ssm_fwd(x, dt, b, c, A_log, Dskip, z, dt_bias, h0, cu_seqlens, out, hT, int(B), int(T), int(D),
                              int(G), int(N), stream, int(dtype), int(flags), workspace, int(workspace_bytes))


def gdn_ssm_bwd(x, dt, b, c, A_log, Dskip, z, dt_bias, h0, cu_seqlens, dout, dhT, dx, ddt, db, dc, dA_log, dD, dz,
                ddt_bias, dh0, B, T, D, G, N, stream, dtype, flags, workspace, workspace_bytes) -> int:
    """Raw C call of the backward pass (0 = NULL).  Returns the status."""
    return load().gdn_ssm_bwd(x, dt, b, c, A_log, Dskip, z, dt_bias, h0, cu_seqlens, dout, dhT, dx, ddt, db, dc,
                              dA_log, dD, dz, ddt_bias, dh0, int(B), int(T), int(D), int(G), int(N), stream,
                              int(dtype), int(flags), workspace, int(workspace_bytes))


def gdn_ssm_workspace_size(B, T, D, G, N, packed, dtype, backward=False) -> int:
    """Workspace bytes ``gdn_ssm_fwd`` (or ``gdn_ssm_bwd``) needs (negative: a status code)."""
    return load().gdn_ssm_workspace_size(int(B), int(T), int(D), int(G), int(N), int(packed), int(dtype),
                                         int(backward))


def gdn_ssm_fwd_recurrent_pool(x, dt, b, c, A_log, Dskip, z, dt_bias, pool, slots, cu_seqlens, out, nslots, B, T, D, G,
                               N, stream, dtype, flags) -> int:
    """Raw C call on a pool of states (0 = NULL).  Returns the status."""
    return load().gdn_ssm_fwd_recurrent_pool(x, dt, b, c, A_log, Dskip, z, dt_bias, pool, slots, cu_seqlens, out,
                                             int(nslots), int(B), int(T), int(D), int(G), int(N), stream, int(dtype),
                                             int(flags))


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(*sizes):
    return gdn_ssm_workspace_size(*sizes)


def _sizes(x, dt, b, c, A_log, D, z, dt_bias, cu_seqlens):
    """(dtype code, B, T, channels, groups, states), the inputs checked against one another.

    (The comparisons stand here and not in _like, which says what is wrong: a call a tensor less on the way of every
    decoded token.)"""
    import torch

    dtype = _storage("x", x)
    B, T = _batch("x", x, cu_seqlens, 1)
    xt, xs, bs, f32 = x.dtype, x.shape, b.shape, torch.float32
    channels = xs[-1]
    if dt.dtype != xt or dt.shape != xs:
        _like("dt", dt, xs, xt)
    if z is not None and (z.dtype != xt or z.shape != xs):
        _like("z", z, xs, xt)
    if len(bs) != len(xs) + 1 or bs[:-2] != xs[:-1]:
        raise ValueError(f"b must be {tuple(xs[:-1])} + (G, N), got {tuple(bs)}")
    G, N = bs[-2:]
    if G < 1 or channels % G:
        raise ValueError(f"{channels} channels do not divide into {G} groups")
    if b.dtype != xt:
        _like("b", b, bs, xt)
    if c.dtype != xt or c.shape != bs:
        _like("c", c, bs, xt)
    if A_log.dtype != f32 or A_log.shape != (channels, N):
        _like("A_log", A_log, (channels, N), f32)
    if D is not None and (D.dtype != f32 or D.shape != (channels,)):
        _like("D", D, (channels,), f32)
    if dt_bias is not None and (dt_bias.dtype != f32 or dt_bias.shape != (channels,)):
        _like("dt_bias", dt_bias, (channels,), f32)
    return dtype, B, T, channels, G, N


def ssm_fwd(x, dt, b, c, A_log, D=None, z=None, dt_bias=None, h0=None, cu_seqlens=None, softplus=True, out=None,
            hT=None, stream=None, workspace=None):
    """The selective scan over whole sequences, on torch device tensors.

    x, dt, z: (B,T,D), float32 or bfloat16; b, c: (B,T,G,N) of the same dtype,
    channel d using group d // (D / G), N 16, 32 or 64 (packed: drop B and pass
    int32 ``cu_seqlens`` of length B+1); A_log: (D,N), D (the skip) and
    dt_bias: (D,), float32; h0: (B,D,N) float32 or None.  Without ``softplus``
    the step is dt + dt_bias itself.  Returns (out, hT), out of x's dtype, hT
    float32; rows of no sequence are not written.  Runs on the current stream
    (or ``stream``, with which the caller orders the tensors' other uses),
    asynchronously.  ``workspace``: a uint8 device tensor of at least
    ``gdn_ssm_workspace_size`` bytes, allocated here when None.
    """
    import torch

    dtype, B, T, channels, G, N = _sizes(x, dt, b, c, A_log, D, z, dt_bias, cu_seqlens)
    state = (B, channels, N)
    _optional("h0", h0, state, torch.float32)
    _optional("out", out, x.shape, x.dtype)
    _optional("hT", hT, state, torch.float32)
    dev = x.device
    _placed(dev, (x, dt, b, c, A_log, D, z, dt_bias, h0, cu_seqlens, out, hT))
    need = _workspace_bytes(B, T, channels, G, N, cu_seqlens is not None, dtype)
    ws, size = _scratch(need, workspace, dev, stream, "gdn_ssm_workspace_size")
    if out is None:
        out = torch.empty_like(x)
    if hT is None:
        hT = torch.empty(state, dtype=torch.float32, device=dev)
    _call("gdn_ssm_fwd", dev, x.data_ptr(), dt.data_ptr(), b.data_ptr(), c.data_ptr(), A_log.data_ptr(), _ptr(D),
          _ptr(z), _ptr(dt_bias), _ptr(h0), _ptr(cu_seqlens), out.data_ptr(), hT.data_ptr(), B, T, channels, G, N,
          _raw_stream(dev, stream), dtype, GDN_SSM_SOFTPLUS if softplus else 0, _ptr(ws), size)
    return out, hT


def ssm_bwd(x, dt, b, c, A_log, dout, D=None, z=None, dt_bias=None, h0=None, cu_seqlens=None, dhT=None, softplus=True,
            want_dh0=True, workspace=None, stream=None):
    """Gradients of <dout, out> + <dhT, hT> for ``ssm_fwd``'s outputs.

    Arguments as for ``ssm_fwd``; dout has out's shape and dtype, dhT is
    (B,D,N) float32 or None (zero).  Returns a dict with dx, ddt, db, dc and dz
    (the inputs' dtype; rows of no sequence are not written), dA_log, dD,
    ddt_bias and dh0 (float32); those of inputs that are None are None, and dh0
    where ``want_dh0`` is false.
    """
    return _backward(x, dt, b, c, A_log, dout, D, z, dt_bias, h0, cu_seqlens, dhT, softplus, want_dh0, workspace,
                     stream, False)


def _backward(x, dt, b, c, A_log, dout, D, z, dt_bias, h0, cu_seqlens, dhT, softplus, want_dh0, workspace, stream,
              clear):
    """``ssm_bwd``; ``clear``: rows of no sequence get zeros."""
    import torch

    dtype, B, T, channels, G, N = _sizes(x, dt, b, c, A_log, D, z, dt_bias, cu_seqlens)
    state = (B, channels, N)
    _like("dout", dout, x.shape, x.dtype)
    _optional("h0", h0, state, torch.float32)
    _optional("dhT", dhT, state, torch.float32)
    dev = x.device
    _placed(dev, (x, dt, b, c, A_log, D, z, dt_bias, h0, cu_seqlens, dout, dhT))
    need = _workspace_bytes(B, T, channels, G, N, cu_seqlens is not None, dtype, True)
    ws, size = _scratch(need, workspace, dev, stream, "gdn_ssm_workspace_size")
    new = torch.zeros_like if clear else torch.empty_like
    maybe = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
    grads = {"dx": new(x), "ddt": new(dt), "db": new(b), "dc": new(c), "dA_log": torch.empty_like(A_log),
             "dD": maybe(D), "dz": None if z is None else new(z), "ddt_bias": maybe(dt_bias),
             "dh0": torch.empty(state, dtype=torch.float32, device=dev) if want_dh0 else None}
    _call("gdn_ssm_bwd", dev, *(_ptr(t) for t in (x, dt, b, c, A_log, D, z, dt_bias, h0, cu_seqlens, dout, dhT)),
          *(_ptr(grads[n]) for n in ("dx", "ddt", "db", "dc", "dA_log", "dD", "dz", "ddt_bias", "dh0")),
          B, T, channels, G, N, _raw_stream(dev, stream), dtype, GDN_SSM_SOFTPLUS if softplus else 0, _ptr(ws), size)
    return grads


def ssm_fwd_recurrent_pool(x, dt, b, c, A_log, pool, slots, D=None, z=None, dt_bias=None, cu_seqlens=None,
                           softplus=True, out=None, stream=None):
    """The scan token by token for decoding, on states in a pool.

    pool: (slots, D, N) float32, updated in place; slots: (B,) int32 on the GPU,
    each sequence's own slot.  A sequence whose slot is outside the pool (-1 for
    a padding row) or an earlier sequence's changes no state and gets zeros.
    Other arguments as for ``ssm_fwd``.  Returns out.
    """
    import torch

    dtype, B, T, channels, G, N = _sizes(x, dt, b, c, A_log, D, z, dt_bias, cu_seqlens)
    nslots = _pool_of(pool, slots, B, (channels, N), torch.float32)
    dev = x.device
    if out is None:
        out = torch.empty_like(x)
    else:
        _like("out", out, x.shape, x.dtype)
    _placed(dev, (x, dt, b, c, A_log, D, z, dt_bias, pool, slots, cu_seqlens, out))
    _call("gdn_ssm_fwd_recurrent_pool", dev, x.data_ptr(), dt.data_ptr(), b.data_ptr(), c.data_ptr(), A_log.data_ptr(),
          _ptr(D), _ptr(z), _ptr(dt_bias), pool.data_ptr(), slots.data_ptr(), _ptr(cu_seqlens), out.data_ptr(),
          nslots, B, T, channels, G, N, _raw_stream(dev, stream), dtype, GDN_SSM_SOFTPLUS if softplus else 0)
    return out


_SCAN = None


def selective_scan(x, dt, b, c, A_log, D=None, z=None, dt_bias=None, h0=None, cu_seqlens=None, softplus=True):
    """(out, hT) of ``ssm_fwd`` as a differentiable torch operation: gradients
    for every tensor but cu_seqlens through ``ssm_bwd``.  With packed sequences
    that leave rows out, those rows' outputs and gradients are zero.  To capture
    a training step into a graph, call ``ssm_fwd`` and ``ssm_bwd`` themselves:
    autograd's own accumulation into leaves that an eager graph still holds
    waits for another stream, which a capture does not survive."""
    global _SCAN
    if _SCAN is None:
        import torch

        class _SelectiveScan(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, dt, b, c, A_log, D, z, dt_bias, h0, cu_seqlens, softplus):
                out = None if cu_seqlens is None else torch.zeros_like(x)
                out, hT = ssm_fwd(x, dt, b, c, A_log, D, z, dt_bias, h0, cu_seqlens, softplus, out=out)
                ctx.save_for_backward(x, dt, b, c, A_log, D, z, dt_bias, h0, cu_seqlens)
                ctx.softplus = softplus
                return out, hT

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dout, dhT):
                x, dt, b, c, A_log, D, z, dt_bias, h0, cu_seqlens = ctx.saved_tensors
                g = _backward(x, dt, b, c, A_log, _flat(dout), D, z, dt_bias, h0, cu_seqlens, _flat(dhT),
                              ctx.softplus, h0 is not None, None, None, cu_seqlens is not None)
                return (*(g[n] for n in ("dx", "ddt", "db", "dc", "dA_log", "dD", "dz", "ddt_bias", "dh0")), None,
                        None)

        _SCAN = _SelectiveScan
    return _SCAN.apply(x, dt, b, c, A_log, D, z, dt_bias, h0, cu_seqlens, softplus)
