"""The short causal convolution before a recurrence (``include/gdn_conv.h``):

y_t = bias + sum_i w_i x_{t-W+1+i} per channel, through SiLU,

for prompts, for training and on a pool of states.  Argument checks and
marshalling only, as in the package's other entry points.
"""
from __future__ import annotations

import functools

from . import GDN_BF16, GDN_F32, load
from .linear import _call, _like, _placed, _ptr, _raw_stream, _scratch

__all__ = ["gdn_conv_fwd", "gdn_conv_bwd", "gdn_conv_workspace_size", "gdn_conv_fwd_pool", "conv_fwd", "conv_bwd",
           "conv_fwd_pool", "causal_conv"]

GDN_CONV_SILU = 1


def gdn_conv_fwd(x, w, bias, h0, cu_seqlens, out, hT, B, T, D, W, stream, dtype, flags) -> int:
    """Raw C call with integer pointers (0 = NULL).  Returns the status."""
    return load().gdn_conv_fwd(x, w, bias, h0, cu_seqlens, out, hT, int(B), int(T), int(D), int(W), stream, int(dtype),
                               int(flags))


def gdn_conv_bwd(x, w, bias, h0, cu_seqlens, dout, dhT, dx, dw, dbias, dh0, B, T, D, W, stream, dtype, flags,
                 workspace, workspace_bytes) -> int:
    """Raw C call of the backward pass (0 = NULL).  Returns the status."""
    return load().gdn_conv_bwd(x, w, bias, h0, cu_seqlens, dout, dhT, dx, dw, dbias, dh0, int(B), int(T), int(D),
                               int(W), stream, int(dtype), int(flags), workspace, int(workspace_bytes))


def gdn_conv_workspace_size(B, T, D, W, packed, dtype) -> int:
    """Workspace bytes ``gdn_conv_bwd`` needs (negative: a status code)."""
    return load().gdn_conv_workspace_size(int(B), int(T), int(D), int(W), int(packed), int(dtype))


def gdn_conv_fwd_pool(x, w, bias, pool, slots, cu_seqlens, out, nslots, B, T, D, W, stream, dtype, flags) -> int:
    """Raw C call on a pool of states (0 = NULL).  Returns the status."""
    return load().gdn_conv_fwd_pool(x, w, bias, pool, slots, cu_seqlens, out, int(nslots), int(B), int(T), int(D),
                                    int(W), stream, int(dtype), int(flags))


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(*sizes):
    return gdn_conv_workspace_size(*sizes)


def _storage(name, t):
    """The dtype code of a tensor of tokens."""
    import torch

    dtype = t.dtype
    if dtype is torch.bfloat16:
        return GDN_BF16
    if dtype is torch.float32:
        return GDN_F32
    raise TypeError(f"{name} dtype must be float32 or bfloat16, got {dtype}")


def _batch(name, t, cu_seqlens, dims):
    """(B, T) of a tensor of tokens with ``dims`` dimensions behind them."""
    import torch

    shape = t.shape
    if cu_seqlens is None:
        if len(shape) != dims + 2:
            raise ValueError(f"{name} must have {dims + 2} dimensions, (B, T, ...)")
        return shape[0], shape[1]
    if cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be one-dimensional, with at least one entry")
    if len(shape) != dims + 1:
        raise ValueError(f"packed {name} must have {dims + 1} dimensions, (T, ...)")
    return cu_seqlens.numel() - 1, shape[0]


def _flat(t):
    """A gradient contiguous and at an address that the kernels take: autograd's may be a part of a larger tensor."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _optional(name, t, shape, dtype):
    if t is not None:
        _like(name, t, shape, dtype)


def _sizes(x, w, bias, cu_seqlens):
    import torch

    dtype = _storage("x", x)
    B, T = _batch("x", x, cu_seqlens, 1)
    D, ws = x.shape[-1], w.shape
    if len(ws) != 2 or ws[0] != D or w.dtype != torch.float32:
        raise ValueError(f"w must be float32 of shape ({D}, W), got {w.dtype} {tuple(ws)}")
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (D,)):
        _like("bias", bias, (D,), torch.float32)
    return dtype, B, T, D, ws[1]


def conv_fwd(x, w, bias=None, h0=None, cu_seqlens=None, silu=True, out=None, hT=None, stream=None):
    """The causal convolution over whole sequences, on torch device tensors.

    x: (B,T,D) float32 or bfloat16 (packed: (T,D) and int32 ``cu_seqlens`` of
    length B+1); w: (D,W) float32, W 2 to 4, the last tap the token's own;
    bias: (D,) float32 or None; h0: (B,W-1,D) of x's dtype, the tokens before
    the first, or None (zeros).  Returns (out, hT), hT the last W-1 tokens;
    rows of no sequence are not written.  Runs on the current stream (or
    ``stream``, with which the caller orders the tensors' other uses),
    asynchronously.
    """
    import torch

    dtype, B, T, D, W = _sizes(x, w, bias, cu_seqlens)
    state = (B, W - 1, D)
    _optional("h0", h0, state, x.dtype)
    _optional("out", out, x.shape, x.dtype)
    _optional("hT", hT, state, x.dtype)
    dev = x.device
    _placed(dev, (x, w, bias, h0, cu_seqlens, out, hT))
    if out is None:
        out = torch.empty_like(x)
    if hT is None:
        hT = torch.empty((B, max(W - 1, 0), D), dtype=x.dtype, device=dev)
    _call("gdn_conv_fwd", dev, x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(h0), _ptr(cu_seqlens), out.data_ptr(),
          hT.data_ptr(), B, T, D, W, _raw_stream(dev, stream), dtype, GDN_CONV_SILU if silu else 0)
    return out, hT


def conv_bwd(x, w, dout, bias=None, h0=None, cu_seqlens=None, dhT=None, silu=True, want_dh0=True, workspace=None,
             stream=None):
    """Gradients of <dout, out> + <dhT, hT> for ``conv_fwd``'s outputs.

    Arguments as for ``conv_fwd``; dout has out's shape and dtype, dhT h0's or
    None (zero).  Returns a dict with dx (x's dtype; rows of no sequence are not
    written), dw (float32), dbias (float32, None without a bias) and dh0 (x's
    dtype, None when ``want_dh0`` is false).  ``workspace``: a uint8 device
    tensor of at least ``gdn_conv_workspace_size`` bytes, allocated here when
    None.
    """
    return _backward(x, w, dout, bias, h0, cu_seqlens, dhT, silu, want_dh0, workspace, stream, False)


def _backward(x, w, dout, bias, h0, cu_seqlens, dhT, silu, want_dh0, workspace, stream, clear):
    """``conv_bwd``; ``clear``: rows of no sequence get zeros."""
    import torch

    dtype, B, T, D, W = _sizes(x, w, bias, cu_seqlens)
    state = (B, W - 1, D)
    _like("dout", dout, x.shape, x.dtype)
    _optional("h0", h0, state, x.dtype)
    _optional("dhT", dhT, state, x.dtype)
    dev = x.device
    _placed(dev, (x, w, bias, h0, cu_seqlens, dout, dhT))
    need = _workspace_bytes(B, T, D, W, cu_seqlens is not None, dtype)
    ws, size = _scratch(need, workspace, dev, stream, "gdn_conv_workspace_size")
    grads = {"dx": torch.zeros_like(x) if clear else torch.empty_like(x), "dw": torch.empty_like(w),
             "dbias": None if bias is None else torch.empty_like(bias),
             "dh0": torch.empty(state, dtype=x.dtype, device=dev) if want_dh0 else None}
    _call("gdn_conv_bwd", dev, _ptr(x), _ptr(w), _ptr(bias), _ptr(h0), _ptr(cu_seqlens), _ptr(dout), _ptr(dhT),
          _ptr(grads["dx"]), _ptr(grads["dw"]), _ptr(grads["dbias"]), _ptr(grads["dh0"]), B, T, D, W,
          _raw_stream(dev, stream), dtype, GDN_CONV_SILU if silu else 0, _ptr(ws), size)
    return grads


def _pool_of(pool, slots, B, state, dtype):
    """The number of a pool's slots, pool and slots checked."""
    import torch

    shape = pool.shape
    if pool.dtype != dtype or shape[1:] != state or not shape:
        raise ValueError(f"pool must be {dtype} of shape (slots, {', '.join(map(str, state))}), got {pool.dtype} "
                         f"{tuple(shape)}")
    if slots.dtype != torch.int32 or slots.shape != (B,):
        _like("slots", slots, (B,), torch.int32)
    return shape[0]


def conv_fwd_pool(x, w, pool, slots, bias=None, cu_seqlens=None, silu=True, out=None, stream=None):
    """``conv_fwd`` for decoding, on states in a pool.

    pool: (slots, W-1, D) of x's dtype, updated in place; slots: (B,) int32 on
    the GPU, each sequence's own slot.  A sequence whose slot is outside the
    pool (-1 for a padding row) or an earlier sequence's changes no state and
    gets zeros.  Other arguments as for ``conv_fwd``.  Returns out.
    """
    import torch

    dtype, B, T, D, W = _sizes(x, w, bias, cu_seqlens)
    nslots = _pool_of(pool, slots, B, (W - 1, D), x.dtype)
    dev = x.device
    if out is None:
        out = torch.empty_like(x)
    else:
        _like("out", out, x.shape, x.dtype)
    _placed(dev, (x, w, bias, pool, slots, cu_seqlens, out))
    _call("gdn_conv_fwd_pool", dev, x.data_ptr(), w.data_ptr(), _ptr(bias), pool.data_ptr(), slots.data_ptr(),
          _ptr(cu_seqlens), out.data_ptr(), nslots, B, T, D, W, _raw_stream(dev, stream), dtype,
          GDN_CONV_SILU if silu else 0)
    return out


_CONV = None


def causal_conv(x, w, bias=None, h0=None, cu_seqlens=None, silu=True):
    """(out, hT) of ``conv_fwd`` as a differentiable torch operation: gradients
    for x, w, bias and h0 through ``conv_bwd``.  With packed sequences that
    leave rows out, those rows' outputs and gradients are zero.  To capture a
    training step into a graph, call ``conv_fwd`` and ``conv_bwd`` themselves:
    autograd's own accumulation into leaves that an eager graph still holds
    waits for another stream, which a capture does not survive."""
    global _CONV
    if _CONV is None:
        import torch

        class _CausalConv(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, w, bias, h0, cu_seqlens, silu):
                out = None if cu_seqlens is None else torch.zeros_like(x)
                out, hT = conv_fwd(x, w, bias, h0, cu_seqlens, silu, out=out)
                ctx.save_for_backward(x, w, bias, h0, cu_seqlens)
                ctx.silu = silu
                return out, hT

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dout, dhT):
                x, w, bias, h0, cu_seqlens = ctx.saved_tensors
                g = _backward(x, w, _flat(dout), bias, h0, cu_seqlens, _flat(dhT), ctx.silu,
                              h0 is not None, None, None, cu_seqlens is not None)
                return g["dx"], g["dw"], g["dbias"], g["dh0"], None, None

        _CONV = _CausalConv
    return _CONV.apply(x, w, bias, h0, cu_seqlens, silu)
