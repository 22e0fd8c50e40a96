"""Norms of every head's query and key with the position rotation
(``include/gdn_qk_norm.h``): y = rotate(w x r), r = (mean or sum of x^2 +
eps)^(-1/2), forwards and backwards.  Argument checks and marshalling only, as
in the package's other entry points.
"""
from __future__ import annotations

from . import load
from .conv import _flat, _storage
from .linear import _call, _like, _placed, _ptr, _raw_stream, _scratch

__all__ = ["gdn_qk_norm_fwd", "gdn_qk_norm_bwd", "gdn_qk_norm_workspace_size", "qk_norm_fwd", "qk_norm_bwd", "qk_norm"]

GDN_NORM_L2 = 1
GDN_NORM_INTERLEAVED = 2


def gdn_qk_norm_fwd(q, k, cos, sin, pos, wq, wk, qo, ko, B, T, Hq, Hk, d, rot, P, eps, stream, dtype, flags) -> int:
    """Raw C call with integer pointers (0 = NULL).  Returns the status."""
    return load().gdn_qk_norm_fwd(q, k, cos, sin, pos, wq, wk, qo, ko, int(B), int(T), int(Hq), int(Hk), int(d),
                                  int(rot), int(P), float(eps), stream, int(dtype), int(flags))


def gdn_qk_norm_bwd(q, k, cos, sin, pos, wq, wk, dqo, dko, dq, dk, dwq, dwk, B, T, Hq, Hk, d, rot, P, eps, stream,
                    dtype, flags, workspace, workspace_bytes) -> int:
    """Raw C call of the backward pass (0 = NULL).  Returns the status."""
    return load().gdn_qk_norm_bwd(q, k, cos, sin, pos, wq, wk, dqo, dko, dq, dk, dwq, dwk, int(B), int(T), int(Hq),
                                  int(Hk), int(d), int(rot), int(P), float(eps), stream, int(dtype), int(flags),
                                  workspace, int(workspace_bytes))


def gdn_qk_norm_workspace_size(B, T, Hq, Hk, d) -> int:
    """Workspace bytes ``gdn_qk_norm_bwd`` needs for the weights' gradients (negative: a status code)."""
    return load().gdn_qk_norm_workspace_size(int(B), int(T), int(Hq), int(Hk), int(d))


def _checked(q, k, cos, sin, pos, wq, wk, norm, interleaved):
    """(dtype code, sizes, table sizes, flags), the inputs checked against one another."""
    import torch

    dtype, f32 = _storage("q", q), torch.float32
    qs, ks = q.shape, k.shape
    lead, d = qs[:-2], qs[-1] if qs else 0
    if len(lead) not in (1, 2) or len(ks) != len(qs) or ks[:-2] != lead or ks[-1] != d:
        raise ValueError("q and k must be (B, T, heads, d), or (T, heads, d) packed, of the same tokens and width")
    if k.dtype != q.dtype:
        raise TypeError(f"q and k must share one dtype, got {q.dtype}, {k.dtype}")
    if norm not in ("rms", "l2"):
        raise ValueError(f"norm must be 'rms' or 'l2', got {norm!r}")
    B, T = lead if len(lead) == 2 else (1, lead[0])
    rot = P = 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    if cos is not None:
        shape = cos.shape
        if len(shape) != 2 or cos.dtype != f32 or shape[0] < 1 or 2 * shape[1] > d:
            raise ValueError(f"cos must be float32 of shape (positions, at most {d // 2}), got {cos.dtype} "
                             f"{tuple(shape)}")
        if sin.dtype != f32 or sin.shape != shape:
            _like("sin", sin, shape, f32)
        P, rot = shape[0], 2 * shape[1]
        if rot and pos is None and len(lead) == 1:
            raise ValueError("packed rows need their positions in pos")
    if pos is not None and (pos.dtype != torch.int32 or pos.shape != lead):
        _like("pos", pos, lead, torch.int32)
    if wq is not None and (wq.dtype != f32 or wq.shape != (d,)):
        _like("wq", wq, (d,), f32)
    if wk is not None and (wk.dtype != f32 or wk.shape != (d,)):
        _like("wk", wk, (d,), f32)
    flags = (GDN_NORM_L2 if norm == "l2" else 0) | (GDN_NORM_INTERLEAVED if interleaved else 0)
    return dtype, (B, T, qs[-2], ks[-2], d), (rot, P), flags


def qk_norm_fwd(q, k, cos=None, sin=None, pos=None, wq=None, wk=None, norm="rms", eps=1e-6, interleaved=False, qo=None,
                ko=None, stream=None):
    """Norm and rotation of queries and keys, on torch device tensors.

    q: (B,T,Hq,d), k: (B,T,Hk,d), or packed without B, float32 or bfloat16, d
    32, 64, 128 or 256; cos, sin: (P, rot/2) float32, the angles of positions 0
    to P-1, or None (no rotation); pos: int32 (B,T) or (T,), each token's
    position, None (with B) for 0 to T-1; wq, wk: (d,) float32 or None (ones).
    ``norm``: "rms" or "l2".  Pairs are channels (i, i + rot/2), or neighbours
    with ``interleaved``.  A token whose position is outside the tables (-1 for
    padding) gets zeros.  Returns (qo, ko).  Runs on the current stream (or
    ``stream``, with which the caller orders the tensors' other uses),
    asynchronously.
    """
    import torch

    dtype, sizes, table, flags = _checked(q, k, cos, sin, pos, wq, wk, norm, interleaved)
    if qo is not None:
        _like("qo", qo, q.shape, q.dtype)
    if ko is not None:
        _like("ko", ko, k.shape, k.dtype)
    dev = q.device
    _placed(dev, (q, k, cos, sin, pos, wq, wk, qo, ko))
    qo = torch.empty_like(q) if qo is None else qo
    ko = torch.empty_like(k) if ko is None else ko
    _call("gdn_qk_norm_fwd", dev, q.data_ptr(), k.data_ptr(), _ptr(cos), _ptr(sin), _ptr(pos), _ptr(wq), _ptr(wk),
          qo.data_ptr(), ko.data_ptr(), *sizes, *table, eps, _raw_stream(dev, stream), dtype, flags)
    return qo, ko


def qk_norm_bwd(q, k, dqo, dko, cos=None, sin=None, pos=None, wq=None, wk=None, norm="rms", eps=1e-6,
                interleaved=False, workspace=None, stream=None):
    """Gradients of <dqo, qo> + <dko, ko> for ``qk_norm_fwd``'s outputs.

    Arguments as for ``qk_norm_fwd``; dqo and dko have qo's and ko's shapes and
    dtype.  Returns a dict with dq, dk (the inputs' dtype) and dwq, dwk
    (float32, None without weights).  ``workspace``: a uint8 device tensor of at
    least ``gdn_qk_norm_workspace_size`` bytes, allocated here when None.
    """
    import torch

    dtype, sizes, table, flags = _checked(q, k, cos, sin, pos, wq, wk, norm, interleaved)
    _like("dqo", dqo, q.shape, q.dtype)
    _like("dko", dko, k.shape, k.dtype)
    dev = q.device
    _placed(dev, (q, k, cos, sin, pos, wq, wk, dqo, dko))
    need = gdn_qk_norm_workspace_size(*sizes) if wq is not None or wk is not None else 0
    ws, size = _scratch(need, workspace, dev, stream, "gdn_qk_norm_workspace_size")
    grads = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dwq": None if wq is None else torch.empty_like(wq),
             "dwk": None if wk is None else torch.empty_like(wk)}
    _call("gdn_qk_norm_bwd", dev, *(_ptr(t) for t in (q, k, cos, sin, pos, wq, wk, dqo, dko)),
          *(_ptr(grads[n]) for n in ("dq", "dk", "dwq", "dwk")), *sizes, *table, eps, _raw_stream(dev, stream), dtype,
          flags, _ptr(ws), size)
    return grads


_NORM = None


def qk_norm(q, k, cos=None, sin=None, pos=None, wq=None, wk=None, norm="rms", eps=1e-6, interleaved=False):
    """(qo, ko) of ``qk_norm_fwd`` as a differentiable torch operation:
    gradients for q, k, wq and wk through ``qk_norm_bwd``.  To capture a training
    step into a graph, call ``qk_norm_fwd`` and ``qk_norm_bwd`` themselves:
    autograd's own accumulation into leaves that an eager graph still holds
    waits for another stream, which a capture does not survive."""
    import torch

    global _NORM
    if _NORM is None:

        class _QkNorm(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, wq, wk, cos, sin, pos, norm, eps, interleaved):
                ctx.save_for_backward(q, k, wq, wk, cos, sin, pos)
                ctx.how = (norm, eps, interleaved)
                return qk_norm_fwd(q, k, cos, sin, pos, wq, wk, *ctx.how)

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dqo, dko):
                q, k, wq, wk, cos, sin, pos = ctx.saved_tensors
                g = qk_norm_bwd(q, k, _flat(dqo), _flat(dko), cos, sin, pos, wq, wk, *ctx.how)
                return g["dq"], g["dk"], g["dwq"], g["dwk"], None, None, None, None, None, None

        _NORM = _QkNorm
    for name, t in (("cos", cos), ("sin", sin)):
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} is a constant of the model: it gets no gradient")
    return _NORM.apply(q, k, wq, wk, cos, sin, pos, norm, eps, interleaved)

