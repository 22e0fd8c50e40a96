"""Linear attention with one fixed decay per head (``include/gdn_linear.h``):

S_t = a_h S_{t-1} + k_t v_t^T,  o_t = S_t^T q_t,  a_h = exp(g_h),

the delta rule without its erase term.  Argument checks and marshalling only,
as in the package's other entry points.
"""
from __future__ import annotations

import functools

from . import GDN_BF16, GDN_F32, GdnError, load, strerror

__all__ = ["gdn_linear_fwd", "gdn_linear_fwd_recurrent", "gdn_linear_bwd", "gdn_linear_workspace_size",
           "linear_fwd", "linear_fwd_recurrent", "linear_bwd", "linear_attention"]


def gdn_linear_fwd(q, k, v, g, h0, cu_seqlens, out, hT, B, T, H, dk, dv, stream, dtype, workspace,
                   workspace_bytes) -> int:
    """Raw C call with integer pointers (0 = NULL).  Returns the status."""
    return load().gdn_linear_fwd(q, k, v, g, h0, cu_seqlens, out, hT, int(B), int(T), int(H), int(dk), int(dv),
                                 stream, int(dtype), workspace, int(workspace_bytes))


def gdn_linear_fwd_recurrent(q, k, v, g, h0, cu_seqlens, out, hT, B, T, H, dk, dv, stream, dtype) -> int:
    """Raw C call of the token-by-token form (0 = NULL).  Returns the status."""
    return load().gdn_linear_fwd_recurrent(q, k, v, g, h0, cu_seqlens, out, hT, int(B), int(T), int(H), int(dk),
                                           int(dv), stream, int(dtype))


def gdn_linear_bwd(q, k, v, g, h0, cu_seqlens, dout, dhT, dq, dk, dv, dh0, B, T, H, dk_, dv_, stream, dtype,
                   workspace, workspace_bytes) -> int:
    """Raw C call of the backward pass (0 = NULL).  Returns the status."""
    return load().gdn_linear_bwd(q, k, v, g, h0, cu_seqlens, dout, dhT, dq, dk, dv, dh0, int(B), int(T), int(H),
                                 int(dk_), int(dv_), stream, int(dtype), workspace, int(workspace_bytes))


def gdn_linear_workspace_size(B, T, H, dk, dv, packed, dtype, backward=False) -> int:
    """Workspace bytes ``gdn_linear_fwd`` (or ``gdn_linear_bwd``) needs (negative: a status code)."""
    return load().gdn_linear_workspace_size(int(B), int(T), int(H), int(dk), int(dv), int(packed), int(dtype),
                                            int(backward))


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(B, T, H, dk, dv, packed, dtype, backward):
    return gdn_linear_workspace_size(B, T, H, dk, dv, packed, dtype, backward)


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _sizes(q, k, v, cu_seqlens):
    """(dtype code, B, T, H, dk, dv) of a call's token tensors, checked against one another."""
    import torch

    qt, qs, vs = q.dtype, q.shape, v.shape
    if qt == torch.bfloat16:
        dtype = GDN_BF16
    elif qt == torch.float32:
        dtype = GDN_F32
    else:
        raise TypeError(f"q/k/v dtype must be float32 or bfloat16, got {qt}")
    if k.dtype != qt or v.dtype != qt:
        raise TypeError(f"q/k/v must share one dtype, got {qt}, {k.dtype}, {v.dtype}")
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32:
            raise TypeError("cu_seqlens must be int32")
        if len(qs) != 3:
            raise ValueError("packed q must be (T, H, dk)")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be one-dimensional, with at least one entry")
        T, H, dk = qs
        B = cu_seqlens.numel() - 1
    else:
        if len(qs) != 4:
            raise ValueError("q must be (B, T, H, dk)")
        B, T, H, dk = qs
    if k.shape != qs or len(vs) != len(qs) or vs[:-1] != qs[:-1]:
        raise ValueError("q, k, v shapes disagree")
    return dtype, B, T, H, dk, vs[-1]


def _placed(dev, tensors):
    """Every tensor contiguous and on the GPU ``dev``."""
    if dev.type != "cuda":
        raise ValueError("all tensors must be on the same GPU device")
    for t in tensors:
        if t is not None:
            if t.device != dev:
                raise ValueError("all tensors must be on the same GPU device")
            if not t.is_contiguous():
                raise ValueError("all tensors must be contiguous")


def _like(name, t, shape, dtype):
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _raw_stream(dev, stream):
    """The handle of ``stream``, or of ``dev``'s current stream."""
    import torch

    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"stream must be one of {dev}, got one of {stream.device}")
        return stream.cuda_stream
    try:
        return torch._C._cuda_getCurrentRawStream(dev.index)  # without the Stream object around it
    except AttributeError:
        return torch.cuda.current_stream(dev).cuda_stream


def _call(name, dev, *args):
    """The C entry point ``name`` with ``dev`` as the current device; raises on its status."""
    import torch

    fn = getattr(load(), name)
    if torch.cuda.current_device() == dev.index:
        rc = fn(*args)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args)
    if rc != 0:
        raise GdnError(rc, strerror(rc), name)


def _decays(g, H):
    import torch

    _like("g", g, (H,), torch.float32)
    if g.requires_grad and torch.is_grad_enabled():
        raise ValueError("g is a constant of the model: it gets no gradient")


def _scratch(need, workspace, dev, stream):
    """The call's workspace: the caller's, or one from the memory of the stream it runs on."""
    import torch

    if need < 0:
        raise GdnError(need, strerror(need), "gdn_linear_workspace_size")
    if workspace is None:
        if need == 0:
            return None, 0
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        else:
            with torch.cuda.stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous() or \
            workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be contiguous, on q's device and hold {need} bytes")
    return workspace, workspace.numel() * workspace.element_size()


def _forward_args(q, k, v, g, h0, cu_seqlens, out, hT, stream):
    import torch

    dtype, B, T, H, dk, dv = _sizes(q, k, v, cu_seqlens)
    _decays(g, H)
    dev = q.device
    _placed(dev, (q, k, v, g, h0, cu_seqlens, out, hT))
    if h0 is not None:
        _like("h0", h0, (B, H, dk, dv), torch.float32)
    if out is None:
        out = torch.empty_like(v)
    else:
        _like("out", out, v.shape, v.dtype)
    if hT is None:
        hT = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    else:
        _like("hT", hT, (B, H, dk, dv), torch.float32)
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _ptr(h0), _ptr(cu_seqlens), out.data_ptr(),
            hT.data_ptr(), B, T, H, dk, dv, _raw_stream(dev, stream), dtype)
    return args, out, hT


def linear_fwd(q, k, v, g, h0=None, cu_seqlens=None, out=None, hT=None, stream=None, workspace=None):
    """Linear attention with a decay per head on torch device tensors (chunkwise form).

    q, k: (B,T,H,dk); v: (B,T,H,dv), one dtype, float32 or bfloat16; g: (H,)
    float32, the natural logarithm of each head's decay, <= 0 (packed: drop B
    and pass int32 ``cu_seqlens`` of length B+1); h0: (B,H,dk,dv) float32 or
    None.  A sequence's rows of a tensor, or a whole packed batch's, are
    fewer than 2^31 bytes.  Returns (out, hT); out has q's dtype, hT is float32; rows of no
    sequence are not written.  Runs on the current stream (or ``stream``, with
    which the caller orders the tensors' other uses), asynchronously.
    ``workspace``: a uint8 device tensor of at least
    ``gdn_linear_workspace_size`` bytes, allocated here when None.
    """
    args, out, hT = _forward_args(q, k, v, g, h0, cu_seqlens, out, hT, stream)
    need = _workspace_bytes(*args[8:13], cu_seqlens is not None, args[14], False)
    ws, size = _scratch(need, workspace, q.device, stream)
    _call("gdn_linear_fwd", q.device, *args, _ptr(ws), size)
    return out, hT


def linear_fwd_recurrent(q, k, v, g, h0=None, cu_seqlens=None, out=None, hT=None, stream=None):
    """Token-by-token form of ``linear_fwd`` (decoding and short sequences)."""
    args, out, hT = _forward_args(q, k, v, g, h0, cu_seqlens, out, hT, stream)
    _call("gdn_linear_fwd_recurrent", q.device, *args)
    return out, hT


def linear_bwd(q, k, v, g, dout, h0=None, cu_seqlens=None, dhT=None, want_dh0=True, workspace=None, stream=None):
    """Gradients of <dout, out> + <dhT, hT> for ``linear_fwd``'s outputs.

    Arguments as for ``linear_fwd``; dout has out's shape and dtype, dhT is
    (B,H,dk,dv) float32 or None (zero).  Returns a dict with dq, dk, dv (the
    inputs' dtype; rows of no sequence are not written) and dh0 (float32, or
    None when ``want_dh0`` is false); g, a constant, has none.
    """
    return _backward(q, k, v, g, dout, h0, cu_seqlens, dhT, want_dh0, workspace, stream, False)


def _backward(q, k, v, g, dout, h0, cu_seqlens, dhT, want_dh0, workspace, stream, clear):
    """``linear_bwd``; ``clear``: rows of no sequence get zeros."""
    import torch

    dtype, B, T, H, dk, dv = _sizes(q, k, v, cu_seqlens)
    _decays(g, H)
    dev = q.device
    _like("dout", dout, v.shape, v.dtype)
    for name, t in (("h0", h0), ("dhT", dhT)):
        if t is not None:
            _like(name, t, (B, H, dk, dv), torch.float32)
    _placed(dev, (q, k, v, g, h0, cu_seqlens, dout, dhT))
    need = _workspace_bytes(B, T, H, dk, dv, cu_seqlens is not None, dtype, True)
    ws, size = _scratch(need, workspace, dev, stream)
    new = torch.zeros_like if clear else torch.empty_like
    grads = {"dq": new(q), "dk": new(k), "dv": new(v),
             "dh0": torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev) if want_dh0 else None}
    _call("gdn_linear_bwd", dev, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(h0), _ptr(cu_seqlens), _ptr(dout), _ptr(dhT),
          _ptr(grads["dq"]), _ptr(grads["dk"]), _ptr(grads["dv"]), _ptr(grads["dh0"]), B, T, H, dk, dv,
          _raw_stream(dev, stream), dtype, _ptr(ws), size)
    return grads


_LINEAR = None


def linear_attention(q, k, v, g, h0=None, cu_seqlens=None):
    """(out, hT) of ``linear_fwd`` as a differentiable torch operation:
    gradients for q, k, v and h0 through ``linear_bwd``.  Arguments as for
    ``linear_fwd``.  With packed sequences that leave rows out, those rows'
    outputs and gradients are zero.  To capture a training step into a graph,
    call ``linear_fwd`` and ``linear_bwd`` themselves: autograd's own
    accumulation into leaves that an eager graph still holds waits for
    another stream, which a capture does not survive."""
    global _LINEAR
    if _LINEAR is None:
        import torch

        class _LinearAttention(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, v, g, h0, cu_seqlens):
                out = None if cu_seqlens is None else torch.zeros_like(v)
                out, hT = linear_fwd(q, k, v, g, h0, cu_seqlens, out=out)
                ctx.save_for_backward(q, k, v, g, h0, cu_seqlens)
                return out, hT

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dout, dhT):
                q, k, v, g, h0, cu_seqlens = ctx.saved_tensors
                gr = _backward(q, k, v, g, dout.contiguous(), h0, cu_seqlens, dhT.contiguous(), h0 is not None,
                               None, None, cu_seqlens is not None)
                return gr["dq"], gr["dk"], gr["dv"], None, gr["dh0"], None

        _LINEAR = _LinearAttention
    _decays(g, q.shape[-2])
    return _LINEAR.apply(q, k, v, g, h0, cu_seqlens)
