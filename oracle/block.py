"""FP64 oracle of what stands around a recurrence: the causal convolution, the
selective scan, and the norms of queries and keys with the position rotation,
each with its gradients.  Plain NumPy, token by token, one sequence at a time
(lists of sequences for packed batches).

With every result comes a bound's magnitude: the same formula over absolute
values, in which an error of some roundings of 2^-24 each can be expressed.
"""
import numpy as np


def sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


# --------------------------------------------------------------- convolution --

def conv(x, w, bias, h0, silu):
    """(out, hT, y, line) of one sequence: x (T, D), w (D, W), h0 (W - 1, D)."""
    T, W = x.shape[0], w.shape[1]
    line = np.concatenate([np.zeros((W - 1, x.shape[1])) if h0 is None else h0, x])
    y = np.zeros(x.shape) + (0 if bias is None else bias)
    for t in range(T):
        for i in range(W):
            y[t] += w[:, i] * line[t + i]
    return (y * sigmoid(y) if silu else y), line[T:], y, line


def conv_bwd(x, w, bias, h0, silu, dout, dhT):
    """(dx, dw, dbias, dh0) of one sequence, and dy."""
    _, _, y, line = conv(x, w, bias, h0, silu)
    T, W = x.shape[0], w.shape[1]
    s = sigmoid(y)
    dy = dout * (s * (1 + y * (1 - s))) if silu else dout
    dline = np.zeros(line.shape)
    if dhT is not None:
        dline[T:] += dhT
    dw = np.zeros(w.shape)
    for t in range(T):
        for i in range(W):
            dline[t + i] += dy[t] * w[:, i]
            dw[:, i] += dy[t] * line[t + i]
    return dline[W - 1:], dw, dy.sum(0), dline[:W - 1], dy


# ----------------------------------------------------------- selective scan --

def ssm(x, dt, b, c, A_log, D, z, dt_bias, h0, soft):
    """One sequence: x, dt, z (T, D), b, c (T, G, N).  A dict of out, hT and what
    the gradients need; mo and mh are the magnitudes of out and hT: the
    recurrence over absolute values with the square roots of its decays
    (themselves where they grow)."""
    T, Dm = x.shape
    G, N = b.shape[1:]
    wide = lambda k: np.repeat(k, Dm // G, axis=-2)  # noqa: E731
    v = dt + (0 if dt_bias is None else dt_bias)
    s = softplus(v) if soft else v
    A = -np.exp(A_log)
    h = np.zeros((Dm, N)) if h0 is None else h0.copy()
    m = np.abs(h)
    skip = 0 if D is None else D
    gate = np.ones(x.shape) if z is None else z * sigmoid(z)
    y, my = np.zeros(x.shape), np.zeros(x.shape)
    before, mbefore, decay = [], [], []
    for t in range(T):
        a, u = np.exp(s[t][:, None] * A), (s[t] * x[t])[:, None] * wide(b[t])
        before.append(h)
        mbefore.append(m)
        decay.append(a)
        h, m = a * h + u, np.maximum(a, np.sqrt(a)) * m + np.abs(u)
        y[t] = (wide(c[t]) * h).sum(-1) + skip * x[t]
        my[t] = (np.abs(wide(c[t])) * m).sum(-1) + np.abs(skip * x[t])
    return dict(out=y * gate, hT=h, mo=my * np.abs(gate), mh=m, y=y, my=my, s=s, v=v, A=A, before=before,
                mbefore=mbefore, decay=decay, gate=gate)


def ssm_bwd(x, dt, b, c, A_log, D, z, dt_bias, h0, soft, dout, dhT):
    """Gradients of one sequence, as a dict; those of the magnitudes under "m" + name."""
    f = ssm(x, dt, b, c, A_log, D, z, dt_bias, h0, soft)
    T, Dm = x.shape
    G, N = b.shape[1:]
    wide = lambda k: np.repeat(k, Dm // G, axis=-2)  # noqa: E731
    group = lambda k: k.reshape(G, Dm // G, N).sum(1)  # noqa: E731
    l = np.zeros((Dm, N)) if dhT is None else dhT.copy()  # noqa: E741
    m = np.abs(l)
    dy = dout * f["gate"]
    skip = 0 if D is None else D
    g = {}
    for p in ("", "m"):
        g.update({p + "dx": skip * dy if not p else np.abs(skip * dy), p + "ddt": np.zeros(x.shape),
                  p + "db": np.zeros(b.shape), p + "dc": np.zeros(b.shape), p + "dA_log": np.zeros(A_log.shape)})
    for t in reversed(range(T)):
        a, u = f["decay"][t], (f["s"][t] * x[t])[:, None]
        h = a * f["before"][t] + u * wide(b[t])
        ra = np.maximum(a, np.sqrt(a))
        mh = ra * f["mbefore"][t] + np.abs(u * wide(b[t]))
        l, m = l + wide(c[t]) * dy[t][:, None], m + np.abs(wide(c[t]) * dy[t][:, None])  # noqa: E741
        for p, L, H, B, ah, ua, ab in (("", l, h, wide(b[t]), a * f["before"][t], u, f["A"]),
                                       ("m", m, mh, np.abs(wide(b[t])), ra * f["mbefore"][t], np.abs(u),
                                        np.abs(f["A"]))):
            Y = dy[t] if not p else np.abs(dy[t])
            X = x[t] if not p else np.abs(x[t])
            lb = (L * B).sum(-1)
            g[p + "db"][t] = group(L * ua)
            g[p + "dc"][t] = group(H * Y[:, None])
            g[p + "dx"][t] += np.abs(f["s"][t]) * lb if p else f["s"][t] * lb
            g[p + "ddt"][t] = (L * ah * ab).sum(-1) + X * lb
            g[p + "dA_log"] += L * ah * (np.abs(f["s"][t]) if p else f["s"][t])[:, None] * ab
        l, m = a * l, ra * m  # noqa: E741
    for p in ("", "m"):
        if soft:
            g[p + "ddt"] *= sigmoid(f["v"])
        g[p + "ddt_bias"] = g[p + "ddt"].sum(0)
    g["dD"], g["mdD"] = (dy * x).sum(0), np.abs(dy * x).sum(0)
    g["dh0"], g["mdh0"] = l, m
    if z is not None:
        q = sigmoid(z)
        g["dz"] = dout * f["y"] * (q * (1 + z * (1 - q)))
        g["mdz"] = np.abs(dout) * f["my"] * q * (1 + np.abs(z))
    return g


# ---------------------------------------------------------- norm, rotation --

def rotate(y, cos, sin, interleaved, back=False):
    """y (rows, H, d) turned by the angles cos, sin (rows, rot / 2)."""
    half = cos.shape[1]
    y = y.copy()
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    u, v = y[..., a], y[..., b]
    c, s = cos[:, None], (-sin if back else sin)[:, None]
    y[..., a], y[..., b] = u * c - v * s, u * s + v * c
    return y


def _turned_magnitude(y, cos, sin, interleaved):
    """|u c| + |v s| and |u s| + |v c| of y >= 0: each the larger of both signs of sin."""
    c, s = np.abs(cos), np.abs(sin)
    return np.maximum(np.abs(rotate(y, c, s, interleaved)), np.abs(rotate(y, c, -s, interleaved)))


def norm(x, w, cos, sin, pos, l2, eps, interleaved):
    """(y, magnitude) of x (rows, H, d)."""
    m = 1 if l2 else x.shape[-1]
    y = x / np.sqrt((x ** 2).sum(-1, keepdims=True) / m + eps) * (1 if w is None else w)
    if cos is None:
        return y, np.abs(y)
    inside = (pos >= 0) & (pos < len(cos))
    at = np.where(inside, pos, 0)
    out = rotate(y, cos[at], sin[at], interleaved)
    mag = _turned_magnitude(np.abs(y), cos[at], sin[at], interleaved)
    on = inside[:, None, None]
    return np.where(on, out, 0), np.where(on, mag, 0)


def norm_bwd(x, w, cos, sin, pos, l2, eps, interleaved, dy):
    """(dx, dw, magnitudes of both) of x (rows, H, d)."""
    m = 1 if l2 else x.shape[-1]
    r = 1 / np.sqrt((x ** 2).sum(-1, keepdims=True) / m + eps)
    u, g, mg = x * r, dy, np.abs(dy)
    on = np.ones((len(x), 1, 1), bool)
    if cos is not None:
        inside = (pos >= 0) & (pos < len(cos))
        at = np.where(inside, pos, 0)
        on = inside[:, None, None]
        g = rotate(dy, cos[at], sin[at], interleaved, back=True)
        mg = _turned_magnitude(mg, cos[at], sin[at], interleaved)
    g, mg = np.where(on, g, 0), np.where(on, mg, 0)
    wide = 1 if w is None else w
    gw, mgw = g * wide, mg * np.abs(wide)
    dx = r * (gw - u * (gw * u).sum(-1, keepdims=True) / m)
    mdx = r * (mgw + np.abs(u) * (mgw * np.abs(u)).sum(-1, keepdims=True) / m)
    return dx, (g * u).sum((0, 1)), mdx, (mg * np.abs(u)).sum((0, 1))
