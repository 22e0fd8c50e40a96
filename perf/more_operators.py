"""What the operators around the recurrences are measured on.

A recurrent block takes its projections through a short causal convolution,
norms and rotates its keys, and runs a recurrence over them; here are the
three pieces that stand beside the delta rule and linear attention:

- ``conv``: the depthwise causal convolution over 2 to 4 tokens with SiLU,
  for prompts, for training steps and token by token on a pool of states;
- ``ssm``: the selective state space scan with its skip and gate,
  h_t = exp(dt_t A) h_{t-1} + dt_t x_t b_t, y_t = c_t . h_t + D x_t, out_t =
  y_t SiLU(z_t), dt_t = softplus(delta_t + bias), for the same three uses;
- ``norm``: the norm of each head's query and key with the position rotation,
  forwards, and forwards and backwards.

``own`` chooses the form of ``run``: elementary torch operations in 32 bits,
or the library's entry points.
"""
import math

import torch

own = False

_BF16, _F32 = "bf16", "f32"


def listed():
    return [
        # the prompts of a batch of the 1,280-channel layer, whose earlier tokens are known
        dict(name="conv prompt batch", op="conv", kind="prompt", B=8, T=4096, D=1280, W=4, dtype=_BF16, packed=False,
             bias=True, h0=True),
        # a training step of a small fp32 model on ragged packed sequences, an odd number of channels
        dict(name="conv train ragged fp32", op="conv", kind="train", B=9, T=3001, D=333, W=3, dtype=_F32, packed=True,
             bias=True, h0=False),
        # a training step of the layer's batch, no bias
        dict(name="conv train batch", op="conv", kind="train", B=4, T=4096, D=1280, W=4, dtype=_BF16, packed=False,
             bias=False, h0=False),
        # one token for each of 128 users whose states are spread over a larger pool
        dict(name="conv decode batch", op="conv", kind="decode", B=128, T=1, D=1280, W=4, dtype=_BF16, bias=True,
             slots=160),
        # a short prompt of a small fp32 model: the call's own latency
        dict(name="ssm prompt short fp32", op="ssm", kind="prompt", B=1, T=77, D=256, G=1, N=16, dtype=_F32,
             packed=False, gate=True, h0=False),
        # the prompts of a batch of the 1,280-channel layer
        dict(name="ssm prompt batch", op="ssm", kind="prompt", B=8, T=4096, D=1280, G=1, N=16, dtype=_BF16,
             packed=False, gate=True, h0=True),
        # one long document: few chains, so the sequence itself has to be split
        dict(name="ssm prompt long", op="ssm", kind="prompt", B=1, T=32768, D=1280, G=1, N=16, dtype=_BF16,
             packed=False, gate=True, h0=False),
        # a training step on ragged packed sequences, 32 states a channel, keys shared by half of the channels
        dict(name="ssm train ragged", op="ssm", kind="train", B=12, T=5003, D=640, G=2, N=32, dtype=_BF16, packed=True,
             gate=True, h0=False),
        # one token for each of 128 users of the layer
        dict(name="ssm decode batch", op="ssm", kind="decode", B=128, T=1, D=1280, G=1, N=16, dtype=_BF16, gate=True,
             slots=160),
        # the queries and keys of the delta rule's headline batch: unit length, a quarter of each head rotated
        dict(name="norm prompt batch", op="norm", kind="prompt", B=4, T=4096, Hq=16, Hk=16, d=128, rot=32, l2=True,
             weight=False, interleaved=False, dtype=_BF16, far=0),
        # a training step of attention heads with learned norm weights, four queries to a key, whole heads rotated
        dict(name="norm train batch", op="norm", kind="train", B=4, T=4096, Hq=16, Hk=4, d=128, rot=128, l2=False,
             weight=True, interleaved=False, dtype=_BF16, far=0),
        # one token for each of 128 users at far positions, adjacent pairs rotated
        dict(name="norm decode batch", op="norm", kind="prompt", B=128, T=1, Hq=16, Hk=4, d=128, rot=128, l2=False,
             weight=True, interleaved=True, dtype=_BF16, far=131072),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op, kind = rng.choice(["conv", "ssm", "norm"]), rng.choice(["prompt", "train", "decode"])
        dtype = _F32 if rng.random() < 0.25 else _BF16
        if kind == "decode":
            B, T = _log_int(rng, 1, 256), rng.randint(1, 6)
        else:
            B, T = _log_int(rng, 1, 48), _log_int(rng, 1, 32768)
        c = dict(op=op, kind=kind, B=B, T=T, dtype=dtype)
        if op == "norm":
            d = rng.choice([32, 64, 128, 256])
            c |= dict(Hq=rng.randint(1, 32), Hk=rng.randint(1, 16), d=d, rot=rng.choice([0, d // 4, d // 2, d]),
                      l2=rng.random() < 0.5, weight=rng.random() < 0.5, interleaved=rng.random() < 0.5,
                      far=131072 if kind == "decode" else 0)
            c["kind"] = "train" if kind == "train" else "prompt"
        else:
            if kind == "decode":
                c |= dict(slots=B + _log_int(rng, 1, 64))
            else:
                c |= dict(packed=rng.random() < 0.5, h0=rng.random() < 0.5)
            if op == "conv":
                c |= dict(D=_log_int(rng, 16, 8192), W=rng.randint(2, 4), bias=rng.random() < 0.5)
            else:
                G = rng.choice([1, 1, 2, 4])
                c |= dict(D=G * _log_int(rng, 16, 2560 // G), G=G, N=rng.choice([16, 16, 32, 64]),
                          gate=rng.random() < 0.75)
        if _cost(c) <= most:
            return c


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 8)


def _rows(c):
    return c["T"] if c.get("packed") else c["B"] * c["T"]


def work(case):
    c = case
    e = 4 if c["dtype"] == _F32 else 2
    n, B, train = _rows(c), c["B"], c["kind"] == "train"
    if c["op"] == "norm":
        # a rotation's two tables are read at the rows' positions, or once for all sequences
        heads, angles = n * (c["Hq"] + c["Hk"]) * c["d"], (n if c["far"] else c["T"]) * c["rot"] * 4
        weights = 8 * c["d"] if c["weight"] else 0
        if not train:
            return {"bytes": 2 * heads * e + angles + weights + 4 * n, "flops": 6 * heads}
        return {"bytes": 4 * heads * e + angles + 2 * weights + 4 * n, "flops": 18 * heads}
    D = c["D"]
    if c["op"] == "conv":
        W, state = c["W"], B * (c["W"] - 1) * D * e
        weights = 4 * D * (W + (1 if c["bias"] else 0))
        flops = n * D * (2 * W + 4)
        if c["kind"] == "decode":
            return {"bytes": 2 * n * D * e + 2 * state + weights + 4 * B, "flops": flops}
        if not train:
            return {"bytes": 2 * n * D * e + state * (2 if c["h0"] else 1) + weights, "flops": flops}
        return {"bytes": 4 * n * D * e + state * (4 if c["h0"] else 2) + 2 * weights, "flops": 3 * flops}
    G, N, state = c["G"], c["N"], B * D * c["N"] * 4
    rows, keys, weights = n * D * e, 2 * n * G * N * e, 4 * D * (N + 2)
    flops, parts = 7 * n * D * N, 3 + (1 if c["gate"] else 0)  # x, delta, (z) and the output
    if c["kind"] == "decode":
        return {"bytes": parts * rows + keys + 2 * state + weights + 4 * B, "flops": flops}
    if not train:
        return {"bytes": parts * rows + keys + state * (2 if c["h0"] else 1) + weights, "flops": flops}
    # with x, delta, (z), dout and the output their gradients and the keys'
    return {"bytes": 2 * parts * rows + 2 * keys + state * (4 if c["h0"] else 2) + 2 * weights, "flops": 3 * flops}


# ------------------------------------------------------------------ inputs --

def _lengths(B, T):
    """B ragged lengths of sum T, the longest some 16 times the shortest."""
    rnd = torch.Generator().manual_seed(1000003 * B + T)
    w = 1 / 16 + torch.rand(B, generator=rnd, dtype=torch.float64) * 15 / 16
    ends = torch.round(torch.cumsum(w, 0) / w.sum() * T).to(torch.int64).tolist()
    ends[-1] = T
    return [b - a for a, b in zip([0] + ends[:-1], ends)]


def _inputs(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = torch.float32 if c["dtype"] == _F32 else torch.bfloat16

    def rand(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * scale

    s = {"case": dict(c)}
    B, T, train = c["B"], c["T"], c["kind"] == "train"
    lead = (T,) if c.get("packed") else (B, T)
    if c["op"] == "norm":
        d, rot = c["d"], c["rot"]
        # channels of unequal size, as a projection gives them
        size = torch.exp(rand(d, scale=0.5))
        s["q"], s["k"] = ((rand(*lead, h, d) * size).to(dt) for h in (c["Hq"], c["Hk"]))
        s["wq"], s["wk"] = (1 + rand(d, scale=0.2), 1 + rand(d, scale=0.2)) if c["weight"] else (None, None)
        s["cos"] = s["sin"] = s["pos"] = None
        if rot:
            P = c["far"] or T
            at = torch.arange(P, device="cuda", dtype=torch.float64)[:, None]
            angle = at * 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
            s["cos"], s["sin"] = torch.cos(angle).float(), torch.sin(angle).float()
            if c["far"]:
                first = torch.randint(0, P - T, (B, 1), generator=gen, device="cuda")
                s["pos"] = (first + torch.arange(T, device="cuda")).to(torch.int32)
            else:
                s["pos"] = torch.arange(T, device="cuda").expand(B, T).to(torch.int32).contiguous()
        if train:
            s["dqo"], s["dko"] = rand(*lead, c["Hq"], d).to(dt), rand(*lead, c["Hk"], d).to(dt)
        return s
    D = c["D"]
    s["cu"] = None
    if c.get("packed"):
        lens = torch.tensor(_lengths(B, T))
        s["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to("cuda", torch.int32)
        s["longest"] = int(lens.max())
    s["x"] = rand(*lead, D).to(dt)
    if c["op"] == "conv":
        W = c["W"]
        s["w"], s["bias"] = rand(D, W, scale=W ** -0.5), rand(D, scale=0.1) if c["bias"] else None
        state, sdt, scale = (W - 1, D), dt, 1.0
    else:
        G, N = c["G"], c["N"]
        s["b"], s["c"] = rand(*lead, G, N).to(dt), rand(*lead, G, N).to(dt)
        # steps of 0.001 to 0.1 and rates of 1 to N, each channel's own: memories of one to some thousand tokens
        step = torch.exp(math.log(1e-3) + math.log(1e2) * torch.rand(D, generator=gen, device="cuda"))
        s["dt"], s["dt_bias"] = rand(*lead, D, scale=0.5).to(dt), step + torch.log(-torch.expm1(-step))
        s["A_log"] = torch.log(torch.arange(1, N + 1, device="cuda")).expand(D, N) + rand(D, N, scale=0.1)
        s["D"], s["z"] = 1 + rand(D, scale=0.2), rand(*lead, D).to(dt) if c["gate"] else None
        state, sdt, scale = (D, N), torch.float32, 0.3
    if c["kind"] == "decode":
        s["pool"] = rand(c["slots"], *state, scale=scale).to(sdt)
        s["slots"] = torch.randperm(c["slots"], generator=gen, device="cuda")[:B].to(torch.int32)
        return s
    s["h0"] = rand(B, *state, scale=scale).to(sdt) if c["h0"] else None
    if train:
        s["dout"], s["dhT"] = rand(*lead, D).to(dt), rand(B, *state, scale=scale).to(sdt)
    return s


def prepare(case, seed):
    return _inputs(case, seed)


# -------------------------------------------------------------- plain forms --

def _padded(t, s):
    """(B, longest, ...) in fp32 of packed rows, zeros behind each sequence."""
    cu = s.get("cu")
    if cu is None:
        return t.float()
    at = cu[:-1, None].long() + torch.arange(s["longest"], device=t.device)
    inside = (at < cu[1:, None]).reshape(*at.shape, *[1] * (t.dim() - 1))
    return torch.where(inside, t[at.clamp(max=t.shape[0] - 1)].float(), 0.0)


def _rows_of(t, s):
    """The rows of ``_padded`` back in their places."""
    cu = s.get("cu")
    if cu is None:
        return t.to(s["x"].dtype)
    inside = torch.arange(t.shape[1], device=t.device) < (cu[1:] - cu[:-1])[:, None]
    return t[inside].to(s["x"].dtype)


def _inside(x, s):
    """Which rows of the padded batch there are, (B, longest)."""
    at = torch.arange(x.shape[1], device=x.device)
    cu = s.get("cu")
    return at < (cu[1:] - cu[:-1])[:, None] if cu is not None else at.expand(x.shape[0], -1) >= 0


def _plain_conv(s, h0):
    """(out, hT) of the convolution over padded rows, with what the backward pass takes on."""
    w, W = s["w"], s["case"]["W"]
    x = _padded(s["x"], s)
    B, T, D = x.shape
    before = h0.float() if h0 is not None else x.new_zeros(B, W - 1, D)
    xs = torch.cat([before, x], 1)
    y = sum(xs[:, i:i + T] * w[:, i] for i in range(W))
    if s["bias"] is not None:
        y = y + s["bias"]
    sig = 1 / (1 + torch.exp(-y))
    lens = _inside(x, s).sum(1)
    last = (lens[:, None] + torch.arange(W - 1, device=x.device))[..., None].expand(-1, -1, D)
    return _rows_of(y * sig, s), torch.gather(xs, 1, last).to(s["x"].dtype), (xs, y, sig, last)


def _plain_conv_bwd(s, kept):
    xs, y, sig, last = kept
    w, W, T, dt = s["w"], s["case"]["W"], y.shape[1], s["x"].dtype
    dy = _padded(s["dout"], s) * (sig * (1 + y * (1 - sig)))
    dxs = torch.zeros_like(xs).scatter_(1, last, s["dhT"].float())
    dxs = dxs + sum(torch.nn.functional.pad(dy * w[:, i], (0, 0, i, W - 1 - i)) for i in range(W))
    dw = torch.stack([(dy * xs[:, i:i + T]).sum((0, 1)) for i in range(W)], 1)
    return (_rows_of(dxs[:, W - 1:], s), dw, dy.sum((0, 1)) if s["bias"] is not None else None,
            dxs[:, :W - 1].to(dt) if s["h0"] is not None else None)


def _states(a, u):
    """h_t = a_t h_{t-1} + u_t along dimension 1 from a zero state: neighbouring steps are joined, and the half of them solved."""
    T = a.shape[1]
    if T == 1:
        return u
    even, odd, m = a[:, 0::2], a[:, 1::2], T // 2
    half = _states(odd * even[:, :m], u[:, 1::2] + odd * u[:, 0:2 * m:2])
    h = torch.empty_like(u)
    h[:, 1::2] = half
    h[:, 0] = u[:, 0]
    h[:, 2::2] = u[:, 2::2] + even[:, 1:] * half[:, :even.shape[1] - 1]
    return h


def _plain_ssm(s, h0):
    """(out, hT) of the scan, with what the backward pass takes on."""
    x, b, c = (_padded(s[n], s) for n in ("x", "b", "c"))
    D, G, N = s["case"]["D"], s["case"]["G"], s["case"]["N"]
    b, c = (t.repeat_interleave(D // G, 2) if G > 1 else t for t in (b, c))
    v = _padded(s["dt"], s) + s["dt_bias"]
    dt = torch.where(_inside(x, s)[..., None], torch.log1p(torch.exp(-v.abs())) + v.clamp(min=0), 0.0)
    A = -torch.exp(s["A_log"])
    a, u = torch.exp(dt[..., None] * A), (dt * x)[..., None] * b
    if h0 is not None:
        u[:, 0] += a[:, 0] * h0
    h = _states(a, u)
    y = (h * c).sum(-1) + s["D"] * x
    z = _padded(s["z"], s) if s["z"] is not None else None
    out = y if z is None else y * z / (1 + torch.exp(-z))
    return _rows_of(out, s), h[:, -1].clone(), (x, b, c, v, dt, A, a, h, y, z)


def _plain_ssm_bwd(s, kept):
    x, b, c, v, dt, A, a, h, y, z = kept
    B, T, D, G, N = x.shape[0], x.shape[1], s["case"]["D"], s["case"]["G"], s["case"]["N"]
    dout, h0, dz = _padded(s["dout"], s), s["h0"], None
    dy = dout
    if z is not None:
        sig = 1 / (1 + torch.exp(-z))
        dy, dz = dout * z * sig, _rows_of(dout * y * (sig * (1 + z * (1 - sig))), s)
    g = dy[..., None] * c
    g[:, -1] += s["dhT"]
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    g = _states(after.flip(1), g.flip(1)).flip(1)
    before = torch.cat([h0[:, None] if h0 is not None else torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    da = g * a * before
    ddt = (da * A).sum(-1) + (g * b).sum(-1) * x
    ddt = torch.where(_inside(x, s)[..., None], ddt / (1 + torch.exp(-v)), 0.0)
    dx = (g * b).sum(-1) * dt + s["D"] * dy
    db, dc = ((p.reshape(B, T, G, D // G, N)).sum(3) for p in (g * (dt * x)[..., None], dy[..., None] * h))
    return (_rows_of(dx, s), _rows_of(ddt, s), _rows_of(db, s), _rows_of(dc, s),
            (da * dt[..., None]).sum((0, 1)) * A, (dy * x).sum((0, 1)), dz, ddt.sum((0, 1)),
            a[:, 0] * g[:, 0] if h0 is not None else None)


def _turned(x, cos, sin, interleaved):
    """The first rows of x turned by their angles; cos and sin (rows, 1, rot / 2)."""
    half = cos.shape[-1]
    if interleaved:
        u, v = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        return torch.cat([torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2), x[..., 2 * half:]], -1)
    u, v = x[..., :half], x[..., half:2 * half]
    return torch.cat([u * cos - v * sin, u * sin + v * cos, x[..., 2 * half:]], -1)


_EPS = 1e-6


def _plain_norm(s):
    c = s["case"]
    angles = None if s["cos"] is None else [t[s["pos"].long()][..., None, :] for t in (s["cos"], s["sin"])]
    outs, grads = [], []
    for n, w in (("q", s["wq"]), ("k", s["wk"])):
        x = s[n].float()
        r = torch.rsqrt((x * x).sum(-1, keepdim=True) / (1 if c["l2"] else c["d"]) + _EPS)
        unit = x * r
        y = unit if w is None else unit * w
        if angles is not None:
            y = _turned(y, *angles, c["interleaved"])
        outs.append(y.to(s[n].dtype))
        if c["kind"] == "train":
            g = s["d" + n + "o"].float()
            if angles is not None:
                g = _turned(g, angles[0], -angles[1], c["interleaved"])
            gw = g if w is None else g * w
            dot = (gw * unit).sum(-1, keepdim=True) / (1 if c["l2"] else c["d"])
            grads += [(r * (gw - unit * dot)).to(s[n].dtype), None if w is None else (g * unit).sum((0, 1, 2))]
    return (*outs, *grads)


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        return _plain_norm(s)
    forward, backward = (_plain_conv, _plain_conv_bwd) if c["op"] == "conv" else (_plain_ssm, _plain_ssm_bwd)
    if c["kind"] == "decode":
        slots = s["slots"].long()
        out, hT, _ = forward(s, s["pool"][slots])
        s["pool"][slots] = hT
        return out, s["pool"]
    out, hT, kept = forward(s, s["h0"])
    return (out, hT) if c["kind"] == "prompt" else (out, hT, *backward(s, kept))


# -------------------------------------------------------- the library's own --

def _library(s):
    import gated_deltanet_recurrence_delta_amd as gdn

    c = s["case"]
    if c["op"] == "norm":
        how = dict(cos=s["cos"], sin=s["sin"], pos=s["pos"], wq=s["wq"], wk=s["wk"], norm="l2" if c["l2"] else "rms",
                   eps=_EPS, interleaved=c["interleaved"])
        outs = gdn.qk_norm_fwd(s["q"], s["k"], **how)
        if c["kind"] == "prompt":
            return outs
        g = gdn.qk_norm_bwd(s["q"], s["k"], s["dqo"], s["dko"], **how)
        return (*outs, g["dq"], g["dwq"], g["dk"], g["dwk"])
    if c["op"] == "conv":
        if c["kind"] == "decode":
            return gdn.conv_fwd_pool(s["x"], s["w"], s["pool"], s["slots"], bias=s["bias"]), s["pool"]
        outs = gdn.conv_fwd(s["x"], s["w"], bias=s["bias"], h0=s["h0"], cu_seqlens=s["cu"])
        if c["kind"] == "prompt":
            return outs
        g = gdn.conv_bwd(s["x"], s["w"], s["dout"], bias=s["bias"], h0=s["h0"], cu_seqlens=s["cu"], dhT=s["dhT"],
                         want_dh0=s["h0"] is not None)
        return (*outs, g["dx"], g["dw"], g["dbias"], g["dh0"])
    args, more = (s["x"], s["dt"], s["b"], s["c"], s["A_log"]), dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    if c["kind"] == "decode":
        return gdn.ssm_fwd_recurrent_pool(*args, s["pool"], s["slots"], **more), s["pool"]
    outs = gdn.ssm_fwd(*args, **more, h0=s["h0"], cu_seqlens=s["cu"])
    if c["kind"] == "prompt":
        return outs
    g = gdn.ssm_bwd(*args, s["dout"], **more, h0=s["h0"], cu_seqlens=s["cu"], dhT=s["dhT"],
                    want_dh0=s["h0"] is not None)
    return (*outs, g["dx"], g["ddt"], g["db"], g["dc"], g["dA_log"], g["dD"], g["dz"], g["ddt_bias"], g["dh0"])


def run(state):
    return _library(state) if own else _plain(state)


# --------------------------------------------------------------- definition --

def _spans(c, s):
    if c.get("packed"):
        cu = s["cu"].tolist()
        return list(zip(cu, cu[1:]))
    return [(i * c["T"], (i + 1) * c["T"]) for i in range(c["B"])]


def _exact_conv(c, s):
    W, D, dt = c["W"], c["D"], torch.float64
    x, w = s["x"].reshape(-1, D).to(dt), s["w"].to(dt)
    starts = s["pool"][s["slots"].long()] if c["kind"] == "decode" else s["h0"]
    out, dx = torch.zeros_like(x), torch.zeros_like(x)
    ends, dh0, dw, db = [], [], torch.zeros_like(w), torch.zeros(D, dtype=dt, device=x.device)
    for i, (lo, hi) in enumerate(_spans(c, s)):
        pre = torch.zeros(W - 1, D, dtype=dt, device=x.device) if starts is None else starts[i].to(dt)
        line = torch.cat([pre, x[lo:hi]])
        taps = torch.stack([line[j:j + hi - lo] for j in range(W)], -1)  # (rows, D, W)
        y = (taps * w).sum(-1)
        if s["bias"] is not None:
            y = y + s["bias"].to(dt)
        out[lo:hi] = y * torch.sigmoid(y)
        ends.append(line[hi - lo:])
        if c["kind"] == "train":
            p = torch.sigmoid(y)
            dy = s["dout"].reshape(-1, D)[lo:hi].to(dt) * (p + y * p * (1 - p))
            dline = torch.zeros_like(line)
            dline[hi - lo:] = s["dhT"][i].to(dt)
            for j in range(W):
                dline[j:j + hi - lo] += dy * w[:, j]
            dw += (taps * dy[..., None]).sum(0)
            db += dy.sum(0)
            dx[lo:hi] = dline[W - 1:]
            dh0.append(dline[:W - 1])
    out, hT = out.reshape(s["x"].shape), torch.stack(ends)
    if c["kind"] == "decode":
        pool = s["pool"].to(dt)
        pool[s["slots"].long()] = hT
        return out, pool
    if c["kind"] == "prompt":
        return out, hT
    return (out, hT, dx.reshape(s["x"].shape), dw, db if s["bias"] is not None else None,
            torch.stack(dh0) if s["h0"] is not None else None)


def _exact_ssm(c, s):
    """The recurrence token by token, and its gradients in the same steps backwards."""
    D, G, N, train = c["D"], c["G"], c["N"], c["kind"] == "train"
    spans = _spans(c, s)
    longest = max(hi - lo for lo, hi in spans)
    if longest * (1e-3 if train else 4e-4) * (1 + c["B"] * D * N / 1e6) > 20 or \
            train and longest * c["B"] * D * N * 8 > 60e9:
        return None
    flat = lambda t, k: t.reshape(-1, *t.shape[-k:]).double()  # noqa: E731
    x, b, cc = flat(s["x"], 1), flat(s["b"], 2), flat(s["c"], 2)
    pre = flat(s["dt"], 1) + s["dt_bias"].double()
    dt = torch.nn.functional.softplus(pre, threshold=40)
    A = -torch.exp(s["A_log"].double())
    z = flat(s["z"], 1) if s["z"] is not None else None
    gate = torch.ones_like(x) if z is None else z * torch.sigmoid(z)
    wide = lambda t: t.repeat_interleave(D // G, -2)  # noqa: E731
    first = s["pool"][s["slots"].long()] if c["kind"] == "decode" else s["h0"]
    h = torch.zeros(c["B"], D, N, dtype=torch.float64, device=x.device) if first is None else first.double()
    begin = torch.tensor([lo for lo, _ in spans], device=x.device)
    count = torch.tensor([hi - lo for lo, hi in spans], device=x.device)
    y, held, skip = torch.zeros_like(x), [], s["D"].double()
    for t in range(longest):
        on = torch.nonzero(count > t).flatten()
        r = begin[on] + t
        if train:
            held.append(h[on])
        step = torch.exp(dt[r][..., None] * A) * h[on] + (dt[r] * x[r])[..., None] * wide(b[r])
        y[r] = (step * wide(cc[r])).sum(-1) + skip * x[r]
        h = h.clone() if len(on) < c["B"] else h
        h[on] = step
    out = (y * gate).reshape(s["x"].shape)
    if c["kind"] == "decode":
        pool = s["pool"].double()
        pool[s["slots"].long()] = h
        return out, pool
    if not train:
        return out, h
    dout, lam = flat(s["dout"], 1), s["dhT"].double()
    dy = dout * gate
    dx, ddt, db, dc, dA = skip * dy, torch.zeros_like(x), torch.zeros_like(b), torch.zeros_like(cc), torch.zeros_like(A)
    for t in reversed(range(longest)):
        on = torch.nonzero(count > t).flatten()
        r = begin[on] + t
        a, was, B1, C1 = torch.exp(dt[r][..., None] * A), held.pop(), wide(b[r]), wide(cc[r])
        now = a * was + (dt[r] * x[r])[..., None] * B1
        l = lam[on] + dy[r][..., None] * C1  # noqa: E741
        dc[r] = (now * dy[r][..., None]).reshape(-1, G, D // G, N).sum(2)
        db[r] = (l * (dt[r] * x[r])[..., None]).reshape(-1, G, D // G, N).sum(2)
        lb, moved = (l * B1).sum(-1), l * a * was
        dx[r] += lb * dt[r]
        ddt[r] = (moved * A).sum(-1) + lb * x[r]
        dA += (moved * dt[r][..., None]).sum(0)
        lam[on] = l * a
    ddt = ddt * torch.sigmoid(pre)
    like = lambda t, n: t.reshape(s[n].shape)  # noqa: E731
    dz = None
    if z is not None:
        p = torch.sigmoid(z)
        dz = like(dout * y * (p + z * p * (1 - p)), "z")
    return (out, h, like(dx, "x"), like(ddt, "dt"), like(db, "b"), like(dc, "c"), dA * A, (dy * x).sum(0), dz,
            ddt.sum(0), lam if s["h0"] is not None else None)


def _exact_norm(c, s):
    d, outs, grads = c["d"], [], []
    turn = None
    if s["cos"] is not None:
        # each pair as a complex number, turned by cos + i sin
        turn = torch.complex(s["cos"].double(), s["sin"].double())[s["pos"].long()][..., None, :]
    half = c["rot"] // 2

    def turned(t, by):
        t = t.clone()
        at = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if c["interleaved"] else (slice(0, half), slice(half, 2 * half))
        p = torch.complex(t[..., at[0]].contiguous(), t[..., at[1]].contiguous()) * by
        t[..., at[0]], t[..., at[1]] = p.real, p.imag
        return t

    for n in "qk":
        x, w = s[n].double(), s["w" + n]
        w = torch.ones(d, dtype=torch.float64, device=x.device) if w is None else w.double()
        size = torch.sqrt((x ** 2).sum(-1, keepdim=True) / (1 if c["l2"] else d) + _EPS)
        y = x / size * w
        outs.append(y if turn is None else turned(y, turn))
        if c["kind"] == "train":
            g = s["d" + n + "o"].double()
            g = g if turn is None else turned(g, turn.conj())
            p = (g * w * x).sum(-1, keepdim=True) / (1 if c["l2"] else d)
            grads += [g * w / size - x * p / size ** 3, (g * x / size).sum((0, 1, 2)) if c["weight"] else None]
    return (*outs, *grads)


def exact(case, seed):
    """The operators' definitions in 64 bits."""
    s = _inputs(case, seed)
    return {"conv": _exact_conv, "ssm": _exact_ssm, "norm": _exact_norm}[case["op"]](case, s)
