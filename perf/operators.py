"""What the linear-attention and state-pool operators are measured on.

Three kinds of work, as a program that trains and serves linear-attention
layers meets them:

- ``prompt`` / ``train``: linear attention with one fixed decay per head,
  S_t = a S_{t-1} + k_t v_t^T, o_t = S_t^T q_t, a = exp(g_h): a prompt's
  forward pass, or one training step's forward and backward pass;
- ``decode`` / ``decode_delta``: the same rule, or the gated delta rule,
  token by token, on states that live in a pool of slots;
- ``move``: slots of such a pool copied, forked, zeroed or compacted.

``own`` chooses the form of ``run``: elementary torch operations in 32 bits,
or the library's entry points.
"""
import math

import torch

own = False

_BF16, _F32 = "bf16", "f32"


def listed():
    return [
        # a short prompt of a small fp32 model: the call's own latency
        dict(name="prompt short fp32", op="prompt", B=1, T=77, H=2, dk=32, dv=32, dtype=_F32, packed=False, h0=False),
        # the batch that the delta rule's headline workload has, states handed on from earlier tokens
        dict(name="prompt batch", op="prompt", B=4, T=4096, H=16, dk=128, dv=128, dtype=_BF16, packed=False, h0=True),
        # 32 prompts of 256 to 4,096 tokens packed back to back
        dict(name="prompt packed", op="prompt", B=32, T=64711, H=16, dk=128, dv=128, dtype=_BF16, packed=True, h0=False),
        # one long document: few chains, so the sequence itself has to be split
        dict(name="prompt long", op="prompt", B=1, T=32768, H=16, dk=128, dv=128, dtype=_BF16, packed=False, h0=False),
        # a small fp32 training step on ragged packed sequences, key and value heads of different widths
        dict(name="train ragged fp32", op="train", B=7, T=2917, H=5, dk=64, dv=32, dtype=_F32, packed=True, h0=True),
        # a training step of the headline batch
        dict(name="train batch", op="train", B=4, T=4096, H=16, dk=128, dv=128, dtype=_BF16, packed=False, h0=True),
        # one token for each of 128 users whose states are spread over a larger pool
        dict(name="decode batch", op="decode", B=128, T=1, H=16, dk=128, dv=128, dtype=_BF16, slots=160),
        # one user, four drafted tokens checked in one call
        dict(name="decode draft", op="decode", B=1, T=4, H=16, dk=128, dv=128, dtype=_BF16, slots=8),
        # the delta rule's decoding batch
        dict(name="decode delta batch", op="decode_delta", B=128, T=1, H=16, dk=128, dv=128, dtype=_BF16, slots=160),
        # a few users of a small delta-rule model in fp32
        dict(name="decode delta few", op="decode_delta", B=3, T=1, H=8, dk=64, dv=64, dtype=_F32, slots=8),
        # one prompt's state forked to a handful of samples, one layer of small heads
        dict(name="move fork", op="move", kind="fork", L=1, slots=16, H=4, dk=64, dv=64, n=6),
        # the states of half of a batch's users moved to the pool's front, all layers at once
        dict(name="move compact", op="move", kind="compact", L=8, slots=128, H=16, dk=128, dv=128, n=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["prompt", "train", "decode", "decode_delta", "move"])
        dk, dv = rng.choice([32, 64, 128]), rng.choice([32, 64, 128])
        dtype = _F32 if rng.random() < 0.25 else _BF16
        if op in ("prompt", "train"):
            packed = rng.random() < 0.5
            B, T, H = _log_int(rng, 1, 48), _log_int(rng, 1, 32768), rng.randint(1, 24)
            c = dict(op=op, B=B, T=T, H=H, dk=dk, dv=dv, dtype=dtype, packed=packed, h0=rng.random() < 0.5)
        elif op == "move":
            slots = _log_int(rng, 4, 512)
            kind = rng.choice(["fork", "compact", "reorder"])
            c = dict(op=op, kind=kind, L=_log_int(rng, 1, 24), slots=slots, H=rng.randint(1, 24), dk=dk, dv=dv,
                     n=rng.randint(1, max(1, slots // 2)))
        else:
            B = _log_int(rng, 1, 256)
            c = dict(op=op, B=B, T=rng.randint(1, 8) if op == "decode" else 1, H=rng.randint(1, 24), dk=dk, dv=dv,
                     dtype=dtype, slots=B + _log_int(rng, 1, 64))
        pool = c.get("L", 1) * c.get("slots", 0) * c["H"] * dk * dv * 4
        if _cost(c) <= most and pool <= 2 << 30:
            return c


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def work(case):
    c = case
    e = 4 if c.get("dtype") == _F32 else 2
    H, dk, dv = c["H"], c["dk"], c["dv"]
    state = H * dk * dv * 4
    if c["op"] == "move":
        # every slot written once, every distinct source read once
        src, dst = _moves(c, 0)
        return {"bytes": c["L"] * state * (len(dst) + len(set(src))), "flops": 0}
    n = c["T"] if c.get("packed") else c["B"] * c["T"]
    io = n * H * (2 * dk + 2 * dv) * e
    if c["op"] == "prompt":
        return {"bytes": io + c["B"] * state * (2 if c["h0"] else 1) + 4 * H, "flops": 4 * n * H * dk * dv}
    if c["op"] == "train":
        # q, k, v, dout and dhT read; out, hT, dq, dk, dv and dh0 written
        return {"bytes": io + n * H * (2 * dk + 2 * dv) * e + c["B"] * state * (4 if c["h0"] else 2) + 4 * H,
                "flops": 12 * n * H * dk * dv}
    if c["op"] == "decode":
        return {"bytes": io + 2 * c["B"] * state + 4 * H + 4 * c["B"], "flops": 4 * n * H * dk * dv}
    return {"bytes": io + 8 * n * H + 2 * c["B"] * state + 4 * c["B"], "flops": 6 * n * H * dk * dv}


# ------------------------------------------------------------------ inputs --

def _lengths(B, T):
    """B ragged lengths of sum T, the longest some 16 times the shortest."""
    rnd = torch.Generator().manual_seed(1000003 * B + T)
    w = 1 / 16 + torch.rand(B, generator=rnd, dtype=torch.float64) * 15 / 16
    ends = torch.round(torch.cumsum(w, 0) / w.sum() * T).to(torch.int64).tolist()
    ends[-1] = T
    return [b - a for a, b in zip([0] + ends[:-1], ends)]


def _moves(c, seed):
    """The (source, target) slots that a scheduler would ask for."""
    rnd = torch.Generator().manual_seed(int(seed) * 7919 + c["slots"])
    perm = torch.randperm(c["slots"], generator=rnd).tolist()
    n = min(c["n"], c["slots"] - 1)
    if c["kind"] == "fork":  # one parent in up to eight children
        parents = max(1, -(-n // 8))
        n = min(n, c["slots"] - parents)
        return [perm[i % parents] for i in range(n)], perm[parents:parents + n]
    if c["kind"] == "compact":  # n users live; those behind the first n slots move into the holes before them
        live = sorted(perm[:n])
        holes = sorted(set(range(n)) - set(live))
        return [s for s in live if s >= n] or [n], holes or [0]
    # beams: each of n slots takes over the state of one of them, some of several
    slots = perm[:n]
    pick = torch.randint(0, n, (n,), generator=rnd).tolist()
    return [slots[i] for i in pick], slots


def _inputs(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = torch.float32 if c.get("dtype") == _F32 else torch.bfloat16

    def rand(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * scale

    s = {"case": dict(c)}
    H, dk, dv = c["H"], c["dk"], c["dv"]
    if c["op"] == "move":
        s["pool"] = rand(c["L"], c["slots"], H, dk, dv)
        s["src"], s["dst"] = _moves(c, seed)
        s["src_dev"] = torch.tensor(s["src"], device="cuda")
        s["dst_dev"] = torch.tensor(s["dst"], device="cuda")
        return s
    B, T = c["B"], c["T"]
    lead = (T, H) if c.get("packed") else (B, T, H)
    norm = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dt)  # noqa: E731
    s["q"], s["k"] = norm(rand(*lead, dk)), norm(rand(*lead, dk))
    s["v"] = rand(*lead, dv).to(dt)
    # memories of one to a few hundred tokens, another one for each head
    s["g"] = -torch.exp2(-8 * torch.rand(H, generator=gen, device="cuda"))
    if c["op"] in ("decode", "decode_delta"):
        s["pool"] = rand(c["slots"], H, dk, dv, scale=0.3)
        s["slots"] = torch.randperm(c["slots"], generator=gen, device="cuda")[:B].to(torch.int32)
        if c["op"] == "decode_delta":
            s["g"] = -torch.nn.functional.softplus(rand(*lead))
            s["beta"] = torch.sigmoid(rand(*lead))
        return s
    s["h0"] = rand(B, H, dk, dv, scale=0.3) if c["h0"] else None
    s["cu"] = None
    if c["packed"]:
        lens = torch.tensor(_lengths(B, T))
        s["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to("cuda", torch.int32)
        s["longest"] = int(lens.max())
    if c["op"] == "train":
        s["dout"] = rand(*lead, dv).to(dt)
        s["dhT"] = rand(B, H, dk, dv, scale=0.3)
    return s


def prepare(case, seed):
    return _inputs(case, seed)


# -------------------------------------------------------------- plain forms --

_CHUNK = 128


def _powers(g, n):
    """exp(n g) for every head and whole number in n, (H, ...), in 32 bits."""
    n = n.to(torch.float64)
    return torch.exp(g.double().view(-1, *[1] * n.dim()) * n).float()


def _attend(x, y, z, g, reverse):
    """sum_j a^|i-j| (x_i . y_j) z_j over j <= i (j >= i if reverse); fp32, (B, H, T, .)."""
    B, H, T, _ = x.shape
    C = min(_CHUNK, T)
    n = -(-T // C)
    x, y, z = (torch.nn.functional.pad(t, (0, 0, 0, n * C - T)).reshape(B, H, n, C, -1) for t in (x, y, z))
    at = torch.arange(C, device=x.device)
    gap = at[:, None] - at[None, :]
    gap = -gap if reverse else gap
    mask = torch.where(gap >= 0, _powers(g, gap.clamp(min=0)), 0.0)
    out = ((x @ y.transpose(-1, -2)) * mask[None, :, None]) @ z
    # each chunk's sum y z^T, decayed to the chunk's far end (the next output's own step not yet taken)
    w_in = _powers(g, at if reverse else C - 1 - at)[None, :, None, :, None]
    w_out = _powers(g, C - at if reverse else at + 1)[None, :, None, :, None]
    held = ((y * w_in).transpose(-1, -2) @ z).reshape(B, H, n, -1)
    far = torch.arange(n, device=x.device)
    far = far[:, None] - far[None, :] - 1
    far = -far - 2 if reverse else far
    carry = torch.where(far >= 0, _powers(g, C * far.clamp(min=0)), 0.0)
    held = (carry[None] @ held).reshape(B, H, n, x.shape[-1], -1)
    out = out + (x * w_out) @ held
    return out.reshape(B, H, n * C, -1)[:, :, :T]


def _padded(t, cu, longest):
    """(B, H, longest, d) in fp32 of packed rows, zeros behind each sequence; (B, T, H, d) likewise."""
    t = t.float()
    if cu is None:
        return t.transpose(1, 2)
    at = cu[:-1, None].long() + torch.arange(longest, device=t.device)
    inside = at < cu[1:, None]
    return torch.where(inside[..., None, None], t[at.clamp(max=t.shape[0] - 1)], 0.0).transpose(1, 2)


def _unpadded(t, cu, dtype):
    t = t.transpose(1, 2)
    if cu is None:
        return t.to(dtype).contiguous()
    inside = torch.arange(t.shape[1], device=t.device) < (cu[1:] - cu[:-1])[:, None]
    return t[inside].to(dtype)


def _plain_forward(q, k, v, g, h0, cu, longest, dtype):
    """(out, hT) of linear attention, with what the backward pass takes on."""
    q, k, v = (_padded(t, cu, longest) for t in (q, k, v))
    B, H, T, _ = q.shape
    lens = torch.full((B,), T, device=q.device) if cu is None else cu[1:] - cu[:-1]
    at = torch.arange(T, device=q.device)
    out = _attend(q, k, v, g, False)
    left = _powers(g, (lens[:, None] - 1 - at).clamp(min=0)).transpose(0, 1)[..., None]  # padded keys are zero
    hT = (k * left).transpose(-1, -2) @ v
    if h0 is not None:
        out = out + (q * _powers(g, at + 1)[None, ..., None]) @ h0
        hT = hT + _powers(g, lens).transpose(0, 1)[..., None, None] * h0
    return _unpadded(out, cu, dtype), hT, (q, k, v, lens, at, left)


def _plain_backward(kept, g, h0, dout, dhT, cu, longest, dtype):
    q, k, v, lens, at, left = kept
    do = _padded(dout, cu, longest)
    seen = _powers(g, at + 1)[None, ..., None]
    dq = _attend(do, v, k, g, False)
    dk = _attend(v, do, q, g, True) + (v * left) @ dhT.transpose(-1, -2)
    dv = _attend(k, q, do, g, True) + (k * left) @ dhT
    dh0 = None
    if h0 is not None:
        dq = dq + (do * seen) @ h0.transpose(-1, -2)
        dh0 = (q * seen).transpose(-1, -2) @ do + _powers(g, lens).transpose(0, 1)[..., None, None] * dhT
    return (*(_unpadded(t, cu, dtype) for t in (dq, dk, dv)), dh0)


def _plain(s):
    c = s["case"]
    if c["op"] == "move":
        s["pool"][:, s["dst_dev"]] = s["pool"][:, s["src_dev"]]
        return s["pool"]
    q, k, v, g = s["q"], s["k"], s["v"], s["g"]
    if c["op"] == "decode_delta":
        S = s["pool"][s["slots"].long()]
        q1, k1, v1 = (t[:, 0].float() for t in (q, k, v))
        a, b = torch.exp(g[:, 0])[..., None], s["beta"][:, 0][..., None]
        S = a[..., None] * S
        u = b * (v1 - (k1[..., None] * S).sum(-2))
        S = S + k1[..., None] * u[..., None, :]
        s["pool"][s["slots"].long()] = S
        return (q1[..., None] * S).sum(-2)[:, None].to(q.dtype), s["pool"]
    if c["op"] == "decode":
        out, hT, _ = _plain_forward(q, k, v, g, s["pool"][s["slots"].long()], None, 0, q.dtype)
        s["pool"][s["slots"].long()] = hT
        return out, s["pool"]
    out, hT, kept = _plain_forward(q, k, v, g, s["h0"], s["cu"], s.get("longest", 0), q.dtype)
    if c["op"] == "prompt":
        return out, hT
    return out, hT, _plain_backward(kept, g, s["h0"], s["dout"], s["dhT"], s["cu"], s.get("longest", 0), q.dtype)


# -------------------------------------------------------- the library's own --

def _library(s):
    import gated_deltanet_recurrence_delta_amd as gdn

    c = s["case"]
    if c["op"] == "move":
        return gdn.state_move(s["pool"], s["src"], s["dst"], dim=1)
    if c["op"] == "decode":
        return gdn.linear_fwd_recurrent_pool(s["q"], s["k"], s["v"], s["g"], s["pool"], s["slots"]), s["pool"]
    if c["op"] == "decode_delta":
        return gdn.fwd_recurrent_pool(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], s["slots"]), s["pool"]
    out, hT = gdn.linear_fwd(s["q"], s["k"], s["v"], s["g"], s["h0"], s["cu"])
    if c["op"] == "prompt":
        return out, hT
    grads = gdn.linear_bwd(s["q"], s["k"], s["v"], s["g"], s["dout"], s["h0"], s["cu"], dhT=s["dhT"],
                           want_dh0=s["h0"] is not None)
    return out, hT, (grads["dq"], grads["dk"], grads["dv"], grads["dh0"])


def run(state):
    return _library(state) if own else _plain(state)


# --------------------------------------------------------------- definition --

def exact(case, seed):
    """The rules token by token in 64 bits."""
    c, s = case, _inputs(case, seed)
    if c["op"] == "move":
        old, new = s["pool"].clone(), s["pool"].double()
        for a, b in zip(s["src"], s["dst"]):
            new[:, b] = old[:, a].double()
        return new
    H, dk, dv = c["H"], c["dk"], c["dv"]
    if c.get("packed"):
        cu = s["cu"].tolist()
    else:
        cu = [i * c["T"] for i in range(c["B"] + 1)]
    lens = [b - a for a, b in zip(cu, cu[1:])]
    # the flops of the longest sequence's steps over all sequences, at what small 64-bit products reach
    if max(lens) * (2e-4 + c["B"] * H * dk * dv * 2e-11) * (3 if c["op"] == "train" else 1) > 20:
        return None
    flat = lambda t: t.reshape(-1, *t.shape[-2:]).double()  # noqa: E731
    q, k, v = (flat(s[n]) for n in "qkv")
    start = torch.tensor(cu[:-1], device="cuda")
    length = torch.tensor(lens, device="cuda")
    out = torch.zeros_like(v)
    pooled = c["op"] in ("decode", "decode_delta")
    if pooled:
        S = s["pool"].double()[s["slots"].long()]
    else:
        S = torch.zeros(c["B"], H, dk, dv, dtype=torch.float64, device="cuda")
        if s["h0"] is not None:
            S += s["h0"]
    if c["op"] == "train":
        do, dq, dK, dV = flat(s["dout"]), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    a = torch.exp(s["g"].double())
    for t in range(max(lens)):
        on = torch.nonzero(length > t).flatten()
        r, whole = start[on] + t, len(on) == c["B"]
        M = S if whole else S[on]
        if c["op"] == "decode_delta":
            M = M * a.reshape(-1, H)[r][..., None, None]
            u = s["beta"].double().reshape(-1, H)[r][..., None] * (v[r] - (M * k[r][..., None]).sum(-2))
            M = M + k[r][..., None] * u[..., None, :]
        else:
            M = M * a[:, None, None] + k[r][..., None] * v[r][..., None, :]
        out[r] = (q[r][..., None, :] @ M)[..., 0, :]
        if c["op"] == "train":
            dq[r] = (M @ do[r][..., None])[..., 0]
        if whole:
            S = M
        else:
            S[on] = M
    out = out.reshape(s["v"].shape)
    if pooled:
        pool = s["pool"].double()
        pool[s["slots"].long()] = S
        return out, pool
    if c["op"] == "prompt":
        return out, S
    G = s["dhT"].double()
    for t in reversed(range(max(lens))):
        on = torch.nonzero(length > t).flatten()
        r = start[on] + t
        M = G[on] + q[r][..., None] * do[r][..., None, :]
        dK[r] = (M @ v[r][..., None])[..., 0]
        dV[r] = (k[r][..., None, :] @ M)[..., 0, :]
        G[on] = M * a[:, None, None]
    return out, S, (dq.reshape(s["q"].shape), dK.reshape(s["k"].shape), dV.reshape(s["v"].shape),
                    G if s["h0"] is not None else None)
