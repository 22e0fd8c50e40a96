"""The operators together, as a layer uses them: convolution, norms with the
rotation and a recurrence, or convolution and selective scan, for a prompt and
then token by token on pools of states, and for training.

Prompt against tokens: both run on the same bf16 inputs, and what one operator
hands to the next is bf16 in both, rounded from fp32 values that differ by fp32
rounding alone; so a value can land on the next bf16 number, 2^-7 of it away.
Such a step in one of an output's inputs moves the output by 2^-7 of one of its
terms: 2^-6 of the outputs' scale is allowed, after the delta rule's own bf16
products 2e-2 (the library's tolerance for it).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import gated_deltanet_recurrence_delta_amd as gdn  # noqa: E402

pytestmark = pytest.mark.gpu


def rand(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).cuda().to(dtype)


def near(a, b, tol):
    a, b = a.double(), b.double()
    assert a.shape == b.shape and (a - b).abs().max() <= tol * b.abs().max()


def test_a_delta_rule_layer_prompt_then_tokens():
    B, T, more, H, d, W = 3, 90, 4, 4, 64, 4
    bf, D = torch.bfloat16, 3 * 4 * 64
    x, w, bias = rand(1, B, T + more, D, dtype=bf), rand(2, D, W, scale=0.5), rand(3, D, scale=0.1)
    g, beta = -torch.nn.functional.softplus(rand(4, B, T + more, H)), torch.sigmoid(rand(5, B, T + more, H))
    a = torch.arange(T + more)[:, None] * 10000.0 ** (-torch.arange(0, d // 4, 2) / (d // 4))
    cos, sin = torch.cos(a).cuda(), torch.sin(a).cuda()

    def keys(y, pos):
        q, k, v = (t.contiguous() for t in y.reshape(*y.shape[:2], 3, H, d).unbind(2))
        q, k = gdn.qk_norm_fwd(q, k, cos, sin, pos, norm="l2")
        return q, k, v

    pos = torch.arange(T + more, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    y, _ = gdn.conv_fwd(x, w, bias)
    whole, _ = gdn.fwd(*keys(y, pos), g, beta)

    convs, states = gdn.StatePool(8, 1, W - 1, D), gdn.StatePool(8, H, d, d)
    pool = convs.states.to(bf)[:, 0]  # bf16 slots beside the recurrence's fp32 ones
    slots = torch.tensor(states.alloc(B), dtype=torch.int32).cuda()
    y, tail = gdn.conv_fwd(x[:, :T].contiguous(), w, bias)
    first, hT = gdn.fwd(*keys(y, pos[:, :T].contiguous()), g[:, :T].contiguous(), beta[:, :T].contiguous())
    pool[slots.long()], states.states[slots.long()] = tail, hT
    near(first, whole[:, :T], 2e-2)
    for t in range(T, T + more):
        s = slice(t, t + 1)
        y = gdn.conv_fwd_pool(x[:, s].contiguous(), w, pool, slots, bias)
        o = gdn.fwd_recurrent_pool(*keys(y, pos[:, s].contiguous()), g[:, s].contiguous(), beta[:, s].contiguous(),
                                   states.states, slots)
        near(o[:, 0], whole[:, t], 2e-2)


def scan_layer(seed, B, T, D, N, dtype):
    return dict(x=rand(seed, B, T, D, dtype=dtype), w=rand(seed + 1, D, 4, scale=0.5), bias=rand(seed + 2, D, scale=0.1),
                dt=rand(seed + 3, B, T, D, dtype=dtype, scale=0.5), b=rand(seed + 4, B, T, 1, N, dtype=dtype),
                c=rand(seed + 5, B, T, 1, N, dtype=dtype), z=rand(seed + 6, B, T, D, dtype=dtype),
                A_log=torch.log(torch.arange(1, N + 1).float()).expand(D, N).contiguous().cuda(),
                D=rand(seed + 7, D), dt_bias=rand(seed + 8, D) - 4)


def test_a_scan_layer_prompt_then_tokens():
    B, T, more, D, N = 3, 150, 3, 96, 16
    p = scan_layer(20, B, T + more, D, N, torch.bfloat16)
    at = lambda s: {n: p[n][:, s].contiguous() for n in ("dt", "b", "c", "z")}  # noqa: E731
    par = {n: p[n] for n in ("A_log", "D", "dt_bias")}
    y, _ = gdn.conv_fwd(p["x"], p["w"], p["bias"])
    whole, hT = gdn.ssm_fwd(y, **at(slice(None)), **par)
    y, tail = gdn.conv_fwd(p["x"][:, :T].contiguous(), p["w"], p["bias"])
    first, h = gdn.ssm_fwd(y, **at(slice(0, T)), **par)
    near(first, whole[:, :T], 2.0 ** -6)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32).cuda()
    convs, states = torch.zeros(5, 3, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(5, D, N, device="cuda")
    convs[slots.long()], states[slots.long()] = tail, h
    for t in range(T, T + more):
        s = slice(t, t + 1)
        y = gdn.conv_fwd_pool(p["x"][:, s].contiguous(), p["w"], convs, slots, p["bias"])
        o = gdn.ssm_fwd_recurrent_pool(y, pool=states, slots=slots, **at(s), **par)
        near(o[:, 0], whole[:, t], 2.0 ** -6)
    near(states[slots.long()], hT, 2.0 ** -6)
    # a fork of a sequence goes on as the sequence does
    gdn.state_move(states, [4], [1])
    assert torch.equal(states[1], states[4])


def test_a_scan_layer_trains():
    """Gradients of the layer against torch's in 64 bits on the CPU.  fp32 chains of some hundred roundings: 1e-4 of
    each gradient's scale."""
    B, T, D, N = 2, 70, 24, 16
    p = {n: t.requires_grad_() for n, t in scan_layer(40, B, T, D, N, torch.float32).items()}
    dout = rand(50, B, T, D)
    y, _ = gdn.causal_conv(p["x"], p["w"], p["bias"])
    out, _ = gdn.selective_scan(y, p["dt"], p["b"], p["c"], p["A_log"], p["D"], p["z"], p["dt_bias"])
    out.backward(dout)

    r = {n: t.detach().double().cpu().requires_grad_() for n, t in p.items()}
    silu = torch.nn.functional.silu
    line = torch.nn.functional.pad(r["x"], (0, 0, 3, 0))
    y = silu(sum(line[:, i:i + T] * r["w"][:, i] for i in range(4)) + r["bias"])
    s = torch.nn.functional.softplus(r["dt"] + r["dt_bias"])
    h, ys = torch.zeros(B, D, N, dtype=torch.float64), []
    for t in range(T):
        h = torch.exp(s[:, t, :, None] * -torch.exp(r["A_log"])) * h + (s * y)[:, t, :, None] * r["b"][:, t]
        ys.append((h * r["c"][:, t]).sum(-1) + r["D"] * y[:, t])
    want = torch.stack(ys, 1) * silu(r["z"])
    want.backward(dout.double().cpu())
    near(out.detach().cpu(), want.detach(), 1e-4)
    for n in p:
        near(p[n].grad.cpu(), r[n].grad, 1e-4)


def test_a_delta_rule_layer_trains():
    """Gradients through convolution, norm with rotation and the delta rule, fp32, as above."""
    B, T, H, d = 2, 40, 2, 32
    D = 3 * H * d
    p = {"x": rand(60, B, T, D), "w": rand(61, D, 4, scale=0.5), "wq": 1 + rand(62, d, scale=0.1),
         "wk": 1 + rand(63, d, scale=0.1), "g": -torch.nn.functional.softplus(rand(64, B, T, H)),
         "beta": torch.sigmoid(rand(65, B, T, H))}
    a = torch.arange(T)[:, None] * 100.0 ** (-torch.arange(0, 16, 2) / 16)
    cos, sin, dout = torch.cos(a).cuda(), torch.sin(a).cuda(), rand(66, B, T, H, d)
    p = {n: t.requires_grad_() for n, t in p.items()}
    y, _ = gdn.causal_conv(p["x"], p["w"])
    q, k, v = (t.contiguous() for t in y.reshape(B, T, 3, H, d).unbind(2))
    q, k = gdn.qk_norm(q, k, cos, sin, wq=p["wq"], wk=p["wk"], norm="l2")
    out, _ = gdn.gated_delta_rule(q, k, v, p["g"], p["beta"])
    out.backward(dout)

    r = {n: t.detach().double().cpu().requires_grad_() for n, t in p.items()}
    C, S = (t.double().cpu()[:, None] for t in (cos, sin))
    line = torch.nn.functional.pad(r["x"], (0, 0, 3, 0))
    y = torch.nn.functional.silu(sum(line[:, i:i + T] * r["w"][:, i] for i in range(4)))
    q, k, v = y.reshape(B, T, 3, H, d).unbind(2)

    def turned(t, w):
        t = t / torch.sqrt((t * t).sum(-1, keepdim=True) + 1e-6) * w
        u, x = t[..., :8], t[..., 8:16]
        return torch.cat([u * C - x * S, u * S + x * C, t[..., 16:]], -1)

    q, k = turned(q, r["wq"]), turned(k, r["wk"])
    M, os = torch.zeros(B, H, d, d, dtype=torch.float64), []
    for t in range(T):
        M = torch.exp(r["g"][:, t])[..., None, None] * M
        u = r["beta"][:, t, :, None] * (v[:, t] - (k[:, t, :, :, None] * M).sum(-2))
        M = M + k[:, t, :, :, None] * u[..., None, :]
        os.append((q[:, t, :, :, None] * M).sum(-2))
    want = torch.stack(os, 1)
    want.backward(dout.double().cpu())
    near(out.detach().cpu(), want.detach(), 1e-4)
    for n in p:
        near(p[n].grad.cpu(), r[n].grad, 1e-4)


def test_a_captured_training_step_of_a_layer():
    """Forwards and backwards through the entry points themselves, while an eager graph of the same leaves lives."""
    p = {n: t.requires_grad_() for n, t in scan_layer(70, 2, 100, 64, 16, torch.bfloat16).items()}
    y, _ = gdn.causal_conv(p["x"], p["w"], p["bias"])
    eager, _ = gdn.selective_scan(y, p["dt"], p["b"], p["c"], p["A_log"], p["D"], p["z"], p["dt_bias"])
    q = {n: t.detach() for n, t in p.items()}
    dout = rand(80, 2, 100, 64, dtype=torch.bfloat16)

    def step():
        y, _ = gdn.conv_fwd(q["x"], q["w"], q["bias"])
        a = (y, q["dt"], q["b"], q["c"], q["A_log"])
        o = dict(D=q["D"], z=q["z"], dt_bias=q["dt_bias"])
        out, _ = gdn.ssm_fwd(*a, **o)
        g = gdn.ssm_bwd(*a, dout, **o)
        return out, g, gdn.conv_bwd(q["x"], q["w"], g["dx"], q["bias"])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, g, gc = step()
    for i in range(3):
        with torch.no_grad():
            q["x"].mul_(0.75)
        torch.cuda.synchronize()
        graph.replay()
        o, h, hc = step()
        assert torch.equal(o, out) and all(torch.equal(g[n], h[n]) for n in g if g[n] is not None)
        assert all(torch.equal(gc[n], hc[n]) for n in gc)
    assert eager.requires_grad


def test_two_calls_at_once():
    """The operators on two streams side by side give the bits they give alone."""
    def work(seed):
        B, T, D, N, H, d = 2, 700, 192, 16, 3, 64
        p = {k: v.detach() for k, v in scan_layer(seed, B, T, D, N, torch.bfloat16).items()}
        a = torch.arange(T)[:, None] * 100.0 ** (-torch.arange(0, 16, 2) / 16)
        cos, sin = torch.cos(a).cuda(), torch.sin(a).cuda()
        q, k, w = rand(seed + 20, B, T, H, d), rand(seed + 21, B, T, H, d), 1 + rand(seed + 22, d, scale=0.1)
        dout = rand(seed + 23, B, T, D, dtype=torch.bfloat16)
        torch.cuda.synchronize()

        def run():
            y, tail = gdn.conv_fwd(p["x"], p["w"], p["bias"])
            scan = (y, p["dt"], p["b"], p["c"], p["A_log"])
            out, hT = gdn.ssm_fwd(*scan, p["D"], p["z"], p["dt_bias"])
            g = gdn.ssm_bwd(*scan, dout, D=p["D"], z=p["z"], dt_bias=p["dt_bias"], dhT=hT)
            h = gdn.conv_bwd(p["x"], p["w"], g["dx"], p["bias"], dhT=tail)
            n = gdn.qk_norm_bwd(q, k, q, k, cos, sin, wq=w, wk=w)
            return [y, tail, out, hT, *g.values(), *h.values(), *n.values()]
        return run

    runs = [work(70), work(90)]
    alone = [run() for run in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(5):
        got = []
        for run, stream in zip(runs, streams):
            with torch.cuda.stream(stream):
                got.append(run())
        torch.cuda.synchronize()
        for one, other in zip(got, alone):
            assert all(torch.equal(u, v) for u, v in zip(one, other))
