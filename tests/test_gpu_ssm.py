"""The selective scan on the GPU against the FP64 oracle (tolerances:
block_case.py)."""
import numpy as np
import pytest

from block_case import check_ssm, check_ssm_bwd, f64

torch = pytest.importorskip("torch")
import gated_deltanet_recurrence_delta_amd as gdn  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
OPTIONS = ("D", "z", "dt_bias", "h0")


def make(seed, dtype, lens, D, G, N, packed, without=(), steps=(1e-3, 0.5)):
    r = np.random.default_rng(seed)
    rows, B = sum(lens), len(lens)
    dev = lambda a, t=torch.float32: torch.from_numpy(np.asarray(a, np.float32)).cuda().to(t)  # noqa: E731
    lead = (rows,) if packed else (B, lens[0] if lens else 0)
    step = np.exp(r.uniform(*np.log(steps), D))
    t = {"x": dev(r.standard_normal((*lead, D)), DT[dtype]), "dt": dev(0.7 * r.standard_normal((*lead, D)), DT[dtype]),
         "b": dev(r.standard_normal((*lead, G, N)), DT[dtype]), "c": dev(r.standard_normal((*lead, G, N)), DT[dtype]),
         "A_log": dev(np.log(np.arange(1, N + 1)) + 0.2 * r.standard_normal((D, N))), "D": dev(r.standard_normal(D)),
         "z": dev(r.standard_normal((*lead, D)), DT[dtype]), "dt_bias": dev(np.log(np.expm1(step))),
         "h0": dev(r.standard_normal((B, D, N)))}
    for n in without:
        t[n] = None
    t["cu_seqlens"] = torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32).cuda() if packed else None
    c = {n: f64(t[n]) for n in ("A_log", "D", "dt_bias", "h0")}
    for n in ("x", "dt", "b", "c", "z"):
        c[n] = None if t[n] is None else f64(t[n]).reshape(rows, *((G, N) if n in "bc" else (D,)))
    c["lens"] = lens
    t["dout"], t["dhT"] = dev(r.standard_normal((*lead, D)), DT[dtype]), dev(r.standard_normal((B, D, N)))
    c["dout"], c["dhT"] = f64(t["dout"]).reshape(rows, D), f64(t["dhT"])
    return t, c


def args(t):
    return [t[n] for n in ("x", "dt", "b", "c", "A_log")], {n: t[n] for n in OPTIONS + ("cu_seqlens",)}


def forward(t, **kw):
    a, o = args(t)
    return gdn.ssm_fwd(*a, **{**o, **kw})


def backward(t, dhT=True, **kw):
    a, o = args(t)
    return gdn.ssm_bwd(*a, t["dout"], **o, dhT=t["dhT"] if dhT else None, **kw)


def check_forward(t, c, dtype, soft=True):
    out, hT = forward(t, softplus=soft)
    check_ssm(c, f64(out).reshape(c["x"].shape), f64(hT), dtype, soft)


def check_backward(t, c, dtype, soft=True, dhT=True):
    g = backward(t, softplus=soft, dhT=dhT)
    g = {n: None if v is None else f64(v).reshape(c[n[1:]].shape) if n[1:] in ("x", "dt", "b", "c", "z") else f64(v)
         for n, v in g.items()}
    check_ssm_bwd(c, g, c["dout"], c["dhT"] if dhT else None, dtype, soft)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [16, 32, 64])
@pytest.mark.parametrize("T", [1, 2, 5, 31, 32, 33, 63, 65, 97, 200])
def test_lengths_and_states(dtype, N, T):
    t, c = make(N + T, dtype, [T] * 2, 72, 1, N, False)
    check_forward(t, c, dtype)
    check_backward(t, c, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [16, 32, 64])
@pytest.mark.parametrize("D,G", [(72, 1), (130, 2)])
def test_cut_sequences(dtype, N, D, G):
    """Longer than what runs token by token."""
    for T in (96 + 4 * N + 1, 401):
        assert gdn.gdn_ssm_workspace_size(1, T, D, G, N, 0, 1) > 0
        check_forward(*make(N + T, dtype, [T], D, G, N, False), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,G", [(1, 1), (7, 1), (64, 1), (65, 1), (130, 2), (96, 4), (12, 12), (300, 1), (520, 2)])
@pytest.mark.parametrize("T", [9, 170])
def test_channels_and_groups(dtype, D, G, T):
    t, c = make(D + G, dtype, [T], D, G, 16 if D != 130 else 32, False)
    check_forward(t, c, dtype)
    check_backward(t, c, dtype)


@pytest.mark.parametrize("without", [("D",), ("z",), ("dt_bias",), ("h0",), ("D", "z", "dt_bias", "h0")])
@pytest.mark.parametrize("soft", [True, False])
def test_options(without, soft):
    t, c = make(5, "f32", [175] * 2, 40, 2, 16, False, without)
    if not soft:
        t["dt"].abs_().mul_(0.1)
        c["dt"] = f64(t["dt"]).reshape(c["x"].shape)
        if t["dt_bias"] is not None:
            t["dt_bias"].abs_().mul_(0.01)
            c["dt_bias"] = f64(t["dt_bias"])
    check_forward(t, c, "f32", soft)
    check_backward(t, c, "f32", soft, dhT="h0" not in without)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[5, 1, 0, 33, 64, 2], [0, 0, 70], [100, 3, 0], [1] * 90, [130, 0, 0, 0, 31]])
def test_packed(dtype, lens):
    t, c = make(len(lens), dtype, lens, 48, 2, 16, True)
    check_forward(t, c, dtype)
    check_backward(t, c, dtype)


@pytest.mark.parametrize("N", [32, 64])
def test_packed_wide_states(N):
    t, c = make(N, "bf16", [77, 0, 3, 40], 50, 1, N, True)
    check_forward(t, c, "bf16")
    check_backward(t, c, "bf16")


def test_enough_channels_for_no_cut():
    """2,048 tiles of channels: sequences run as they are, and cut ones agree with them."""
    T, B, D = 170, 2048, 8
    assert gdn.gdn_ssm_workspace_size(B, T, D, 1, 16, 0, 1) == 0
    t, c = make(1, "bf16", [T] * B, D, 1, 16, False)
    out, hT = forward(t)
    for n in (0, 1000, B - 1):
        part = {k: v[n:n + 1] if k in ("x", "dt", "b", "c", "z", "h0") else v for k, v in t.items()}
        one = {k: c[k] for k in ("A_log", "D", "dt_bias")}
        one.update({k: c[k][n * T:(n + 1) * T] for k in ("x", "dt", "b", "c", "z")}, h0=c["h0"][n:n + 1], lens=[T])
        check_ssm(one, f64(out[n]), f64(hT[n:n + 1]), "bf16", True)
        check_forward(part, one, "bf16")


def test_long_memories():
    """Steps so small that a state outlives thousands of tokens, over many segments."""
    t, c = make(2, "f32", [3000], 16, 1, 16, False, steps=(1e-6, 1e-4))
    t["dt"].zero_()
    c["dt"] *= 0
    check_forward(t, c, "f32")
    check_backward(t, c, "f32")


def test_small_steps_keep_their_precision():
    """softplus of large negative arguments: relative, not absolute."""
    t, c = make(3, "f32", [4], 8, 1, 16, False, without=("dt_bias", "h0", "D", "z"))
    for v in (-5.0, -12.0, -30.0, -60.0):
        t["dt"].fill_(v)
        c["dt"][:] = v
        check_forward(t, c, "f32")


def test_steps_so_large_that_nothing_is_left():
    t, c = make(4, "f32", [70], 24, 1, 16, False, without=("dt_bias",))
    t["dt"].fill_(200.0)
    c["dt"][:] = 200.0
    check_forward(t, c, "f32")
    check_backward(t, c, "f32")


@pytest.mark.parametrize("T", [3, 70, 201, 402])
def test_rates_beyond_the_numbers(T):
    """exp(A_log) infinite: nothing is remembered; zero: nothing is forgotten."""
    t, c = make(20, "f32", [T], 20, 1, 16, False)
    t["A_log"][:, 0], t["A_log"][:, 1] = 100.0, -200.0
    c["A_log"][:, 0], c["A_log"][:, 1] = 100.0, -200.0
    check_forward(t, c, "f32")
    g = backward(t)
    ok = torch.ones(16, dtype=torch.bool, device="cuda")
    ok[0] = False
    for n in ("dx", "ddt", "db", "dc", "dD", "dz", "ddt_bias", "dh0"):
        assert g[n].isfinite().all(), n
    assert g["dA_log"][:, ok].isfinite().all() and not g["dA_log"][:, 1].any()


@pytest.mark.parametrize("T", [30, 200])
def test_rows_of_no_sequence_are_left(T):
    t, c = make(6, "bf16", [T], 40, 1, 16, True)
    lo, hi = 3, T - 5
    t["cu_seqlens"] = torch.tensor([lo, lo, hi], dtype=torch.int32).cuda()
    t["h0"], t["dhT"] = t["h0"].repeat(2, 1, 1), t["dhT"].repeat(2, 1, 1)
    out = torch.full_like(t["x"], 77)
    forward(t, out=out)
    assert (out[:lo] == 77).all() and (out[hi:] == 77).all()
    want = backward(t)
    names = ("x", "dt", "b", "c", "A_log") + OPTIONS
    for n in names:
        t[n].requires_grad_()
    a, o = args(t)
    y, hT = gdn.selective_scan(*a, **o)
    assert (y[:lo] == 0).all() and (y[hi:] == 0).all() and torch.equal(y[lo:hi], out[lo:hi])
    grads = torch.autograd.grad([y, hT], [t[n] for n in names], [t["dout"], t["dhT"]])
    for n, g in zip(names, grads):
        if n in ("x", "dt", "b", "c", "z"):
            assert (g[:lo] == 0).all() and (g[hi:] == 0).all() and torch.equal(g[lo:hi], want["d" + n][lo:hi]), n
        else:
            assert torch.equal(g, want["d" + n]), n


def test_groups_of_several_workgroups_leave_rows():
    """db and dc of a group whose channels are several workgroups' (a launch of their own)."""
    t, c = make(7, "bf16", [60], 600, 1, 16, True)
    t["cu_seqlens"] = torch.tensor([10, 50], dtype=torch.int32).cuda()
    fill = torch.full_like(t["b"], 3)
    grads = {}
    a, o = args(t)
    from gated_deltanet_recurrence_delta_amd import ssm
    real, torch_empty = ssm._call, {}

    def call(name, dev, *p):  # fills db and dc before they are written
        for q in torch_empty["k"]:
            q.copy_(fill)
        return real(name, dev, *p)

    like = torch.empty_like

    def empty_like(x, **k):
        y = like(x, **k)
        if x.shape == fill.shape:
            torch_empty.setdefault("k", []).append(y)
        return y

    torch.empty_like, ssm._call = empty_like, call
    try:
        grads = gdn.ssm_bwd(*a, t["dout"], **o)
    finally:
        torch.empty_like, ssm._call = like, real
    for n in ("db", "dc"):
        assert (grads[n][:10] == 3).all() and (grads[n][50:] == 3).all() and (grads[n][10:50] != 3).any()


@pytest.mark.parametrize("T", [20, 300])
def test_in_place_states(T):
    t, _ = make(8, "bf16", [T] * 2, 72, 1, 16, False)
    out, hT = forward(t)
    h = t["h0"].clone()
    o, h2 = forward(t, h0=h, hT=h)
    assert h2 is h and torch.equal(o, out) and torch.equal(h, hT)


def test_split_sequences():
    """A sequence's second part from the first one's state."""
    t, c = make(9, "f32", [150], 32, 1, 16, False)
    a, o = args(t)
    cut = lambda s: ([v[:, s].contiguous() if v.dim() > 2 else v for v in a],  # noqa: E731
                     {**o, "z": o["z"][:, s].contiguous()})
    a1, o1 = cut(slice(0, 80))
    a2, o2 = cut(slice(80, 150))
    out1, h1 = gdn.ssm_fwd(*a1, **o1)
    out2, h2 = gdn.ssm_fwd(*a2, **{**o2, "h0": h1})
    check_ssm(c, f64(torch.cat([out1, out2], 1))[0], f64(h2), "f32", True)


def test_no_tokens():
    t, c = make(10, "f32", [0, 0], 24, 1, 16, True)
    out, hT = forward(t)
    assert torch.equal(hT, t["h0"])
    g = backward(t)
    assert torch.equal(g["dh0"], t["dhT"])
    assert not g["dA_log"].any() and not g["dD"].any() and not g["ddt_bias"].any()
    a, o = args(t)
    g = gdn.ssm_bwd(*a, t["dout"], **{**o, "cu_seqlens": t["cu_seqlens"][:1], "h0": None})
    assert not g["dA_log"].any() and g["dh0"].shape[0] == 0


def test_non_finite_values_stay_with_their_channel():
    t, _ = make(11, "f32", [190], 20, 1, 16, False)
    out, hT = forward(t)
    for n, bad in (("x", float("nan")), ("z", float("inf")), ("dt", float("nan"))):
        u = {**t, n: t[n].clone()}
        u[n][0, 40, 7] = bad
        o, h = forward(u)
        rest = torch.arange(20, device="cuda") != 7
        assert torch.equal(o[..., rest], out[..., rest]) and torch.equal(h[:, rest], hT[:, rest]), n
        assert not torch.equal(o[0, 40:, 7], out[0, 40:, 7])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D,G,N", [(1, 1, 64, 1, 16), (5, 1, 1280, 1, 16), (3, 4, 33, 3, 32), (70, 1, 8, 2, 64),
                                       (2, 90, 40, 1, 16)])
def test_pool(dtype, B, T, D, G, N):
    t, c = make(B, dtype, [T] * B, D, G, N, False)
    r = np.random.default_rng(B)
    pool = torch.from_numpy(r.standard_normal((B + 5, D, N)).astype(np.float32)).cuda()
    slots = torch.from_numpy(r.permutation(B + 5)[:B].astype(np.int32)).cuda()
    before = pool.clone()
    c["h0"] = f64(before[slots.long()])
    a, o = args(t)
    o = {k: o[k] for k in ("D", "z", "dt_bias")}
    out = gdn.ssm_fwd_recurrent_pool(*a, pool, slots, **o)
    check_ssm(c, f64(out).reshape(B * T, D), f64(pool[slots.long()]), dtype, True)
    rest = torch.ones(B + 5, dtype=torch.bool)
    rest[slots.long().cpu()] = False
    assert torch.equal(pool[rest.cuda()], before[rest.cuda()])
    # packed: the same
    other = before.clone()
    cu = torch.arange(0, B * T + 1, T, dtype=torch.int32).cuda()
    flat = lambda v: v.reshape(B * T, *v.shape[2:])  # noqa: E731
    p = gdn.ssm_fwd_recurrent_pool(*[flat(v) for v in a[:4]], a[4], other, slots, D=o["D"], z=flat(o["z"]),
                                   dt_bias=o["dt_bias"], cu_seqlens=cu)
    assert torch.equal(p, flat(out)) and torch.equal(other, pool)


def test_pool_bad_slots():
    t, c = make(12, "bf16", [2] * 5, 64, 1, 16, False)
    pool = torch.randn(6, 64, 16, device="cuda")
    a, o = args(t)
    o = {k: o[k] for k in ("D", "z", "dt_bias")}
    want_pool = pool.clone()
    want = gdn.ssm_fwd_recurrent_pool(*[v[:1] for v in a[:4]], a[4], want_pool, torch.tensor([4], dtype=torch.int32).cuda(),
                                      D=o["D"], z=o["z"][:1], dt_bias=o["dt_bias"])
    bad = torch.tensor([4, -1, 4, 6, 2 ** 31 - 1], dtype=torch.int32).cuda()
    out = gdn.ssm_fwd_recurrent_pool(*a, pool, bad, **o)
    assert torch.equal(out[:1], want) and not out[1:].any() and torch.equal(pool, want_pool)


def test_captured_step_takes_each_replay_s_inputs():
    t, c = make(13, "bf16", [1] * 3, 64, 1, 16, False)
    pool = torch.randn(4, 64, 16, device="cuda")
    slots = torch.tensor([2, 0, 3], dtype=torch.int32).cuda()
    a, o = args(t)
    o = {k: o[k] for k in ("D", "z", "dt_bias")}
    ref_pool, out = pool.clone(), torch.empty_like(t["x"])
    gdn.ssm_fwd_recurrent_pool(*a, pool.clone(), slots, **o, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.ssm_fwd_recurrent_pool(*a, pool, slots, **o, out=out)
    for i in range(4):
        t["x"].copy_(torch.randn(t["x"].shape, generator=torch.Generator().manual_seed(i)).cuda())
        slots.copy_(torch.roll(slots, 1))
        torch.cuda.synchronize()
        graph.replay()
        want = gdn.ssm_fwd_recurrent_pool(*a, ref_pool, slots, **o)
        assert torch.equal(out, want) and torch.equal(pool, ref_pool)


def test_captured_training_step():
    """Forwards and backwards of a packed batch in a graph whose offsets change between replays."""
    t, _ = make(14, "bf16", [70, 50, 80], 64, 1, 16, True)
    offsets = [[0, 70, 120, 200], [0, 0, 199, 200], [0, 100, 101, 200], [0, 200, 200, 200]]
    forward(t), backward(t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, hT = forward(t)
        g = backward(t)
    for o in offsets:
        t["cu_seqlens"].copy_(torch.tensor(o, dtype=torch.int32))
        t["x"].mul_(-1.25)
        torch.cuda.synchronize()
        graph.replay()
        w, wh = forward(t)
        wg = backward(t)
        assert torch.equal(out, w) and torch.equal(hT, wh)
        assert all(torch.equal(g[n], wg[n]) for n in g), o


def test_another_stream():
    t, _ = make(15, "bf16", [150, 9], 64, 1, 16, True)
    want, g = forward(t), backward(t)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    out, hT = forward(t, stream=stream)
    g2 = backward(t, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(hT, want[1])
    assert all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("offsets", [[0, 90, 40, 120], [5, 3, 999, -7], [120, 0, 0, 0], [-5, 400, 400, 400]])
def test_offsets_outside_or_falling_stay_inside_the_tensors(offsets):
    t, _ = make(16, "f32", [120], 64, 1, 16, True)
    t["cu_seqlens"] = torch.tensor(offsets, dtype=torch.int32).cuda()
    t["h0"], t["dhT"] = t["h0"].repeat(3, 1, 1), t["dhT"].repeat(3, 1, 1)
    whole, states = torch.full((3, 120, 64), 7.0, device="cuda"), torch.full((5, 64, 16), 7.0, device="cuda")
    need = gdn.gdn_ssm_workspace_size(3, 120, 64, 1, 16, 1, 0)
    ws = torch.full((3, need), 7, dtype=torch.uint8, device="cuda")
    forward(t, out=whole[1], hT=states[1:4], workspace=ws[1])
    assert (whole[0] == 7).all() and (whole[2] == 7).all() and (states[0] == 7).all() and (states[4] == 7).all()
    assert (ws[0] == 7).all() and (ws[2] == 7).all()
    need = gdn.gdn_ssm_workspace_size(3, 120, 64, 1, 16, 1, 0, 1)
    ws = torch.full((3, need), 7, dtype=torch.uint8, device="cuda")
    backward(t, workspace=ws[1])
    assert (ws[0] == 7).all() and (ws[2] == 7).all()


def test_twice_the_same():
    t, _ = make(17, "f32", [300, 41], 96, 1, 32, True)
    a, b = forward(t), forward(t)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    a, b = backward(t), backward(t)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_state_gradients_in_place():
    """dh0 in dhT's place, few states of many segments: the join's threads share them."""
    t, _ = make(31, "bf16", [1800], 40, 1, 16, False)
    want = backward(t)
    a, o = args(t)
    D, N = 40, 16
    size = gdn.gdn_ssm_workspace_size(1, 1800, D, 1, N, False, gdn.GDN_BF16, True)
    for _ in range(3):
        g = {n: torch.empty_like(want[n]) for n in want}
        g["dh0"] = t["dhT"].clone()
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        ptr = lambda v: 0 if v is None else v.data_ptr()  # noqa: E731
        rc = gdn.gdn_ssm_bwd(*(ptr(v) for v in (*a, o["D"], o["z"], o["dt_bias"], o["h0"], None, t["dout"], g["dh0"])),
                             *(ptr(g[n]) for n in ("dx", "ddt", "db", "dc", "dA_log", "dD", "dz", "ddt_bias", "dh0")),
                             1, 1800, D, 1, N, torch.cuda.current_stream().cuda_stream, gdn.GDN_BF16, 1, ptr(ws), size)
        assert rc == 0
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(g[n], want[n]), n


def test_gradients_that_start_anywhere():
    """A gradient that autograd gives as a part of a larger tensor."""
    t, _ = make(32, "bf16", [3, 4], 7, 1, 16, True)
    want = backward(t)
    a, o = args(t)
    leaves = [v.requires_grad_() for v in (*a, o["D"], o["z"], o["dt_bias"], o["h0"])]
    out, hT = gdn.selective_scan(*leaves, t["cu_seqlens"])
    both = torch.cat([torch.zeros(1, 7, dtype=out.dtype, device="cuda"), out])
    got = torch.autograd.grad([both, hT], leaves, [torch.cat([torch.zeros_like(both[:1]), t["dout"]]), t["dhT"]])
    for v, n in zip(got, ("dx", "ddt", "db", "dc", "dA_log", "dD", "dz", "ddt_bias", "dh0")):
        assert torch.equal(v, want[n]), n


@pytest.mark.parametrize("first,again", [(0, 1), (0, 64), (63, 255), (0, 256), (255, 256), (300, 599), (511, 512)])
def test_pool_slots_named_again_far_behind(first, again):
    """Of two sequences with one slot the first has it, however many lie between."""
    t, _ = make(33, "bf16", [1] * 600, 24, 1, 16, False)
    pool = torch.randn(600, 24, 16, device="cuda")
    slots = torch.randperm(600, device="cuda").int()
    slots[again] = slots[first]
    want_pool, keep = pool.clone(), torch.arange(600, device="cuda") != again
    a, o = args(t)
    o = {k: o[k] for k in ("D", "z", "dt_bias")}
    want = gdn.ssm_fwd_recurrent_pool(*[v[keep] for v in a[:4]], a[4], want_pool, slots[keep], D=o["D"],
                                      z=o["z"][keep], dt_bias=o["dt_bias"])
    out = gdn.ssm_fwd_recurrent_pool(*a, pool, slots, **o)
    assert torch.equal(out[keep], want) and not out[again].any() and torch.equal(pool, want_pool)


@pytest.mark.parametrize("N", [16, 64])
def test_more_states_than_the_caches_hold(N):
    """The same bits for a batch whose states go past the caches as for its halves."""
    D = 130 * 1024 // N
    t, _ = make(34, "bf16", [1] * 72, D, 1, N, False)  # 130 KiB times 4 bytes a sequence
    pool = torch.randn(80, D, N, device="cuda")
    slots = torch.randperm(80, device="cuda")[:72].int()
    halves = pool.clone()
    a, o = args(t)
    o = {k: o[k] for k in ("D", "z", "dt_bias")}
    out = gdn.ssm_fwd_recurrent_pool(*a, pool, slots, **o)
    parts = [gdn.ssm_fwd_recurrent_pool(*[v[s] for v in a[:4]], a[4], halves, slots[s], D=o["D"], z=o["z"][s],
                                        dt_bias=o["dt_bias"]) for s in (slice(0, 36), slice(36, 72))]
    assert torch.equal(out, torch.cat(parts)) and torch.equal(pool, halves)


@pytest.mark.parametrize("N,D", [(16, 300), (32, 150), (64, 75)])
@pytest.mark.parametrize("B", [40, 60, 80, 110, 120])
def test_backward_segments_of_every_length(N, D, B):
    """More sequences take longer segments, of two blocks of tokens up to all there may be."""
    t, c = make(B, "bf16", [50] * B, D, 1, N, False)
    check_backward(t, c, "bf16")


@pytest.mark.parametrize("D", [16, 33])
def test_few_states_of_many_segments(D):
    t, c = make(35, "f32", [6100, 5], D, 1, 16, True)
    check_forward(t, c, "f32")
    check_backward(t, c, "f32")


@pytest.mark.parametrize("N", [16, 32, 64])
@pytest.mark.parametrize("T", [4, 5, 6, 31])
def test_many_sequences_of_few_tokens(N, T):
    """More waves than the device needs: a lane a channel from five tokens on, no cut."""
    assert gdn.gdn_ssm_workspace_size(1100, T, 8, 1, N, 0, 1) == 0
    check_forward(*make(N + T, "bf16", [T] * 1100, 8, 1, N, False), "bf16")


@pytest.mark.parametrize("N", [16, 32, 64])
def test_packed_sequences_cut(N):
    lens = [433, 1, 0, 7, 20, 8, 431]
    assert gdn.gdn_ssm_workspace_size(len(lens), sum(lens), 40, 1, N, 1, 1) > 0
    check_forward(*make(N, "bf16", lens, 40, 1, N, True), "bf16")


@pytest.mark.parametrize("T", [1, 2, 3])
def test_many_sequences_of_one_to_three_tokens(T):
    check_forward(*make(T, "f32", [T] * 1030, 9, 3, 16, False), "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [0, 1, 70, 402])
def test_gradients_of_rates_beyond_the_numbers(dtype, T):
    """A state that keeps nothing has no say in its rate: exp(s A) = 0 makes every term of the gradient zero."""
    t, c = make(36, dtype, [T], 20, 1, 16, True)
    t["A_log"][:, 0], t["A_log"][3, 5], t["A_log"][:, 1] = 100.0, 89.0, float("inf")
    g = backward(t)["dA_log"]
    assert g.isfinite().all()
    assert not g[:, :2].any() and not g[3, 5].any() and g[:3, 2:].any() == (T > 0)


# (groups of one channel: a tile of channels each, so that few channels are many waves)
UNEVEN = [0, 0, 1, 733, 3] + [2] * 40 + [0, 65, 64, 63, 128, 300, 129] + [1] * 40 + [0, 0]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [16, 64])
def test_uneven_packed_sequences(dtype, N):
    """Long sequences among so many that they alone would fill the device: the long ones are cut all the same."""
    D, rows = 48, sum(UNEVEN)
    assert gdn.gdn_ssm_workspace_size(len(UNEVEN), rows, D, D, N, 1, 1) > 0
    t, c = make(N, dtype, UNEVEN, D, D, N, True)
    check_forward(t, c, dtype)
    out, hT = forward(t)
    h = t["h0"].clone()
    o, h2 = forward(t, h0=h, hT=h)
    assert h2 is h and torch.equal(o, out) and torch.equal(h, hT)


def test_uneven_packed_sequences_with_rows_of_none():
    """Rows before the first and behind the last sequence; the same bits without them."""
    D, N, rows, lead, tail = 48, 16, sum(UNEVEN), 70, 90
    t, c = make(37, "bf16", [lead] + UNEVEN[1:-1] + [tail], D, D, N, True)
    t["cu_seqlens"], t["h0"] = t["cu_seqlens"][1:-1].contiguous(), t["h0"][1:-1].contiguous()
    out = torch.full_like(t["x"], 77)
    _, hT = forward(t, out=out)
    assert (out[:lead] == 77).all() and (out[-tail:] == 77).all()
    lens = UNEVEN[1:-1]
    c = {**c, "h0": c["h0"][1:-1], "lens": lens, **{n: c[n][lead:-tail] for n in ("x", "dt", "b", "c", "z")}}
    check_ssm(c, f64(out[lead:-tail]), f64(hT), "bf16", True)


@pytest.mark.parametrize("seed", range(4))
def test_uneven_packed_offsets_that_fall_stay_inside(seed):
    """Any offsets: what lies beside the tensors and the workspace is left."""
    r = np.random.default_rng(seed)
    B, D, N, T = 90, 48, 16, 1500
    t, _ = make(38, "f32", [T], D, D, N, True)
    offsets = r.integers(-50, T + 50, B + 1).astype(np.int32)
    if seed == 0:
        offsets[::2] = np.sort(offsets[::2])
    t["cu_seqlens"], t["h0"] = torch.from_numpy(offsets).cuda(), torch.zeros(B, D, N, device="cuda")
    whole, states = torch.full((3, T, D), 7.0, device="cuda"), torch.full((B + 2, D, N), 7.0, device="cuda")
    need = gdn.gdn_ssm_workspace_size(B, T, D, D, N, 1, 0)
    assert need > 0
    ws = torch.full((3, need), 7, dtype=torch.uint8, device="cuda")
    forward(t, out=whole[1], hT=states[1:B + 1], workspace=ws[1])
    assert (whole[0] == 7).all() and (whole[2] == 7).all() and (states[0] == 7).all() and (states[B + 1] == 7).all()
    assert (ws[0] == 7).all() and (ws[2] == 7).all()


def test_uneven_packed_sequences_captured():
    """A graph takes each replay's offsets: even, uneven, one sequence with everything."""
    B, D, N, T = 90, 48, 16, 1440
    t, _ = make(39, "bf16", [16] * B, D, D, N, True)
    even = np.arange(0, T + 1, 16)
    offsets = [even, np.concatenate([[0] * 45, [T] * 46]), np.concatenate([np.arange(45), T - 45 + np.arange(46)]),
               np.concatenate([[5], np.sort(np.random.default_rng(1).integers(5, T, 89)), [T - 9]])]
    forward(t)
    torch.cuda.synchronize()
    out, hT = torch.zeros_like(t["x"]), torch.zeros_like(t["h0"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward(t, out=out, hT=hT)
    for o in offsets:
        t["cu_seqlens"].copy_(torch.from_numpy(o.astype(np.int32)))
        t["x"].mul_(-1.25)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        w, wh = forward(t, out=torch.zeros_like(out))
        assert torch.equal(out, w) and torch.equal(hT, wh)
