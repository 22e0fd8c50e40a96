"""The causal convolution on the GPU against the FP64 oracle (tolerances:
block_case.py)."""
import numpy as np
import pytest

from block_case import check_conv, check_conv_bwd, f64, spans, within

torch = pytest.importorskip("torch")
import gated_deltanet_recurrence_delta_amd as gdn  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(seed, dtype, lens, D, W, packed, bias=True, h0=True):
    """Device tensors and their float64 values (rows flat) of sequences of these lengths."""
    r = np.random.default_rng(seed)
    rows, B = sum(lens), len(lens)
    dev = lambda a, t: torch.from_numpy(np.asarray(a, np.float32)).cuda().to(t)  # noqa: E731
    lead = (rows,) if packed else (B, lens[0] if lens else 0)
    t = {"x": dev(r.standard_normal((*lead, D)), DT[dtype]), "w": dev(r.standard_normal((D, W)), torch.float32),
         "bias": dev(r.standard_normal(D), torch.float32) if bias else None,
         "h0": dev(r.standard_normal((B, W - 1, D)), DT[dtype]) if h0 else None,
         "cu_seqlens": torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32).cuda() if packed else None}
    t["dout"] = dev(r.standard_normal((*lead, D)), DT[dtype])
    t["dhT"] = dev(r.standard_normal((B, W - 1, D)), DT[dtype])
    c = {n: f64(t[n]) for n in ("w", "bias", "h0")}
    c["x"], c["dout"], c["dhT"] = f64(t["x"]).reshape(rows, D), f64(t["dout"]).reshape(rows, D), f64(t["dhT"])
    c["lens"] = lens
    return t, c


def forward(t, **kw):
    return gdn.conv_fwd(t["x"], t["w"], t["bias"], t["h0"], t["cu_seqlens"], **kw)


def backward(t, dhT=True, **kw):
    return gdn.conv_bwd(t["x"], t["w"], t["dout"], t["bias"], t["h0"], t["cu_seqlens"],
                        dhT=t["dhT"] if dhT else None, **kw)


def both(t, c, dtype, silu=True, dhT=True):
    D = t["x"].shape[-1]
    out, hT = forward(t, silu=silu)
    check_conv(c, f64(out).reshape(-1, D), f64(hT), dtype, silu)
    g = {n: f64(v) for n, v in backward(t, dhT=dhT, silu=silu).items()}
    g["dx"] = g["dx"].reshape(-1, D)
    check_conv_bwd(c, g, c["dout"], c["dhT"] if dhT else None, dtype, silu)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 16, 17, 33, 70])
def test_lengths_and_widths(dtype, W, T):
    both(*make(W * 100 + T, dtype, [T] * 2, 72, W, False), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 7, 8, 12, 63, 64, 65, 130, 193, 257, 300, 512, 520, 577])
def test_channels(dtype, D):
    both(*make(D, dtype, [19] * 2, D, 4, False), dtype)


@pytest.mark.parametrize("bias,h0,silu,dhT", [(False, False, True, False), (True, False, False, True),
                                              (False, True, False, False)])
def test_options(bias, h0, silu, dhT):
    both(*make(3, "bf16", [40] * 2, 64, 4, False, bias, h0), "bf16", silu, dhT)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[5, 1, 0, 33, 2], [0, 0, 7], [64, 3, 0], [1] * 80, [0], [130, 0, 0, 0, 17]])
def test_packed(dtype, lens):
    both(*make(len(lens), dtype, lens, 40, 4, True), dtype)


def test_long_and_many_sequences():
    both(*make(5, "bf16", [700, 90] + [3] * 130, 24, 3, True), "bf16")


def test_a_sequence_does_not_depend_on_its_batch():
    """Bit for bit: alone, in a dense batch, in a packed one."""
    t, _ = make(6, "bf16", [37] * 3, 64, 4, False)
    out, hT = forward(t)
    for n in range(3):
        o, h = gdn.conv_fwd(t["x"][n:n + 1], t["w"], t["bias"], t["h0"][n:n + 1])
        assert torch.equal(o[0], out[n]) and torch.equal(h[0], hT[n])
    cu = torch.tensor([0, 37, 74, 111], dtype=torch.int32).cuda()
    o, h = gdn.conv_fwd(t["x"].reshape(111, 64), t["w"], t["bias"], t["h0"], cu)
    assert torch.equal(o, out.reshape(111, 64)) and torch.equal(h, hT)
    # a sequence in two parts
    o1, h1 = gdn.conv_fwd(t["x"][:, :5].contiguous(), t["w"], t["bias"], t["h0"])
    o2, h2 = gdn.conv_fwd(t["x"][:, 5:].contiguous(), t["w"], t["bias"], h1)
    assert torch.equal(torch.cat([o1, o2], 1), out) and torch.equal(h2, hT)


def test_rows_of_no_sequence_are_left():
    t, c = make(7, "f32", [10], 16, 4, True)
    t["cu_seqlens"] = torch.tensor([2, 2, 7], dtype=torch.int32).cuda()
    t["h0"], t["dhT"] = t["h0"].repeat(2, 1, 1), t["dhT"].repeat(2, 1, 1)
    out = torch.full_like(t["x"], 77)
    gdn.conv_fwd(t["x"], t["w"], t["bias"], t["h0"], t["cu_seqlens"], out=out)
    assert (out[:2] == 77).all() and (out[7:] == 77).all() and (out[2:7] != 77).all()
    for n in ("x", "w", "bias", "h0"):
        t[n].requires_grad_()
    o, _ = gdn.causal_conv(t["x"], t["w"], t["bias"], t["h0"], t["cu_seqlens"])
    assert (o[:2] == 0).all() and (o[7:] == 0).all() and torch.equal(o[2:7], out[2:7])
    o.sum().backward()
    assert (t["x"].grad[:2] == 0).all() and (t["x"].grad[7:] == 0).all() and (t["x"].grad[2:7] != 0).any()


def test_in_place_state():
    for T in (2, 100):
        t, _ = make(8, "bf16", [T] * 2, 64, 4, False)
        out, hT = forward(t)
        h = t["h0"].clone()
        o, h2 = gdn.conv_fwd(t["x"], t["w"], t["bias"], h, hT=h)
        assert h2 is h and torch.equal(h, hT) and torch.equal(o, out)


def test_operation():
    """causal_conv's gradients are conv_bwd's."""
    t, _ = make(9, "bf16", [21, 4], 32, 4, True)
    want = backward(t)
    leaves = [t[n].requires_grad_() for n in ("x", "w", "bias", "h0")]
    out, hT = gdn.causal_conv(*leaves, t["cu_seqlens"])
    got = torch.autograd.grad([out, hT], leaves, [t["dout"], t["dhT"]])
    for a, n in zip(got, ("dx", "dw", "dbias", "dh0")):
        assert torch.equal(a, want[n]), n


def test_no_tokens():
    t, c = make(10, "f32", [0, 0], 16, 3, True)
    out, hT = forward(t)
    assert torch.equal(hT, t["h0"])
    g = backward(t)
    assert torch.equal(g["dh0"], t["dhT"]) and not g["dw"].any() and not g["dbias"].any()
    g = gdn.conv_bwd(t["x"], t["w"], t["dout"], t["bias"], None, t["cu_seqlens"][:1])
    assert not g["dw"].any() and not g["dbias"].any()


def test_non_finite_tokens_stay_with_their_taps():
    t, _ = make(11, "f32", [30], 16, 4, False)
    out, _ = forward(t)
    for bad in (float("nan"), float("inf")):
        x = t["x"].clone()
        x[0, 11, 5] = bad
        o, _ = gdn.conv_fwd(x, t["w"], t["bias"], t["h0"])
        hit = torch.zeros_like(o, dtype=torch.bool)
        hit[0, 11:15, 5] = True
        assert torch.equal(o[~hit], out[~hit])
        assert not torch.equal(o[hit], out[hit])


def pool_case(seed, dtype, B, T, D, W, nslots):
    t, c = make(seed, dtype, [T] * B, D, W, False, h0=False)
    r = np.random.default_rng(seed)
    pool = torch.from_numpy(r.standard_normal((nslots, W - 1, D)).astype(np.float32)).cuda().to(DT[dtype])
    slots = torch.from_numpy(r.permutation(nslots)[:B].astype(np.int32)).cuda()
    return t, c, pool, slots


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D,W", [(1, 1, 64, 4), (5, 1, 1280, 4), (3, 4, 33, 3), (130, 1, 8, 2), (2, 30, 16, 4)])
def test_pool(dtype, B, T, D, W):
    t, c, pool, slots = pool_case(B, dtype, B, T, D, W, B + 5)
    before = pool.clone()
    c["h0"] = f64(before[slots.long()])
    out = gdn.conv_fwd_pool(t["x"], t["w"], pool, slots, t["bias"])
    check_conv(c, f64(out).reshape(B * T, D), f64(pool[slots.long()]), dtype, True)
    rest = torch.ones(B + 5, dtype=torch.bool)
    rest[slots.long().cpu()] = False
    assert torch.equal(pool[rest.cuda()], before[rest.cuda()])


def test_pool_bad_slots():
    """Outside the pool, and named twice: zeros, and no state changes."""
    t, c, pool, slots = pool_case(3, "bf16", 5, 2, 64, 4, 6)
    want_pool, want = pool.clone(), None
    want = gdn.conv_fwd_pool(t["x"][:1], t["w"], want_pool, slots[:1], t["bias"])
    bad = torch.tensor([slots[0].item(), -1, slots[0].item(), 6, 2 ** 31 - 1], dtype=torch.int32).cuda()
    out = gdn.conv_fwd_pool(t["x"], t["w"], pool, bad, t["bias"])
    assert torch.equal(out[:1], want) and not out[1:].any() and torch.equal(pool, want_pool)


def test_pool_packed_equals_dense():
    t, c, pool, slots = pool_case(4, "f32", 4, 3, 20, 4, 4)
    other = pool.clone()
    out = gdn.conv_fwd_pool(t["x"], t["w"], pool, slots, t["bias"])
    cu = torch.tensor([0, 3, 6, 9, 12], dtype=torch.int32).cuda()
    o = gdn.conv_fwd_pool(t["x"].reshape(12, 20), t["w"], other, slots, t["bias"], cu_seqlens=cu)
    assert torch.equal(o, out.reshape(12, 20)) and torch.equal(other, pool)


def test_captured_step_takes_each_replay_s_inputs():
    t, c, pool, slots = pool_case(5, "bf16", 3, 1, 64, 4, 4)
    ref_pool = pool.clone()
    out = torch.empty_like(t["x"])
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        gdn.conv_fwd_pool(t["x"], t["w"], pool.clone(), slots, t["bias"], out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.conv_fwd_pool(t["x"], t["w"], pool, slots, t["bias"], out=out)
    for i in range(4):
        t["x"].copy_(torch.randn(t["x"].shape, generator=torch.Generator().manual_seed(i)).cuda())
        slots.copy_(torch.roll(slots, 1))
        torch.cuda.synchronize()
        graph.replay()
        want = gdn.conv_fwd_pool(t["x"], t["w"], ref_pool, slots, t["bias"])
        assert torch.equal(out, want) and torch.equal(pool, ref_pool)


def test_another_stream():
    t, _ = make(12, "bf16", [50, 9], 64, 4, True)
    want, g = forward(t), backward(t)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    out, hT = forward(t, stream=stream)
    g2 = backward(t, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(hT, want[1])
    assert all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("offsets", [[0, 9, 4, 12], [5, 3, 99, -7], [12, 0, 0, 0], [-5, 40, 40, 40]])
def test_offsets_outside_or_falling_stay_inside_the_tensors(offsets):
    """What lies beside the tensors is left, whatever the offsets say."""
    D, W, n = 32, 4, 12
    whole = torch.full((3, n, D), 7.0, device="cuda")
    cu = torch.tensor(offsets, dtype=torch.int32).cuda()
    w = torch.randn(D, W, device="cuda")
    hT = torch.full((5, W - 1, D), 7.0, device="cuda")
    x = torch.randn(n, D, device="cuda")
    gdn.conv_fwd(x, w, None, None, cu, out=whole[1], hT=hT[1:4])
    assert (whole[0] == 7).all() and (whole[2] == 7).all() and (hT[0] == 7).all() and (hT[4] == 7).all()
    pool = torch.full((5, W - 1, D), 7.0, device="cuda")
    slots = torch.tensor([1, 0, 2], dtype=torch.int32).cuda()
    gdn.conv_fwd_pool(x, w, pool[1:4], slots, cu_seqlens=cu, out=whole[1])
    assert (whole[0] == 7).all() and (whole[2] == 7).all() and (pool[0] == 7).all() and (pool[4] == 7).all()
    gdn.conv_bwd(x, w, x, None, None, cu)
    torch.cuda.synchronize()


def test_twice_the_same():
    t, _ = make(13, "f32", [300, 41], 96, 4, True)
    a, b = forward(t), forward(t)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    a, b = backward(t), backward(t)
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("packed", [False, True])
def test_in_place_states_of_cut_sequences(packed):
    """hT in h0's place where the first segment reads what another one would write."""
    for dtype, W in (("bf16", 4), ("f32", 2)):
        t, _ = make(21, dtype, [700, 700, 1, 2, 0, 3] if packed else [700] * 3, 520, W, packed)
        out, hT = forward(t)
        for _ in range(3):
            h = t["h0"].clone()
            o, h2 = gdn.conv_fwd(t["x"], t["w"], t["bias"], h, t["cu_seqlens"], hT=h)
            assert h2 is h and torch.equal(h, hT) and torch.equal(o, out)


def test_gradients_that_start_anywhere():
    """A gradient that autograd gives as a part of a larger tensor."""
    t, _ = make(22, "bf16", [3, 4], 7, 3, True)
    want = backward(t)
    leaves = [t[n].requires_grad_() for n in ("x", "w", "bias", "h0")]
    out, hT = gdn.causal_conv(*leaves, t["cu_seqlens"])
    both = torch.cat([torch.zeros(1, 7, dtype=out.dtype, device="cuda"), out])
    states = torch.cat([torch.zeros(1, 2, 7, dtype=out.dtype, device="cuda"), hT])
    first = torch.zeros_like(both[:1])
    got = torch.autograd.grad([both, states], leaves,
                              [torch.cat([first, t["dout"]]), torch.cat([torch.zeros_like(states[:1]), t["dhT"]])])
    for a, n in zip(got, ("dx", "dw", "dbias", "dh0")):
        assert torch.equal(a, want[n]), n


@pytest.mark.parametrize("first,again", [(0, 1), (0, 64), (63, 255), (0, 256), (255, 256), (300, 599), (511, 512)])
def test_pool_slots_named_again_far_behind(first, again):
    """Of two sequences with one slot the first has it, however many lie between."""
    t, c, pool, slots = pool_case(23, "bf16", 600, 1, 16, 3, 600)
    slots[again] = slots[first]
    want_pool, keep = pool.clone(), torch.arange(600, device="cuda") != again
    want = gdn.conv_fwd_pool(t["x"][keep], t["w"], want_pool, slots[keep], t["bias"])
    out = gdn.conv_fwd_pool(t["x"], t["w"], pool, slots, t["bias"])
    assert torch.equal(out[keep], want) and not out[again].any() and torch.equal(pool, want_pool)
