"""Linear attention with a decay per head on the GPU, against the FP64 oracle.

Tolerances come from the arithmetic.  With A the same sums over absolute
values (the oracle on |q|, |k|, |v|, |h0|), every rounding of relative size r
to a term of a sum moves the sum by at most r A:

- fp32 sums of n terms: n 2^-24 A, n the row width, a chunk's rows (64 at
  most) and four roundings for each 64 rows on the way; decay powers are
  within 2^-24;
- bf16: the masked scores or the state, and (for the outputs) the products'
  other operand being exact, one rounding of 2^-8 A, and the output's own
  2^-8 |out|; values that enter the state keep 16 bits at least, 2^-16 A.

A decay near one is applied as m + (a^n - 1) m, in one rounding: no factor's own
rounding adds up over the chunks.
"""
import numpy as np
import pytest

from oracle import linear

torch = pytest.importorskip("torch")
import gated_deltanet_recurrence_delta_amd as gdn  # noqa: E402

pytestmark = pytest.mark.gpu

EPS = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


def make(seed, dtype, lead, H, dk, dv, B, h0=True, packed=False, slow=False):
    r = np.random.default_rng(seed)
    shape = (lead, H) if packed else (B, lead, H)
    dev = lambda x: torch.from_numpy(np.asarray(x, np.float32)).cuda()  # noqa: E731
    c = {n: dev(r.standard_normal(shape + (d,)) / np.sqrt(d)).to(DT[dtype]) for n, d in (("q", dk), ("k", dk))}
    c["v"] = dev(r.standard_normal(shape + (dv,))).to(DT[dtype])
    c["dout"] = dev(r.standard_normal(shape + (dv,))).to(DT[dtype])
    # from no memory to one longer than the sequence
    c["g"] = dev(-np.exp2(r.uniform(-9 if slow else -6, 2, H)))
    c["h0"] = dev(r.standard_normal((B, H, dk, dv))) if h0 else None
    c["dhT"] = dev(r.standard_normal((B, H, dk, dv))) if h0 else None
    return c


def oracle_of(c, bounds=None, absolute=False):
    """out, hT and the gradients, over packed sequences if bounds are given."""
    f = (lambda t: None if t is None else np.abs(f64(t))) if absolute else (lambda t: None if t is None else f64(t))
    g = f64(c["g"])
    if bounds is None:
        out, hT = linear.fwd(f(c["q"]), f(c["k"]), f(c["v"]), g, f(c["h0"]))
        return dict(out=out, hT=hT, **linear.bwd(f(c["q"]), f(c["k"]), f(c["v"]), g, f(c["dout"]), f(c["h0"]),
                                                 f(c["dhT"])))
    r = dict(out=np.zeros(c["v"].shape), dq=np.zeros(c["q"].shape), dk=np.zeros(c["k"].shape),
             dv=np.zeros(c["v"].shape), hT=[], dh0=[])
    for n, (b, e) in enumerate(zip(bounds, bounds[1:])):
        q, k, v, do = (f(c[x])[None, b:e] for x in ("q", "k", "v", "dout"))
        st = lambda x: None if c[x] is None else f(c[x])[n:n + 1]  # noqa: E731
        o, h = linear.fwd(q, k, v, g, st("h0"))
        gr = linear.bwd(q, k, v, g, do, st("h0"), st("dhT"))
        r["out"][b:e] = o[0]
        r["hT"].append(h[0])
        for x in ("dq", "dk", "dv"):
            r[x][b:e] = gr[x][0]
        r["dh0"].append(gr["dh0"][0])
    shape = (0,) + c["q"].shape[1:] + (c["v"].shape[-1],)
    r["hT"], r["dh0"] = (np.stack(r[x]) if r[x] else np.zeros(shape) for x in ("hT", "dh0"))
    return r


def check(got, c, dtype, bounds=None, recurrent=False):
    ref, mag = oracle_of(c, bounds), oracle_of(c, bounds, absolute=True)
    T = max([e - b for b, e in zip(bounds, bounds[1:])] or [0]) if bounds else c["q"].shape[1]
    d = max(c["q"].shape[-1], c["v"].shape[-1])
    terms = d + 3 * T + 10 if recurrent else d + 64 + 4 * (T / 64 + 1) + 10
    for name, x in got.items():
        assert x.shape == ref[name].shape, name
        state = name in ("hT", "dh0")
        tol = terms * 2.0 ** -24 * mag[name]
        if dtype == "bf16" and not recurrent:
            tol = tol + (2.0 ** -16 if state else 2.0 ** -8 + 2.0 ** -16) * mag[name]
        if not state:
            tol = tol + EPS[dtype] * (np.abs(ref[name]) + tol)
        err = np.abs(f64(x) - ref[name])
        bad = ~(err <= tol + 1e-37)
        assert not bad.any(), (name, int(bad.sum()), float((err / (tol + 1e-37)).max()), np.argwhere(bad)[:4].tolist())


def run_all(c, cu=None):
    out, hT = gdn.linear_fwd(c["q"], c["k"], c["v"], c["g"], c["h0"], cu)
    grads = gdn.linear_bwd(c["q"], c["k"], c["v"], c["g"], c["dout"], c["h0"], cu, dhT=c["dhT"])
    torch.cuda.synchronize()
    return dict(out=out, hT=hT, **grads)


DIMS = [(32, 32), (64, 64), (128, 128), (128, 32), (32, 64), (64, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("T", [1, 16, 31, 32, 33, 63, 64, 65, 130, 321])
def test_dense(dtype, dk, dv, T):
    c = make(T * 7 + dk + dv, dtype, T, 3, dk, dv, 2)
    check(run_all(c), c, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(32, 32), (128, 128), (64, 128)])
def test_without_states(dtype, dk, dv):
    c = make(dk + 1, dtype, 100, 2, dk, dv, 2, h0=False)
    check(run_all(c), c, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 64), (128, 128), (64, 32)])
@pytest.mark.parametrize("T", [1024, 1601, 2111])
def test_segments(dtype, dk, dv, T):
    """Few chains, so that long sequences are cut: slow decays carry through every cut."""
    assert gdn.gdn_linear_workspace_size(1, T, 2, dk, dv, 0, 1) > 0
    c = make(T + dk, dtype, T, 2, dk, dv, 1, slow=True)
    c["g"][0] = 0.0  # no decay at all
    check(run_all(c), c, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(32, 64), (128, 128)])
@pytest.mark.parametrize("bounds", [[0, 5], [0, 0, 1, 1, 65, 193, 193], [0, 300, 301, 364, 500], [0, 1300, 1300, 1310],
                                    [0, 3, 1027, 2300], [0], [0, 0]])
def test_packed(dtype, dk, dv, bounds):
    c = make(len(bounds), dtype, bounds[-1], 2, dk, dv, len(bounds) - 1, packed=True, slow=True)
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    check(run_all(c, cu), c, dtype, bounds)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [90, 1300])
def test_rows_of_no_sequence_stay(dtype, T):
    """Offsets that begin late and end early, and ones outside the tensors."""
    c = make(T, dtype, T, 2, 64, 64, 2, packed=True)
    for cu, bounds in (([7, 40, T - 9], [7, 40, T - 9]), ([-5, 40, T + 100], [0, 40, T]), ([9, 3, 30], [9, 9, 30])):
        cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
        out = torch.full_like(c["v"], 777.0)
        out, hT = gdn.linear_fwd(c["q"], c["k"], c["v"], c["g"], c["h0"], cut, out=out)
        if cu[1] < cu[0]:  # an end before its begin: empty, and the next sequence is rows 3 to 30
            ref = oracle_of(c, [3, 30])
            assert torch.equal(hT[0], c["h0"][0])
            assert bool((out[:3] == 777).all()) and bool((out[30:] == 777).all())
            del ref
            continue
        inside = torch.zeros(T, dtype=torch.bool, device="cuda")
        inside[bounds[0]:bounds[-1]] = True
        assert bool((out[~inside] == 777).all())
        check(dict(out=torch.where(inside[:, None, None], out, 0), hT=hT), c, dtype, bounds)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("T", [1, 2, 5, 40])
def test_recurrent(dtype, dk, dv, T):
    c = make(T + dv, dtype, T, 3, dk, dv, 2)
    out, hT = gdn.linear_fwd_recurrent(c["q"], c["k"], c["v"], c["g"], c["h0"])
    check(dict(out=out, hT=hT), c, dtype, recurrent=True)
    bounds = [0, T, T, 2 * T]
    c = make(T, dtype, 2 * T, 3, dk, dv, 3, packed=True)
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    out, hT = gdn.linear_fwd_recurrent(c["q"], c["k"], c["v"], c["g"], c["h0"], cu)
    check(dict(out=out, hT=hT), c, dtype, bounds, recurrent=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slow_decay_over_many_tokens(dtype):
    """A constant decay's rounding does not add up: 4,096 tokens at a decay that 24 bits cannot hold."""
    c = make(3, dtype, 4096, 1, 32, 32, 1)
    c["g"].fill_(-1.0e-5)
    check(run_all(c), c, dtype)
    out, hT = gdn.linear_fwd_recurrent(c["q"], c["k"], c["v"], c["g"], c["h0"])
    check(dict(out=out, hT=hT), c, dtype, recurrent=True)


@pytest.mark.parametrize("T", [100, 1500])
def test_forgetting_at_every_token(T):
    """g = -inf: out_t = (q_t . k_t) v_t, the state the last token's product."""
    c = make(4, "f32", T, 2, 64, 64, 1)
    c["g"].fill_(-float("inf"))
    for call in (gdn.linear_fwd, gdn.linear_fwd_recurrent):
        out, hT = call(c["q"], c["k"], c["v"], c["g"], c["h0"])
        q, k, v = (f64(c[n]) for n in "qkv")
        mag = np.sum(np.abs(q * k), -1, keepdims=True) * np.abs(v)
        assert (np.abs(f64(out) - np.sum(q * k, -1, keepdims=True) * v) <= 150 * 2.0 ** -24 * mag + 1e-37).all()
        last = k[:, -1, :, :, None] * v[:, -1, :, None, :]
        assert (np.abs(f64(hT) - last) <= 4 * 2.0 ** -24 * np.abs(last) + 1e-37).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_values_stay_in_their_chain(dtype, bad):
    T = 150
    c = make(5, dtype, T, 3, 64, 64, 2)
    clean = run_all(c)
    for n in ("q", "k", "v", "dout"):
        c[n][1, 70, 1] = bad
    dirty = run_all(c)
    for n in clean:
        a, b = clean[n].clone(), dirty[n].clone()
        if n in ("hT", "dh0"):
            assert not bool(torch.isfinite(b[1, 1]).all())
            a[1, 1] = b[1, 1] = 0
        else:
            assert not bool(torch.isfinite(b[1, 70, 1]).all())
            a[1, :, 1] = b[1, :, 1] = 0
        assert torch.equal(a, b), n
    assert bool(torch.isfinite(dirty["out"][1, :64, 1].float()).all())  # the chunks before


def test_no_value_outside_a_sequence_is_read():
    """Rows between and behind the sequences may hold anything."""
    c = make(6, "bf16", 700, 2, 64, 64, 2, packed=True)
    cu = torch.tensor([0, 200, 331], dtype=torch.int32, device="cuda")
    a = run_all(c, cu)
    for n in ("q", "k", "v", "dout"):
        c[n][331:] = float("nan")
    b = run_all(c, cu)
    for n in a:
        x, y = (a[n], b[n]) if n in ("hT", "dh0") else (a[n][:331], b[n][:331])
        assert torch.equal(x, y), n


@pytest.mark.parametrize("T", [130, 1700])
def test_in_place_states_and_determinism(T):
    c = make(7, "bf16", T, 2, 128, 128, 1)
    a, b = run_all(c), run_all(c)
    assert all(torch.equal(a[n], b[n]) for n in a)
    h = c["h0"].clone()
    out, hT = gdn.linear_fwd(c["q"], c["k"], c["v"], c["g"], h, hT=h)
    assert hT.data_ptr() == h.data_ptr()
    check(dict(out=out, hT=hT), c, "bf16")
    h = c["h0"].clone()
    out, hT = gdn.linear_fwd_recurrent(c["q"], c["k"], c["v"], c["g"], h, hT=h)
    check(dict(out=out, hT=hT), c, "bf16", recurrent=True)
    # dh0 in dhT's place, through the raw call
    d = c["dhT"].clone()
    g = {n: torch.empty_like(c[n[1]]) for n in ("dq", "dk", "dv")}
    size = gdn.gdn_linear_workspace_size(1, T, 2, 128, 128, 0, gdn.GDN_BF16, True)
    ws = torch.empty(max(1, size), dtype=torch.uint8, device="cuda")
    rc = gdn.gdn_linear_bwd(*(c[n].data_ptr() for n in ("q", "k", "v", "g", "h0")), 0, c["dout"].data_ptr(),
                            d.data_ptr(), *(g[n].data_ptr() for n in ("dq", "dk", "dv")), d.data_ptr(), 1, T, 2, 128,
                            128, torch.cuda.current_stream().cuda_stream, gdn.GDN_BF16, ws.data_ptr(), ws.numel())
    assert rc == 0
    check(dict(dh0=d, **g), c, "bf16")


@pytest.mark.parametrize("T", [77, 1300])
def test_outputs_alone_are_written(T):
    c = make(8, "bf16", T, 2, 64, 32, 1)
    n = c["v"].numel()
    buf = torch.full((n + 8192,), 555.0, dtype=torch.bfloat16, device="cuda")
    st = torch.full((2 * 64 * 32 + 8192,), 555.0, device="cuda")
    out, hT = buf[4096:4096 + n].view_as(c["v"]), st[4096:-4096].view(1, 2, 64, 32)
    size = gdn.gdn_linear_workspace_size(1, T, 2, 64, 32, 0, gdn.GDN_BF16)
    ws = torch.full((size + 8192,), 55, dtype=torch.uint8, device="cuda")
    gdn.linear_fwd(c["q"], c["k"], c["v"], c["g"], c["h0"], out=out, hT=hT, workspace=ws[4096:4096 + size])
    check(dict(out=out, hT=hT), c, "bf16")
    for x, v in ((buf, 555), (st, 555), (ws, 55)):
        assert bool((x[:4096] == v).all()) and bool((x[-4096:] == v).all())


@pytest.mark.parametrize("T,dk,dv", [(200, 64, 64), (1500, 128, 64), (1500, 128, 128)])
def test_autograd(T, dk, dv):
    c = make(9, "bf16", T, 2, dk, dv, 1)
    leaves = [c[n].clone().requires_grad_() for n in ("q", "k", "v", "h0")]
    out, hT = gdn.linear_attention(*leaves[:3], c["g"], leaves[3])
    grads = torch.autograd.grad([out, hT], leaves, [c["dout"], c["dhT"]])
    check(dict(out=out, hT=hT, **dict(zip(("dq", "dk", "dv", "dh0"), grads))), c, "bf16")
    # the outputs alone, with a gradient that is one value read many times
    out, _ = gdn.linear_attention(*leaves[:3], c["g"])
    (dq,) = torch.autograd.grad(out.float().sum(), leaves[:1])
    ones = dict(c, dout=torch.ones_like(c["dout"]), h0=None, dhT=None)
    check(dict(dq=dq), ones, "bf16")
    # rows of no sequence get zeros
    q, k, v = (x[0].detach().clone().requires_grad_() for x in leaves[:3])
    cu = torch.tensor([3, T - 5], dtype=torch.int32, device="cuda")
    out, _ = gdn.linear_attention(q, k, v, c["g"], None, cu)
    for x in (out, *torch.autograd.grad(out.float().sum(), (q, k, v))):
        assert not bool(x[:3].any()) and not bool(x[T - 5:].any()) and bool(torch.isfinite(x.float()).all())


def test_gradients_against_differences():
    """The outputs are linear in each input: in fp32 a difference over a whole step is exact up to rounding."""
    c = make(10, "f32", 150, 2, 32, 32, 1)
    grads = run_all(c)

    def loss(d):
        out, hT = gdn.linear_fwd(d["q"], d["k"], d["v"], c["g"], d["h0"])
        return float((out.double() * c["dout"].double()).sum() + (hT.double() * c["dhT"].double()).sum())

    for n in ("q", "k", "v", "h0"):
        step = torch.randn(c[n].shape, generator=torch.Generator().manual_seed(1)).cuda()
        diff = (loss({**c, n: c[n] + step}) - loss({**c, n: c[n] - step})) / 2
        want = float((grads["d" + n].double() * step.double()).sum())
        # the losses' own rounding, of sums of absolute values
        a = oracle_of(dict(c, **{n: c[n].abs() + step.abs()}), absolute=True)
        mag = float((a["out"] * np.abs(f64(c["dout"]))).sum() + (a["hT"] * np.abs(f64(c["dhT"]))).sum())
        assert abs(diff - want) <= 3 * 150 * 2.0 ** -24 * mag


@pytest.mark.parametrize("T,cut", [(65, False), (1300, True)])
def test_graph_and_streams(T, cut):
    """Captured calls follow their inputs from replay to replay; two captures keep apart; a stream of one's own."""
    cs = [make(11 + i, "bf16", T, 2, 64, 64, 1) for i in range(3)]
    want = [run_all(c) for c in cs]
    live = {n: x.clone() for n, x in cs[0].items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_all(live)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out, hT = gdn.linear_fwd(live["q"], live["k"], live["v"], live["g"], live["h0"])
            grads = gdn.linear_bwd(live["q"], live["k"], live["v"], live["g"], live["dout"], live["h0"],
                                   dhT=live["dhT"])
        graphs.append((graph, dict(out=out, hT=hT, **grads)))
    for r in range(6):
        for n in live:
            live[n].copy_(cs[r % 3][n])
        graph, got = graphs[r % 2]
        graph.replay()
        other = run_all(cs[(r + 1) % 3])
        torch.cuda.synchronize()
        for n in got:
            assert torch.equal(got[n], want[r % 3][n]), (r, n)
            assert torch.equal(other[n], want[(r + 1) % 3][n]), (r, n)
    # both graphs at once on two streams: their workspaces are their own
    for n in live:
        live[n].copy_(cs[1][n])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s, (graph, _) in zip(streams, graphs):
        with torch.cuda.stream(s):
            graph.replay()
    out, hT = gdn.linear_fwd(cs[2]["q"], cs[2]["k"], cs[2]["v"], cs[2]["g"], cs[2]["h0"], stream=streams[0])
    torch.cuda.synchronize()
    for _, got in graphs:
        assert all(torch.equal(got[n], want[1][n]) for n in got)
    assert torch.equal(out, want[2]["out"]) and torch.equal(hT, want[2]["hT"])


def test_refused_on_the_gpu():
    c = make(12, "bf16", 40, 2, 64, 64, 1)
    with pytest.raises(ValueError, match="contiguous"):
        gdn.linear_fwd(c["q"].transpose(1, 2).contiguous().transpose(1, 2), c["k"], c["v"], c["g"])
    odd = torch.empty(c["q"].numel() + 4, dtype=torch.bfloat16, device="cuda")[4:].view_as(c["q"])
    with pytest.raises(gdn.GdnError, match="gdn_linear_fwd failed"):
        gdn.linear_fwd(odd, c["k"], c["v"], c["g"])
    with pytest.raises(gdn.GdnError):
        gdn.linear_fwd(c["q"], c["k"], c["v"], c["g"], out=c["v"])
    with pytest.raises(ValueError):
        gdn.linear_fwd(c["q"], c["k"], c["v"], c["g"], out=torch.empty(1, 40, 2, 32, device="cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_tokens(dtype):
    """Sequences of no tokens hand their states on, in both directions."""
    c = make(13, dtype, 0, 2, 64, 64, 3)
    got = run_all(c)
    assert torch.equal(got["hT"], c["h0"]) and torch.equal(got["dh0"], c["dhT"]) and got["out"].numel() == 0
    out, hT = gdn.linear_fwd_recurrent(c["q"], c["k"], c["v"], c["g"])
    assert not bool(hT.any()) and out.shape == c["v"].shape


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B", [64, 65, 700])
def test_many_packed_sequences(dtype, B):
    """As many sequences as are put in order of length, and more; some long enough to be cut, some a whole
    number of segments."""
    r = np.random.default_rng(B)
    lens = r.integers(0, 5, B)
    lens[[3, 11, B // 2, B - 1]] = [400, 256, 333, 128]
    bounds = [0, *np.cumsum(lens).tolist()]
    c = make(B, dtype, bounds[-1], 1, 32, 32, B, packed=True, slow=True)
    check(run_all(c, torch.tensor(bounds, dtype=torch.int32, device="cuda")), c, dtype, bounds)


@pytest.mark.parametrize("dk,dv", [(32, 32), (128, 128)])
@pytest.mark.parametrize("H", [1, 7, 19])
def test_odd_heads(dk, dv, H):
    c = make(H, "bf16", 70, H, dk, dv, 3)
    check(run_all(c), c, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_rows_are_left_out_of_cut_sequences(dtype):
    """A fast decay in a cut sequence: what is left out is below e^-40 of its own size."""
    c = make(14, dtype, 3000, 2, 64, 64, 1)
    c["g"].copy_(torch.tensor([-0.5, -8.0]))
    assert gdn.gdn_linear_workspace_size(1, 3000, 2, 64, 64, 0, gdn.GDN_BF16) > 0
    check(run_all(c), c, dtype)
