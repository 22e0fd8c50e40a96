"""States in a pool on the GPU: token-by-token forms on slots against the FP64
rule, slot moves against indexing, and a serving run of them together.

Tolerances: fp32 sums of n terms are within n 2^-24 of the same sums over
absolute values; n is the row width and, a token, the update's four roundings
and the delta rule's second sum over the row.  bf16 outputs add 2^-8.
"""
import numpy as np
import pytest

from oracle import linear

torch = pytest.importorskip("torch")
import gated_deltanet_recurrence_delta_amd as gdn  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


def make(seed, dtype, B, T, H, dk, dv, nslots):
    r = np.random.default_rng(seed)
    dev = lambda x: torch.from_numpy(np.asarray(x, np.float32)).cuda()  # noqa: E731
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
    c = {n: dev(unit(r.standard_normal((B, T, H, dk)))).to(DT[dtype]) for n in "qk"}
    c["v"] = dev(r.standard_normal((B, T, H, dv))).to(DT[dtype])
    c["g"] = dev(-np.exp(r.standard_normal((B, T, H))))
    c["beta"] = dev(r.uniform(0, 1, (B, T, H)))
    c["gh"] = dev(-np.exp2(r.uniform(-6, 2, H)))
    c["pool"] = dev(r.standard_normal((nslots, H, dk, dv)))
    c["slots"] = torch.from_numpy(r.permutation(nslots)[:B].astype(np.int32)).cuda()
    return c


def bounds(c, S, delta):
    """(out, states, tolerance of each) for start states S."""
    q, k, v = (f64(c[n]) for n in "qkv")
    if delta:
        g, beta = f64(c["g"]), f64(c["beta"])
        out, hT = linear.delta(q, k, v, g, beta, S)
        # |v| and |k| M with the prediction's sign turned: the sums over absolute values
        M, mo = np.abs(S), np.zeros(v.shape)
        for t in range(q.shape[1]):
            M = np.exp(g[:, t])[..., None, None] * M
            p = np.matmul(np.abs(k)[:, t, :, None, :], M)[:, :, 0]
            u = beta[:, t][..., None] * (np.abs(v[:, t]) + p)
            # o is formed as a M^T q + u (k . q)
            mo[:, t] = np.matmul(np.abs(q)[:, t, :, None, :], M)[:, :, 0] + u * np.sum(np.abs(q * k)[:, t], -1)[..., None]
            M = M + np.abs(k)[:, t, :, :, None] * u[:, :, None, :]
    else:
        gh = f64(c["gh"])
        out, hT = linear.fwd(q, k, v, gh, S)
        mo, M = linear.fwd(np.abs(q), np.abs(k), np.abs(v), gh, np.abs(S))
    # the delta rule's decays are single fp32 exponentials: 2^-22 each at |g| < 20
    n = (2 * q.shape[-1] + 16) * q.shape[1] * 2.0 ** -24
    e = 2.0 ** -8 if c["q"].dtype == torch.bfloat16 else 2.0 ** -24
    return out, hT, n * mo + e * (np.abs(out) + n * mo), n * M


def call(c, delta, **kw):
    if delta:
        return gdn.fwd_recurrent_pool(c["q"], c["k"], c["v"], c["g"], c["beta"], c["pool"], c["slots"], **kw)
    return gdn.linear_fwd_recurrent_pool(c["q"], c["k"], c["v"], c["gh"], c["pool"], c["slots"], **kw)


def check(c, delta, valid=None, **kw):
    before = c["pool"].clone()
    slots = c["slots"].tolist()
    valid = list(range(len(slots))) if valid is None else valid
    S = np.zeros((len(slots),) + tuple(before.shape[1:]))
    for i in valid:
        S[i] = f64(before[slots[i]])
    out, hT, to, th = bounds(c, S, delta)
    got = call(c, delta, **kw)
    torch.cuda.synchronize()
    touched = set()
    for i in range(len(slots)):
        if i in valid:
            touched.add(slots[i])
            assert (np.abs(f64(got[i]) - out[i]) <= to[i] + 1e-37).all(), i
            assert (np.abs(f64(c["pool"][slots[i]]) - hT[i]) <= th[i] + 1e-37).all(), i
        else:
            assert not bool(got[i].any())
    for s in set(range(before.shape[0])) - touched:
        assert torch.equal(c["pool"][s], before[s]), s
    return got


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 3])
def test_decode(delta, dtype, dk, dv, T):
    check(make(dk + dv + T, dtype, 5, T, 3, dk, dv, 9), delta)


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("B,H", [(1, 1), (300, 2), (40, 17)])
def test_batches(delta, B, H):
    check(make(B, "bf16", B, 1, H, 64, 64, B + 3), delta)


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(32, 64), (32, 128), (64, 128), (128, 64), (128, 128)])
def test_many_chains(delta, dtype, dk, dv):
    """Enough chains that one workgroup takes all of a chain's columns."""
    check(make(dk + 7 * dv, dtype, 90, 2, 3, dk, dv, 91), delta)


@pytest.mark.parametrize("delta", [False, True])
def test_slots_of_no_sequence(delta):
    """Padding rows, slots outside the pool, and a slot named again: no state changes, zeros come out."""
    c = make(1, "bf16", 8, 2, 2, 64, 128, 6)
    c["slots"] = torch.tensor([4, -1, 2, 4, 6, 1 << 30, 2, 0], dtype=torch.int32, device="cuda")
    c["v"][1] = c["q"][4] = float("nan")  # a padding row may hold anything
    c["k"][3] = float("inf")
    check(c, delta, valid=[0, 2, 7], out=torch.full_like(c["v"], 9.0))


@pytest.mark.parametrize("delta", [False, True])
def test_packed(delta):
    """Ragged lengths, none among them; rows of no sequence stay as they were."""
    c = make(2, "f32", 1, 20, 3, 32, 64, 6)
    lens, first = [3, 0, 1, 7], 2
    cu = torch.tensor(np.cumsum([first] + lens), dtype=torch.int32, device="cuda")
    rows = {n: c[n][0] for n in ("q", "k", "v", "g", "beta")}
    before = c["pool"].clone()
    slots = torch.tensor([3, 5, 0, 1], dtype=torch.int32, device="cuda")
    out = torch.full_like(rows["v"], 9.0)
    got = call(dict(c, **rows, slots=slots), delta, cu_seqlens=cu, out=out)
    assert bool((got[:2] == 9).all()) and bool((got[13:] == 9).all())
    at = first
    for n, s in zip(lens, slots.tolist()):
        one = dict(c, slots=slots, **{x: rows[x][None, at:at + n] for x in rows})
        o, h, to, th = bounds(one, f64(before[s])[None], delta)
        assert (np.abs(f64(got[at:at + n]) - o[0]) <= to[0] + 1e-37).all()
        assert (np.abs(f64(c["pool"][s]) - h[0]) <= th[0] + 1e-37).all()
        at += n
    assert torch.equal(c["pool"][[2, 4]], before[[2, 4]]) and torch.equal(c["pool"][5], before[5])


def test_as_without_a_pool():
    """The pool's form gives what the form on a batch of states gives."""
    c = make(3, "bf16", 6, 4, 3, 128, 64, 6)
    h0 = c["pool"][c["slots"].long()].clone()
    out, hT = gdn.linear_fwd_recurrent(c["q"], c["k"], c["v"], c["gh"], h0)
    got = call(c, False)
    assert torch.equal(got, out) and torch.equal(c["pool"][c["slots"].long()], hT)


@pytest.mark.parametrize("delta", [False, True])
def test_graph(delta):
    """A captured step follows tokens, slots and states from replay to replay, padding rows among them."""
    c = make(4, "bf16", 4, 1, 2, 64, 64, 8)
    ref = {n: x.clone() for n, x in c.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(c, delta)
    c["pool"].copy_(ref["pool"])
    for step in range(6):
        new = make(50 + step, "bf16", 4, 1, 2, 64, 64, 8)
        if step % 2:
            new["slots"][3] = -1
        for n in ("q", "k", "v", "g", "beta", "gh", "slots"):
            c[n].copy_(new[n])
            ref[n].copy_(new[n])
        graph.replay()
        want = call(ref, delta)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(c["pool"], ref["pool"]), step


# ----------------------------------------------------------------- moves --

def indexed(pool, src, dst, dim):
    """The move by torch's own indexing, on the host."""
    p = pool.cpu().transpose(0, dim).contiguous()
    old = p.clone()
    for s, d in zip(src, dst):
        p[d] = old[s] if s >= 0 else 0
    return p.transpose(0, dim).contiguous()


@pytest.mark.parametrize("shape,dim", [((7, 4), 0), ((40, 3, 2, 4), 0), ((3, 33, 260), 1), ((2, 3, 9, 5000), 2),
                                       ((2, 700, 8), 1)])
@pytest.mark.parametrize("kind", ["random", "clear", "permutation", "cycle", "one source", "shift"])
def test_moves(shape, dim, kind):
    r = np.random.default_rng(len(kind) + shape[dim])
    N = shape[dim]
    dst = r.permutation(N)[:max(1, N - 2)].tolist()
    n = len(dst)
    src = {"random": r.integers(0, N, n).tolist(), "clear": r.integers(-1, 1, n).tolist(),
           "permutation": r.permutation(dst).tolist(), "cycle": dst[1:] + dst[:1], "one source": [dst[0]] * n,
           "shift": dst[1:] + [N - 1]}[kind]
    pool = torch.from_numpy(r.standard_normal(shape).astype(np.float32)).cuda()
    want = indexed(pool, src, dst, dim)
    assert gdn.state_move(pool, src, dst, dim=dim) is pool
    assert torch.equal(pool.cpu(), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.uint8, torch.int64])
def test_moves_of_any_type(dtype):
    pool = torch.arange(6 * 32).reshape(6, 32).to(dtype).cuda()
    want = indexed(pool, [0, 5, 2], [5, 2, 1], 0)
    gdn.state_move(pool, np.array([0, 5, 2]), torch.tensor([5, 2, 1]))
    assert torch.equal(pool.cpu(), want)
    gdn.state_move(pool, [], [])
    gdn.state_move(pool[:0], [], [])
    assert torch.equal(pool.cpu(), want)


def test_moves_keep_to_the_pool():
    buf = torch.arange(4096.0 * 3, device="cuda")
    pool = buf[4096:8192].view(4, 1024)
    gdn.state_move(pool, [0, 1, 2, 3], [3, 0, 1, 2])
    assert torch.equal(buf[:4096], torch.arange(4096.0, device="cuda"))
    assert torch.equal(buf[8192:], torch.arange(8192.0, 12288.0, device="cuda"))
    with pytest.raises(gdn.GdnError, match="gdn_state_move failed"):
        gdn.state_move(buf[4096:4096 + 12].view(4, 3), [0], [1])  # 12 bytes a slot
    with pytest.raises(gdn.GdnError):
        gdn.state_move(buf[4097:4097 + 32].view(4, 8), [0], [1])  # not 16-byte aligned
    with pytest.raises(ValueError):
        gdn.state_move(buf[:4096].view(64, 64).t(), [0], [1])
    with pytest.raises(TypeError):
        gdn.state_move(pool, torch.tensor([0], device="cuda"), [1])


def test_moves_in_a_graph():
    pool = torch.randn(9, 64, device="cuda")
    ref = pool.clone()
    src, dst = [1, 2, 0, 4, 4, -1], [0, 1, 2, 5, 6, 7]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.state_move(pool, src, dst)
    for _ in range(4):
        graph.replay()
        ref = indexed(ref, src, dst, 0)
        torch.cuda.synchronize()
        assert torch.equal(pool.cpu(), ref)


def test_offsets_beyond_32_bits():
    """A pool of more than 4 GiB: its last slots move and decode as the first do."""
    H, d, N = 16, 128, 4200  # 1 MiB a slot
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("less than 8 GiB of GPU memory is free")
    pool = torch.zeros(N, H, d, d, device="cuda")
    c = make(5, "bf16", 2, 1, H, d, d, 2)
    pool[0].copy_(c["pool"][0])
    gdn.state_move(pool, [0, 0], [N - 1, 3000])
    c["slots"].copy_(torch.tensor([N - 1, 3000]))
    small = dict(c, pool=torch.stack([c["pool"][0], c["pool"][0]]), slots=torch.arange(2, dtype=torch.int32).cuda())
    out = gdn.linear_fwd_recurrent_pool(c["q"], c["k"], c["v"], c["gh"], pool, c["slots"])
    want = gdn.linear_fwd_recurrent_pool(c["q"], c["k"], c["v"], c["gh"], small["pool"], small["slots"])
    assert torch.equal(out, want)
    assert torch.equal(pool[N - 1], small["pool"][0]) and torch.equal(pool[3000], small["pool"][1])


# ------------------------------------------------------- all of it at once --

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_serving_run(dtype):
    """Packed prompts, their states into slots, a fork, decoding, a user leaving, compaction, more decoding --
    against the rule over each user's whole history in 64 bits."""
    H, dk, dv, layers = 2, 64, 64, 2
    r = np.random.default_rng(6)
    dev = lambda x: torch.from_numpy(np.asarray(x, np.float32)).cuda()  # noqa: E731
    g = dev(-np.exp2(r.uniform(-7, 1, H)))
    pool = gdn.StatePool(6, H, dk, dv, layers=layers)
    lens = [70, 1, 33]
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    history = [{} for _ in range(layers)]  # per layer: user -> q, k, v rows so far
    token = lambda n: [dev(r.standard_normal((n, H, d)) / 8).to(DT[dtype]) for d in (dk, dk, dv)]  # noqa: E731
    users = dict(enumerate(pool.alloc(3)))  # user -> slot
    for layer in range(layers):
        rows = token(sum(lens))
        _, hT = gdn.linear_fwd(*rows, g, cu_seqlens=cu)
        pool.states[layer, torch.tensor(list(users.values()), device="cuda")] = hT
        for u, (b, e) in enumerate(zip(cu.tolist(), cu.tolist()[1:])):
            history[layer][u] = [x[b:e] for x in rows]

    def decode(who):
        slots = torch.tensor([users[u] for u in who] + [-1], dtype=torch.int32, device="cuda")
        for layer in range(layers):
            new = [x[:, None] for x in token(len(who) + 1)]
            out = gdn.linear_fwd_recurrent_pool(*new, g, pool.states[layer], slots)
            assert not bool(out[-1].any())
            for i, u in enumerate(who):
                h = history[layer][u] = [torch.cat([a, b[i]]) for a, b in zip(history[layer][u], new)]
                q, k, v = (f64(x)[None] for x in h)
                o, S = linear.fwd(q, k, v, f64(g))
                mo, mS = linear.fwd(np.abs(q), np.abs(k), np.abs(v), f64(g))
                # the prompt's chunks (bf16: values of 16 bits at least), then the tokens, each with its own sums
                n = (2.0 ** -16 if dtype == "bf16" else 0) + (64 + 64 + 4 * 4 + 3 * 8 + 20) * 2.0 ** -24
                e = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
                assert (np.abs(f64(out[i, 0]) - o[0, -1]) <= n * mo[0, -1] + e * (np.abs(o[0, -1]) + n * mo[0, -1])).all()
                assert (np.abs(f64(pool.states[layer, users[u]]) - S[0]) <= n * mS[0]).all()

    decode([0, 1, 2])
    a, b = pool.fork(users[2], 2)
    users.update({3: a, 4: b})
    for layer in range(layers):
        history[layer][3] = history[layer][4] = history[layer][2]
    decode([4, 0, 3, 2, 1])
    for u in (0, 2):
        pool.free([users.pop(u)])
    moved = pool.compact()
    assert moved
    users = {u: moved.get(s, s) for u, s in users.items()}
    assert sorted(users.values()) == [0, 1, 2]
    decode([1, 3, 4])
    (users[5],) = pool.alloc()
    for layer in range(layers):
        history[layer][5] = [torch.empty(0, H, d, device="cuda", dtype=DT[dtype]) for d in (dk, dk, dv)]
    decode([5, 3])
