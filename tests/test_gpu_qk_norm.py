"""Norms of queries and keys with the rotation on the GPU against the FP64
oracle (tolerances: block_case.py)."""
import numpy as np
import pytest

from block_case import U, check_norm, check_norm_bwd, f64, within
from oracle import block

torch = pytest.importorskip("torch")
import gated_deltanet_recurrence_delta_amd as gdn  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(seed, dtype, lead, Hq, Hk, d, rot, P, weight=True, far=False):
    r = np.random.default_rng(seed)
    dev = lambda a, t=torch.float32: torch.from_numpy(np.asarray(a, np.float32)).cuda().to(t)  # noqa: E731
    t = {"q": dev(3 * r.standard_normal((*lead, Hq, d)), DT[dtype]), "k": dev(r.standard_normal((*lead, Hk, d)), DT[dtype]),
         "dqo": dev(r.standard_normal((*lead, Hq, d)), DT[dtype]), "dko": dev(r.standard_normal((*lead, Hk, d)), DT[dtype])}
    how = {"wq": dev(r.standard_normal(d)) if weight else None, "wk": dev(r.standard_normal(d)) if weight else None,
           "cos": None, "sin": None, "pos": None}
    if rot:
        a = np.arange(P)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
        how["cos"], how["sin"] = dev(np.cos(a)), dev(np.sin(a))
        how["pos"] = torch.from_numpy(r.integers(0, P, lead).astype(np.int32)).cuda()
    return t, how


def check(t, how, dtype, norm, interleaved, eps=1e-6, back=True):
    outs = gdn.qk_norm_fwd(t["q"], t["k"], **how, norm=norm, eps=eps, interleaved=interleaved)
    g = gdn.qk_norm_bwd(t["q"], t["k"], t["dqo"], t["dko"], **how, norm=norm, eps=eps, interleaved=interleaved)
    cos, sin = f64(how["cos"]), f64(how["sin"])
    lead = t["q"].shape[:-2]
    pos = None if cos is None else f64(how["pos"]).astype(int).reshape(-1) if how["pos"] is not None else \
        np.tile(np.arange(lead[-1]), lead[0])
    for n, y in zip("qk", outs):
        flat = lambda a: f64(a).reshape(-1, *a.shape[-2:])  # noqa: E731
        x, w = flat(t[n]), f64(how["w" + n])
        check_norm(x, w, cos, sin, pos, norm == "l2", np.float64(np.float32(eps)), interleaved, dtype, flat(y))
        check_norm_bwd(x, w, cos, sin, pos, norm == "l2", np.float64(np.float32(eps)), interleaved, dtype,
                       flat(t["d" + n + "o"]), flat(g["d" + n]), f64(g["dw" + n]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("part", [0, 0.25, 0.5, 1])
@pytest.mark.parametrize("interleaved", [False, True])
def test_widths_and_rotations(dtype, d, part, interleaved):
    t, how = make(d, dtype, (2, 5), 3, 2, d, int(d * part), 40)
    check(t, how, dtype, "rms", interleaved)


@pytest.mark.parametrize("rot", [2, 6, 10, 30, 62])
@pytest.mark.parametrize("interleaved", [False, True])
def test_odd_rotations(rot, interleaved):
    check(*make(rot, "f32", (7,), 2, 3, 64, rot, 9), "f32", "l2", interleaved)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("Hq,Hk,lead", [(1, 1, (1, 1)), (5, 1, (3, 1)), (9, 7, (1, 33)), (16, 4, (4, 6)), (33, 2, (11,))])
def test_heads_and_batches(dtype, norm, Hq, Hk, lead):
    for weight in (True, False):
        check(*make(Hq, dtype, lead, Hq, Hk, 64, 32, 12, weight), dtype, norm, False)


def test_many_rows():
    """Units of several heads, and more of them than workgroups."""
    check(*make(1, "bf16", (2, 2100), 12, 3, 128, 64, 2100), "bf16", "rms", False)


def test_positions_by_default():
    t, how = make(2, "f32", (3, 9), 2, 1, 32, 16, 9)
    how["pos"] = None
    check(t, how, "f32", "rms", True)
    how["pos"] = torch.arange(9, dtype=torch.int32).expand(3, 9).contiguous().cuda()
    check(t, how, "f32", "rms", True)


def test_far_positions():
    check(*make(3, "f32", (5, 1), 4, 2, 64, 64, 1 << 18), "f32", "rms", False)


def test_positions_outside_the_tables_give_zeros():
    t, how = make(4, "bf16", (6,), 2, 2, 64, 64, 10)
    how["pos"] = torch.tensor([3, -1, 10, 2 ** 31 - 1, -2 ** 31, 9], dtype=torch.int32).cuda()
    qo, ko = gdn.qk_norm_fwd(t["q"], t["k"], **how)
    assert not qo[1:5].any() and not ko[1:5].any() and qo[0].any() and ko[5].any()
    check(t, how, "bf16", "rms", False)


def test_short_tables_without_positions():
    t, how = make(5, "f32", (2, 7), 2, 1, 32, 32, 4)
    how["pos"] = None
    qo, _ = gdn.qk_norm_fwd(t["q"], t["k"], **how)
    assert qo[:, :4].any() and not qo[:, 4:].any()


def test_zero_rows_and_non_finite_values():
    t, how = make(6, "f32", (4,), 2, 2, 64, 16, 4)
    t["q"][1, 0] = 0
    check(t, how, "f32", "l2", False)
    want, _ = gdn.qk_norm_fwd(t["q"], t["k"], **how)
    t["q"][2, 1, 7] = float("nan")
    t["q"][3, 0, 20] = float("inf")
    got, ko = gdn.qk_norm_fwd(t["q"], t["k"], **how)
    same = torch.ones(4, 2, dtype=torch.bool)
    same[2, 1] = same[3, 0] = False
    assert torch.equal(got[same.cuda()], want[same.cuda()])
    assert got[2, 1].isnan().all() and got[3, 0, 20].isnan()
    g = gdn.qk_norm_bwd(t["q"], t["k"], t["dqo"], t["dko"], **how)
    assert g["dq"][same.cuda()].isfinite().all() and g["dk"].isfinite().all()


def test_no_rows():
    t, how = make(7, "f32", (0, 5), 2, 2, 64, 16, 4)
    qo, ko = gdn.qk_norm_fwd(t["q"], t["k"], **how)
    assert qo.shape == t["q"].shape
    g = gdn.qk_norm_bwd(t["q"], t["k"], t["dqo"], t["dko"], **how)
    assert not g["dwq"].any() and not g["dwk"].any()


def test_one_side_s_weights():
    t, how = make(8, "f32", (3, 5), 4, 2, 64, 32, 8)
    how["wq"] = None
    check(t, how, "f32", "rms", False)


def test_a_row_does_not_depend_on_its_batch():
    t, how = make(9, "bf16", (40, 30), 8, 2, 128, 128, 64)
    qo, ko = gdn.qk_norm_fwd(t["q"], t["k"], **how)
    one = {**how, "pos": how["pos"][17:18]}
    a, b = gdn.qk_norm_fwd(t["q"][17:18], t["k"][17:18], **one)
    assert torch.equal(a[0], qo[17]) and torch.equal(b[0], ko[17])


def test_operation():
    t, how = make(10, "bf16", (2, 9), 4, 2, 64, 32, 9)
    want = gdn.qk_norm_bwd(t["q"], t["k"], t["dqo"], t["dko"], **how)
    leaves = [t["q"].requires_grad_(), t["k"].requires_grad_(), how["wq"].requires_grad_(), how["wk"].requires_grad_()]
    qo, ko = gdn.qk_norm(t["q"], t["k"], **how)
    got = torch.autograd.grad([qo, ko], leaves, [t["dqo"], t["dko"]])
    for a, n in zip(got, ("dq", "dk", "dwq", "dwk")):
        assert torch.equal(a, want[n]), n


def test_captured_and_another_stream():
    t, how = make(11, "bf16", (16, 1), 8, 2, 128, 64, 50)
    qo, ko = torch.empty_like(t["q"]), torch.empty_like(t["k"])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    want = gdn.qk_norm_fwd(t["q"], t["k"], **how)
    gdn.qk_norm_fwd(t["q"], t["k"], **how, qo=qo, ko=ko, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.qk_norm_fwd(t["q"], t["k"], **how, qo=qo, ko=ko)
    for i in range(4):
        how["pos"].copy_((how["pos"] + 7) % 50)
        t["q"].mul_(-1.5)
        torch.cuda.synchronize()
        graph.replay()
        want = gdn.qk_norm_fwd(t["q"], t["k"], **how)
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])


def test_twice_the_same():
    t, how = make(12, "f32", (3, 200), 5, 5, 64, 64, 200)
    a, b = (gdn.qk_norm_bwd(t["q"], t["k"], t["dqo"], t["dko"], **how) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("dtype,d,rot,interleaved,tokens,Hq,Hk", [
    ("bf16", 256, 64, False, 2600, 13, 5),   # queries two heads a unit, the last one's unit a single head
    ("f32", 256, 256, True, 5100, 13, 2),    # four, and one
    ("bf16", 256, 128, False, 10100, 13, 7), # eight and five; keys four and three
    ("f32", 256, 30, False, 10100, 3, 15),   # keys eight and seven; queries one
    ("bf16", 128, 0, False, 9400, 7, 8),     # two, keys two without a remainder
    ("bf16", 32, 32, True, 87400, 3, 1),     # two, and one
])
def test_units_of_several_heads(dtype, d, rot, interleaved, tokens, Hq, Hk):
    """A unit has 2, 4 or 8 heads from 8,192 waves of units on (d / 512 of one a head): the last of a token's units may
    have fewer.  The weights' sums take at most 16 rows of a lane, 64 lanes of a workgroup, 2,048 / 32 workgroups and 32
    sums of those: 176 roundings, whatever the number of rows, after a row's own d / 2 + 16."""
    t, how = make(tokens + Hq, dtype, (tokens,), Hq, Hk, d, rot, 60)
    if rot:
        how["pos"][::7] = -1
    qo, ko = gdn.qk_norm_fwd(t["q"], t["k"], **how, interleaved=interleaved)
    g = gdn.qk_norm_bwd(t["q"], t["k"], t["dqo"], t["dko"], **how, interleaved=interleaved)
    cos, sin, pos = (f64(how[n]) for n in ("cos", "sin", "pos"))
    pos = None if pos is None else pos.astype(int)
    for n, y in (("q", qo), ("k", ko)):
        a = (f64(t[n]), f64(how["w" + n]), cos, sin, pos, False, np.float64(np.float32(1e-6)), interleaved)
        dy = f64(t["d" + n + "o"])
        check_norm(*a, dtype, f64(y))
        check_norm_bwd(*a, dtype, dy, f64(g["d" + n]), None)
        _, dw, _, mw = block.norm_bwd(*a, dy)
        within("dw" + n, g["dw" + n], dw, (d / 2 + 16 + 176) * U * mw)
