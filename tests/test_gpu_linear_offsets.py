"""Packed offsets that do not ascend, on the GPU against the FP64 oracle.

An end before its begin is an empty sequence, and any offsets give each
sequence its own rows and states, whether or not the batch is one that is cut
into segments.  Tolerances are those of test_gpu_linear.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import gated_deltanet_recurrence_delta_amd as gdn  # noqa: E402
from test_gpu_linear import check, make  # noqa: E402

pytestmark = pytest.mark.gpu

FILL = 777.0
REVERSED_65 = [256, 0] + list(range(10, 10 * 64 + 1, 10))  # no row twice


def run(c, cu):
    """Every output, those of rows over a fill that has to stay where no sequence is."""
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    T = c["q"].shape[0]
    out = torch.full_like(c["v"], FILL)
    hT = torch.full((len(cu) - 1, *c["q"].shape[1:], c["v"].shape[-1]), FILL, device="cuda")
    gdn.linear_fwd(c["q"], c["k"], c["v"], c["g"], c["h0"], cut, out=out, hT=hT)
    got = dict(out=out, hT=hT, dh0=torch.full_like(hT, FILL),
               **{n: torch.full_like(c[n[1]], FILL) for n in ("dq", "dk", "dv")})
    H, dk = c["q"].shape[1:]
    dv, dtype = c["v"].shape[-1], gdn.GDN_BF16 if c["q"].dtype == torch.bfloat16 else gdn.GDN_F32
    size = gdn.gdn_linear_workspace_size(len(cu) - 1, T, H, dk, dv, 1, dtype, True)
    ws = torch.empty(max(1, size), dtype=torch.uint8, device="cuda")
    ptr = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
    rc = gdn.gdn_linear_bwd(*(ptr(c[n]) for n in ("q", "k", "v", "g", "h0")), cut.data_ptr(), ptr(c["dout"]),
                            ptr(c["dhT"]), *(got[n].data_ptr() for n in ("dq", "dk", "dv", "dh0")), len(cu) - 1, T, H,
                            dk, dv, torch.cuda.current_stream().cuda_stream, dtype, ws.data_ptr(), ws.numel())
    assert rc == 0
    inside = torch.zeros(T, dtype=torch.bool, device="cuda")
    at = [min(max(x, 0), T) for x in cu]
    for b, e in zip(at, at[1:]):
        inside[b:e] = True
    torch.cuda.synchronize()
    for n in ("out", "dq", "dk", "dv"):
        assert bool((got[n][~inside] == FILL).all()), n
        got[n] = torch.where(inside[:, None, None], got[n], 0)
    return got, at


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 32), (128, 128)])
@pytest.mark.parametrize("cu,T", [([9, 3, 30], 90), ([9, 3, 300], 1300), ([700, 1300, 0, 700], 1300),
                                  ([-5, 1000, 1400], 1300), ([1300, 600, 600, 0], 1300), (REVERSED_65, 1000)])
def test_offsets_that_fall(dtype, dk, dv, cu, T):
    """Each sequence's rows and states; an empty sequence hands its state on in both directions."""
    c = make(len(cu) + T, dtype, T, 1, dk, dv, len(cu) - 1, packed=True, slow=True)
    if T == 1300:
        assert gdn.gdn_linear_workspace_size(len(cu) - 1, T, 1, dk, dv, 1, 1) > 0  # a batch that is cut
    got, at = run(c, cu)
    check(got, c, dtype, at)
    for n, (b, e) in enumerate(zip(at, at[1:])):
        if e <= b:
            assert torch.equal(got["hT"][n], c["h0"][n]) and torch.equal(got["dh0"][n], c["dhT"][n])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("between", [[], [0] * 70])
def test_sequences_that_overlap(dtype, between):
    """The same rows in two sequences: without states both write the same values, and each has its own hT and dh0."""
    T = 2048
    cu = [0, T, *between, 0, T]
    c = make(1, dtype, T, 2, 64, 64, len(cu) - 1, h0=False, packed=True, slow=True)
    got, at = run(c, cu)
    check(got, c, dtype, at)
    for n in ("hT", "dh0"):
        assert torch.equal(got[n][0], got[n][-1]) and not bool(got[n][1].any())
    # with states of their own, the rows race and the states do not
    c["h0"] = torch.from_numpy(np.random.default_rng(2).standard_normal(got["hT"].shape).astype(np.float32)).cuda()
    got, at = run(c, cu)
    check(dict(hT=got["hT"], dh0=got["dh0"]), c, dtype, at)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 32)])
def test_a_graph_takes_each_replays_offsets(dk, dv):
    """Captured with one set of offsets, replayed with others: ascending, falling, with rows of no sequence."""
    T, some = 1500, [[0, 700, 1500, 1500], [0, 0, 1, 1500], [600, 1500, 0, 600], [5, 400, 400, 1490], [1500, 0, 0, 900]]
    c = make(dk + dv, "bf16", T, 2, dk, dv, 3, packed=True, slow=True)
    assert gdn.gdn_linear_workspace_size(3, T, 2, dk, dv, 1, 1) > 0
    cu = torch.tensor(some[0], dtype=torch.int32, device="cuda")

    def call(cu):
        out, hT = gdn.linear_fwd(c["q"], c["k"], c["v"], c["g"], c["h0"], cu)
        return dict(out=out, hT=hT, **gdn.linear_bwd(c["q"], c["k"], c["v"], c["g"], c["dout"], c["h0"], cu, dhT=c["dhT"]))

    call(cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(cu)
    for at in some[1:] + some:
        cu.copy_(torch.tensor(at, dtype=torch.int32))
        graph.replay()
        want = call(cu)
        torch.cuda.synchronize()
        inside = torch.zeros(T, dtype=torch.bool, device="cuda")
        for b, e in zip(at, at[1:]):
            inside[b:e] = True
        for n in got:
            x, y = (got[n], want[n]) if n in ("hT", "dh0") else (got[n][inside], want[n][inside])
            assert torch.equal(x, y), (at, n)  # rows of no sequence hold what the graph's memory held
