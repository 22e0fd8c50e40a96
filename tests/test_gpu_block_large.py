"""Tensors of more than 2^31 elements: their last rows equal those of a small
call on the same rows."""
import pytest

from block_case import f64, within

torch = pytest.importorskip("torch")
import gated_deltanet_recurrence_delta_amd as gdn  # noqa: E402

pytestmark = pytest.mark.gpu
ROWS, D, TAIL = (1 << 20) + 77, 2056, 150


def big(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")
    x[-2 * TAIL:] = (torch.randn(2 * TAIL, *shape[1:], generator=g, device="cuda") * scale).to(torch.bfloat16)
    return x


@pytest.fixture(autouse=True)
def _room():
    yield
    torch.cuda.empty_cache()


def test_convolution():
    x, w = big(1, ROWS, D), torch.randn(D, 4, device="cuda")
    cu = torch.tensor([0, ROWS], dtype=torch.int32, device="cuda")
    out, hT = gdn.conv_fwd(x, w, cu_seqlens=cu)
    small, h = gdn.conv_fwd(x[None, -TAIL:].contiguous(), w, h0=x[None, -TAIL - 3:-TAIL].contiguous())
    assert torch.equal(out[-TAIL:], small[0]) and torch.equal(hT, h)
    g = gdn.conv_bwd(x, w, x, cu_seqlens=cu)
    s = gdn.conv_bwd(x[None, -TAIL:].contiguous(), w, x[None, -TAIL:].contiguous(),
                     h0=x[None, -TAIL - 3:-TAIL].contiguous())
    assert torch.equal(g["dx"][-TAIL + 3:], s["dx"][0, 3:])


def test_scan():
    """The last sequence of a packed batch; it is cut elsewhere in the small call, so that fp32 sums of some 200
    tokens differ: 2^-12 of the outputs' scale, after 2^-8 for bf16."""
    N = 16
    cu = torch.tensor([0, ROWS - TAIL, ROWS], dtype=torch.int32, device="cuda")
    x, dt, dout = big(2, ROWS, D), big(3, ROWS, D, scale=0.3), big(4, ROWS, D)
    b, c = big(5, ROWS, 1, N), big(6, ROWS, 1, N)
    A_log, bias = torch.log(torch.arange(1, N + 1.0, device="cuda")).repeat(D, 1), torch.full((D,), -3.0, device="cuda")
    out, hT = gdn.ssm_fwd(x, dt, b, c, A_log, dt_bias=bias, cu_seqlens=cu)
    last = lambda t: t[None, -TAIL:].contiguous()  # noqa: E731
    small = [last(t) for t in (x, dt, b, c)]
    o, h = gdn.ssm_fwd(*small, A_log, dt_bias=bias)
    tol = lambda t: 2.0 ** -8 * abs(f64(t)) + 2.0 ** -12 * float(t.abs().max())  # noqa: E731
    within("out", out[-TAIL:], f64(o[0]), tol(o[0]))
    within("hT", hT[1], f64(h[0]), tol(h[0]))
    del out, hT
    g = gdn.ssm_bwd(x, dt, b, c, A_log, dout, dt_bias=bias, cu_seqlens=cu)
    s = gdn.ssm_bwd(*small, A_log, last(dout), dt_bias=bias)
    for n in ("dx", "ddt", "db", "dc"):
        within(n, g[n][-TAIL:], f64(s[n][0]), tol(s[n][0]))
    within("dh0", g["dh0"][1], f64(s["dh0"][0]), tol(s["dh0"][0]))


def test_norm():
    rows, H, d = 140000, 64, 256
    q = big(7, rows, H, d)
    k, pos = q[:, :1].contiguous(), torch.arange(rows, dtype=torch.int32, device="cuda") % 50
    a = torch.arange(50, device="cuda")[:, None] / 10 * torch.arange(1, 33, device="cuda")
    how = dict(cos=torch.cos(a), sin=torch.sin(a), wq=torch.rand(d, device="cuda"))
    qo, ko = gdn.qk_norm_fwd(q, k, pos=pos, **how)
    last = lambda t: t[-TAIL:].contiguous()  # noqa: E731
    so, to = gdn.qk_norm_fwd(last(q), last(k), pos=last(pos), **how)
    assert torch.equal(qo[-TAIL:], so) and torch.equal(ko[-TAIL:], to)
    g = gdn.qk_norm_bwd(q, k, qo, ko, pos=pos, **how)
    s = gdn.qk_norm_bwd(last(q), last(k), so, to, pos=last(pos), **how)
    assert torch.equal(g["dq"][-TAIL:], s["dq"]) and torch.equal(g["dk"][-TAIL:], s["dk"])
