"""Linear attention on tensors just under the 2 GiB that its row offsets reach,
against the FP64 oracle at both ends.  A fast decay makes an end depend on the
rows near it alone: 236 rows further on e^-236 of a value is left, nothing in
any of the types.  Tolerances are those of test_gpu_linear."""
import pytest

torch = pytest.importorskip("torch")
import gated_deltanet_recurrence_delta_amd as gdn  # noqa: E402
from test_gpu_linear import check  # noqa: E402

pytestmark = pytest.mark.gpu

NEAR, FAR = 64, 300  # rows compared, rows that the oracle sees


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype,H,dk,dv", [("bf16", 64, 128, 128), ("f32", 40, 64, 128), ("bf16", 700, 32, 64)])
def test_both_ends(dtype, H, dk, dv, packed):
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("less than 40 GiB of GPU memory are free")
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    T = ((1 << 31) - 1) // (H * max(dk, dv) * dt.itemsize)
    gen = torch.Generator(device="cuda").manual_seed(H)
    rand = lambda d: torch.randn(T, H, d, generator=gen, device="cuda", dtype=dt)  # noqa: E731
    q, k, v, dout = rand(dk).mul_(dk ** -0.5), rand(dk).mul_(dk ** -0.5), rand(dv), rand(dv)
    g = torch.full((H,), -1.0, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda") if packed else None
    lead = (lambda t: t) if packed else (lambda t: t[None])
    out, hT = gdn.linear_fwd(lead(q), lead(k), lead(v), g, None, cu)
    got = dict(out=out, hT=hT, **gdn.linear_bwd(lead(q), lead(k), lead(v), g, lead(dout), None, cu))
    heads = [0, H // 2, H - 1]
    rows = lambda n, s: got[n][s] if packed else got[n][0, s]  # noqa: E731
    for end in (slice(0, FAR), slice(T - FAR, T)):
        c = {n: t[end][:, heads][None].contiguous() for n, t in (("q", q), ("k", k), ("v", v), ("dout", dout))}
        c.update(g=g[heads], h0=None, dhT=None)
        part = {n: rows(n, end)[:, heads][None].clone() for n in ("out", "dq", "dk", "dv")}
        state = {"dh0" if end.start == 0 else "hT": got["dh0" if end.start == 0 else "hT"][:, heads]}
        # what the window's cut end takes part in is not compared: those rows get the oracle's own values
        near_first = end.start == 0
        for names, keep_first in ((("out", "dq"), True), (("dk", "dv"), False)):
            if keep_first != near_first:
                for n in names:
                    edge = slice(0, FAR - NEAR) if keep_first else slice(NEAR, FAR)
                    part[n][:, edge] = oracle_rows(c, n)[:, edge].to(dt)
        check({**part, **state}, c, dtype)


def oracle_rows(c, name):
    from test_gpu_linear import oracle_of

    return torch.from_numpy(oracle_of(c)[name]).cuda()
