"""Linear attention with a positive g, against the FP64 oracle: computed as it
stands wherever the states themselves are finite.  Tolerances are those of
test_gpu_linear."""
import pytest

torch = pytest.importorskip("torch")
import gated_deltanet_recurrence_delta_amd as gdn  # noqa: E402
from test_gpu_linear import check, make, run_all  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 32), (128, 128)])
@pytest.mark.parametrize("packed", [False, True])
def test_zeros_before_a_growing_state(dtype, dk, dv, packed):
    """A cut sequence whose state is zero until the last rows: a segment's power is past fp32, 0 is still 0."""
    T, some = 2048, 40
    assert gdn.gdn_linear_workspace_size(1, T, 2, dk, dv, packed, 1) > 0
    c = make(dk + dv, dtype, T, 2, dk, dv, 1, h0=False, packed=packed)
    c["g"].copy_(torch.tensor([0.8, 0.75]))  # over 128 rows e^96 at least, over 64 e^51.2 at most
    rows = (lambda t: t) if packed else (lambda t: t[0])
    rows(c["k"])[:-some] = 0
    rows(c["dout"])[some:] = 0  # and the backward's, until the first
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda") if packed else None
    got = run_all(c, cu)
    assert all(bool(torch.isfinite(x).all()) for x in got.values())
    check(got, c, dtype, [0, T] if packed else None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_growing_state(dtype):
    """Growth that stays finite over every row, in a cut sequence."""
    c = make(3, dtype, 1300, 2, 64, 64, 1)
    c["g"].copy_(torch.tensor([0.03, 0.001]))  # e^39 at the end
    check(run_all(c), c, dtype)
