"""Slot moves of more than one launch on the GPU: full launches of single
pairs, then a list longer than a launch."""
import pytest

torch = pytest.importorskip("torch")
import gated_deltanet_recurrence_delta_amd as gdn  # noqa: E402
from test_gpu_pool import indexed  # noqa: E402
from test_move_plan import chain, cycle, singles, tree  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", [319, 320, 321, 640])
@pytest.mark.parametrize("kind", [chain, cycle, tree])
def test_a_long_list_behind_full_launches(first, kind):
    s, d, at = singles(first, 0)
    s2, d2, at = kind(330, at)
    pool = torch.randn(2, at, 20, generator=torch.Generator().manual_seed(first)).cuda()
    want = indexed(pool, s + s2, d + d2, 1)
    gdn.state_move(pool, s + s2, d + d2, dim=1)
    assert torch.equal(pool.cpu(), want)
