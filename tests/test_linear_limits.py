"""The largest sizes that linear attention takes: a packed batch is bounded as
the one sequence that it may be."""
import pytest

import gated_deltanet_recurrence_delta_amd as gdn

INVALID = -1


@pytest.mark.parametrize("packed", [0, 1])
@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("dtype,T,H,dk,dv", [(1, 1 << 19, 16, 128, 128), (1, 1 << 19, 16, 32, 128), (0, 1 << 17, 32, 128, 64),
                                             (1, 1 << 25, 1, 32, 32)])
def test_rows_of_two_gib_are_refused(packed, backward, dtype, T, H, dk, dv):
    assert T * H * max(dk, dv) * (2 if dtype == 1 else 4) == 1 << 31
    for B in (1, 40):
        assert gdn.gdn_linear_workspace_size(B, T - 1, H, dk, dv, packed, dtype, backward) >= 0
        assert gdn.gdn_linear_workspace_size(B, T, H, dk, dv, packed, dtype, backward) == INVALID
        rows = (1 << 40, 2 << 40, 3 << 40, 4 << 40, 0, 5 << 40 if packed else 0)
        if backward:
            rc = gdn.gdn_linear_bwd(*rows, 6 << 40, 0, 7 << 40, 8 << 40, 9 << 40, 0, B, T, H, dk, dv, None, dtype, 0, 0)
        else:
            rc = gdn.gdn_linear_fwd(*rows, 6 << 40, 7 << 40, B, T, H, dk, dv, None, dtype, 0, 0)
        assert rc == INVALID
