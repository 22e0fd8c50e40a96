"""A pool of states whose move fails keeps its books: nobody holds slots that
nobody was given, and nothing has moved."""
import pytest

import gated_deltanet_recurrence_delta_amd as gdn
from gated_deltanet_recurrence_delta_amd import pool as gdn_pool

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("layers", [None, 2])
def test_slots_come_back_when_a_move_fails(monkeypatch, layers):
    p = gdn.StatePool(6, 1, 2, 2, layers=layers, device="cpu")
    monkeypatch.setattr(gdn_pool, "state_move", lambda pool, src, dst, dim=0, stream=None: pool)
    a, b, c = p.alloc(3)
    p.free([a])

    def fails(*_, **__):
        raise gdn.GdnError(-3, "launch", "gdn_state_move")

    with monkeypatch.context() as m:
        m.setattr(gdn_pool, "state_move", fails)
        for call in (lambda: p.alloc(2), lambda: p.fork(b, 3), lambda: p.compact(), lambda: p.copy([b], [c])):
            with pytest.raises(gdn.GdnError):
                call()
            assert p.live == [b, c] and p.free_slots == 4
    assert p.alloc(4) == [a, 3, 4, 5] and p.free_slots == 0  # the lowest first, as if nothing had been
