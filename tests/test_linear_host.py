"""Host side of linear attention and the state pool: the headers' functions
are exported, bad calls are refused before anything is launched, and a pool's
bookkeeping."""
import ctypes
import os
import random
import re

import pytest

import gated_deltanet_recurrence_delta_amd as gdn
from gated_deltanet_recurrence_delta_amd import pool as gdn_pool

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED = 0, -1, -2
# Aligned dummy device addresses, far apart: validation never reads them.
A = {n: (i + 1) << 40 for i, n in enumerate(
    ["q", "k", "v", "g", "beta", "h0", "cu_seqlens", "out", "hT", "dout", "dhT", "dq", "dk", "dv", "dh0", "pool",
     "slots", "workspace"])}


def test_headers_are_exported():
    lib = ctypes.CDLL(gdn.lib_path())
    want = {"gdn_linear.h": ["gdn_linear_bwd", "gdn_linear_fwd", "gdn_linear_fwd_recurrent",
                             "gdn_linear_workspace_size"],
            "gdn_pool.h": ["gdn_fwd_recurrent_pool", "gdn_linear_fwd_recurrent_pool", "gdn_state_move"]}
    for header, names in want.items():
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
        assert sorted(set(re.findall(r"\b(gdn_\w+)\s*\(", text))) == names
        for name in names:
            assert hasattr(lib, name) and name in gdn.__all__ and callable(getattr(gdn, name))


def _fwd(**kw):
    a = dict(q=A["q"], k=A["k"], v=A["v"], g=A["g"], h0=0, cu_seqlens=0, out=A["out"], hT=A["hT"], B=0, T=8, H=1,
             dk=32, dv=32, stream=None, dtype=1, workspace=0, workspace_bytes=0)
    a.update(kw)
    return gdn.gdn_linear_fwd(**a)


def _rec(**kw):
    a = dict(q=A["q"], k=A["k"], v=A["v"], g=A["g"], h0=0, cu_seqlens=0, out=A["out"], hT=A["hT"], B=0, T=8, H=1,
             dk=32, dv=32, stream=None, dtype=1)
    a.update(kw)
    return gdn.gdn_linear_fwd_recurrent(**a)


def _bwd(**kw):
    a = dict(q=A["q"], k=A["k"], v=A["v"], g=A["g"], h0=0, cu_seqlens=0, dout=A["dout"], dhT=0, dq=A["dq"],
             dk=A["dk"], dv=A["dv"], dh0=0, B=0, T=8, H=1, dk_=32, dv_=32, stream=None, dtype=1, workspace=0,
             workspace_bytes=0)
    if "dk_" not in kw and "dv_" not in kw:
        kw = {{"dk": "dk_", "dv": "dv_"}.get(n, n) if isinstance(x, int) and x < 1 << 40 and n in ("dk", "dv")
              and x != 0 else n: x for n, x in kw.items()}
    a.update(kw)
    return gdn.gdn_linear_bwd(**a)


def _pool(delta, **kw):
    a = dict(q=A["q"], k=A["k"], v=A["v"], g=A["g"], pool=A["pool"], slots=A["slots"], cu_seqlens=0, out=A["out"],
             nslots=4, B=0, T=1, H=1, dk=32, dv=32, stream=None, dtype=1)
    if delta:
        a["beta"] = A["beta"]
    a.update(kw)
    return (gdn.gdn_fwd_recurrent_pool if delta else gdn.gdn_linear_fwd_recurrent_pool)(**a)


CALLS = [_fwd, _rec, _bwd, lambda **kw: _pool(True, **kw), lambda **kw: _pool(False, **kw)]


@pytest.mark.parametrize("call", CALLS)
def test_sizes(call):
    assert call() == OK  # no sequence: nothing to do
    for kw in (dict(B=-1), dict(T=-1), dict(H=0), dict(dtype=2), dict(dtype=-1), dict(H=65536)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(dk=16), dict(dv=256), dict(dk=96)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(dk=-1), dict(dv=-32)):
        assert call(**kw) == INVALID, kw


@pytest.mark.parametrize("call,names", [
    (_fwd, ["q", "k", "v", "g", "out", "hT"]), (_rec, ["q", "k", "v", "g", "out", "hT"]),
    (_bwd, ["q", "k", "v", "g", "dout", "dq", "dk", "dv"]),
    (CALLS[3], ["q", "k", "v", "g", "beta", "out", "pool", "slots"]),
    (CALLS[4], ["q", "k", "v", "g", "out", "pool", "slots"])])
def test_missing_and_misaligned_pointers(call, names):
    for n in names:
        assert call(B=1, **{n: 0}) == INVALID, n
        assert call(B=1, **{n: A[n] + (2 if n in ("g", "beta", "slots") else 8)}) == INVALID, n


def test_overlapping_outputs():
    b = 8 * 32 * 2  # bytes of a tensor of 8 rows
    assert _fwd(B=1, out=A["v"]) == INVALID
    assert _fwd(B=1, out=A["q"] + b - 16) == INVALID
    assert _fwd(B=1, hT=A["out"] + b - 16) == INVALID
    assert _fwd(B=1, h0=A["hT"] + 16) == INVALID  # a shifted state; h0 == hT alone is in place
    assert _rec(B=1, out=A["k"] + b - 16) == INVALID
    assert _rec(B=1, h0=A["hT"] - 16) == INVALID
    assert _bwd(B=1, dq=A["dout"]) == INVALID
    assert _bwd(B=1, dq=A["dk"]) == INVALID
    assert _bwd(B=1, dh0=A["dhT"] + 16, dhT=A["dhT"]) == INVALID
    assert _bwd(B=1, dh0=A["h0"], h0=A["h0"]) == INVALID
    for delta in (False, True):
        assert _pool(delta, B=1, out=A["pool"] + 4 * 32 * 32 * 4 - 16) == INVALID
        assert _pool(delta, B=1, out=A["v"]) == INVALID
        assert _pool(delta, B=1, nslots=-1) == INVALID


def test_workspace():
    size = gdn.gdn_linear_workspace_size
    assert size(64, 4096, 16, 128, 128, 0, 1) == 0  # enough chains: nothing is cut
    assert size(1, 200, 1, 128, 128, 0, 1) == 0  # too short
    need = size(1, 32768, 2, 128, 128, 0, 1)
    assert need > 0 and need % (2 * 128 * 128 * 4) == 0
    assert size(3, 32768, 2, 128, 128, 1, 1) > 0
    assert size(1, 32768, 2, 128, 64, 0, 1, 1) > 0
    # however many sequences: about as many segment states as the device has compute units
    for B in (1, 100, 5000):
        assert 0 <= size(B, 200000, 16, 128, 128, 1, 1) <= 256 * 128 * 128 * 4
    for packed in (0, 1):
        for backward in (0, 1):  # no rows, no sequences
            assert size(3, 0, 2, 128, 64, packed, 1, backward) == 0
            assert size(0, 100, 2, 64, 64, packed, 0, backward) == 0
    assert size(1, 32768, 0, 128, 128, 0, 1) == INVALID
    assert size(1, 32768, 2, 48, 128, 0, 1) == UNSUPPORTED
    a = dict(B=1, T=32768, H=2, dk=128, dv=128)
    assert _fwd(**a, workspace=A["workspace"], workspace_bytes=need - 1) == INVALID
    assert _fwd(**a, workspace=0, workspace_bytes=need) == INVALID
    assert _fwd(**a, workspace=A["workspace"] + 8, workspace_bytes=2 * need) == INVALID
    assert _fwd(**a, workspace=A["q"] + 16, workspace_bytes=need) == INVALID  # over an input
    b = dict(B=1, T=32768, H=2, dk_=128, dv_=128)
    assert _bwd(**b, workspace=A["workspace"], workspace_bytes=size(1, 32768, 2, 128, 128, 0, 1, 1) - 1) == INVALID


def test_rows_beyond_32_bit_offsets_are_refused():
    # 2^23 rows of 2 heads of 128 bf16 values are 2^32 bytes
    assert _fwd(B=1, T=1 << 23, H=2, dk=128, dv=128) == INVALID
    assert _bwd(B=1, T=1 << 23, H=2, dk_=128, dv_=128) == INVALID


def _move(src, dst, n=None, pool=A["pool"], outer=1, slots=8, slot_bytes=64):
    arr = lambda x: (ctypes.c_int32 * max(1, len(x)))(*x)  # noqa: E731
    return gdn.gdn_state_move(pool, outer, slots, slot_bytes, arr(src), arr(dst), len(src) if n is None else n, None)


def test_move_refusals():
    assert _move([], []) == OK
    assert _move([3], [3]) == OK  # a slot onto itself: nothing to do
    for src, dst in (([8], [0]), ([-2], [0]), ([0], [8]), ([0], [-1]), ([0, 1], [2, 2])):
        assert _move(src, dst) == INVALID, (src, dst)
    for kw in (dict(n=-1), dict(outer=-1), dict(slots=-1), dict(slot_bytes=0), dict(slot_bytes=24), dict(pool=0),
               dict(pool=A["pool"] + 8)):
        assert _move([0], [1], **kw) == INVALID, kw


# ---------------------------------------------------------------- python --

def test_python_refusals():
    torch = pytest.importorskip("torch")
    q = torch.zeros(1, 4, 2, 32)
    g = torch.zeros(2)
    for call in (gdn.linear_fwd, gdn.linear_fwd_recurrent, gdn.linear_attention):
        with pytest.raises(ValueError, match="GPU"):
            call(q, q, q, g)
        with pytest.raises(ValueError, match="g must"):
            call(q, q, q, torch.zeros(1, 4, 2))
        with pytest.raises(ValueError, match="no gradient"):
            call(q, q, q, g.clone().requires_grad_())
        with pytest.raises(TypeError):
            call(q.double(), q, q, g)
        with pytest.raises(TypeError):
            call(q, q.bfloat16(), q, g)
        with pytest.raises(ValueError):
            call(q, q[:, :3], q, g)
        with pytest.raises(TypeError):
            call(q[0], q[0], q[0], g, None, torch.tensor([0, 4]))  # int64 offsets
    with pytest.raises(ValueError):
        gdn.linear_bwd(q, q, q, g, q[..., :16])
    with pytest.raises(ValueError):
        gdn.linear_fwd_recurrent_pool(q, q, q, g, torch.zeros(4, 2, 32, 64), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        gdn.linear_fwd_recurrent_pool(q, q, q, g, torch.zeros(4, 2, 32, 32), torch.zeros(1))
    with pytest.raises(ValueError):
        gdn.fwd_recurrent_pool(q, q, q, g, g, torch.zeros(4, 2, 32, 32), torch.zeros(1, dtype=torch.int32))
    pool = torch.zeros(3, 8, 4)
    for src, dst in (([0], [8]), ([8], [0]), ([-2], [0]), ([0, 1], [2, 2]), ([0, 1], [2]), ([1 << 40], [0])):
        with pytest.raises(ValueError):
            gdn.state_move(pool, src, dst, dim=1)
    with pytest.raises(ValueError):
        gdn.state_move(pool, [0], [1], dim=3)
    with pytest.raises(TypeError):
        gdn.state_move(pool, [0.5], [1], dim=1)
    with pytest.raises(ValueError, match="GPU"):
        gdn.state_move(pool, [0], [1], dim=1)


def test_pool_bookkeeping(monkeypatch):
    """Every operation against a model that keeps each user's value."""
    torch = pytest.importorskip("torch")

    def move(pool, src, dst, dim=0, stream=None):
        old = pool.clone()
        for s, d in zip(src, dst):
            pool.select(dim, d).copy_(old.select(dim, s) if s >= 0 else torch.zeros_like(old.select(dim, d)))
        return pool

    monkeypatch.setattr(gdn_pool, "state_move", move)
    rnd = random.Random(0)
    for layers in (None, 2):
        p = gdn.StatePool(9, 1, 2, 2, layers=layers, device="cpu")
        of = {}  # slot -> value
        for step in range(300):
            do = rnd.choice(["alloc", "fork", "copy", "free", "compact", "write"])
            if do == "alloc" and p.free_slots:
                for s in p.alloc(rnd.randint(0, p.free_slots)):
                    of[s] = 0.0
            elif do == "fork" and of and p.free_slots:
                s = rnd.choice(sorted(of))
                for t in p.fork(s, rnd.randint(1, p.free_slots)):
                    of[t] = of[s]
            elif do == "copy" and of:
                dst = rnd.sample(sorted(of), rnd.randint(0, len(of)))
                src = [rnd.choice(sorted(of)) for _ in dst]
                p.copy(src, dst)
                of.update({d: v for d, v in zip(dst, [of[s] for s in src])})
            elif do == "free" and of:
                gone = rnd.sample(sorted(of), rnd.randint(0, len(of)))
                p.free(gone)
                for s in gone:
                    del of[s]
            elif do == "compact":
                moved = p.compact()
                of = {moved.get(s, s): v for s, v in of.items()}
                assert sorted(of) == list(range(len(of)))
            elif do == "write" and of:
                s = rnd.choice(sorted(of))
                of[s] = float(step)
                p.states.select(0 if layers is None else 1, s).fill_(of[s])
            assert p.live == sorted(of) and p.free_slots == 9 - len(of)
            for s, v in of.items():
                assert bool((p.states.select(0 if layers is None else 1, s) == v).all())
    p = gdn.StatePool(3, 1, 2, 2, device="cpu")
    a, b = p.alloc(2)
    for bad in (lambda: p.alloc(2), lambda: p.fork(2), lambda: p.free([a, a]), lambda: p.free([2]),
                lambda: p.copy([a], [2]), lambda: p.copy([a, b], [a])):
        with pytest.raises(ValueError):
            bad()
    assert p.live == [a, b] and p.free_slots == 1
