"""Host side of convolution, selective scan and norms: the headers' functions
are exported, bad calls are refused before anything is launched, and the
binding's checks of tensors."""
import ctypes
import os
import re

import pytest

import gated_deltanet_recurrence_delta_amd as gdn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED = 0, -1, -2
# Aligned dummy device addresses, far apart: validation never reads them.
NAMES = ("x w bias h0 cu_seqlens out hT dout dhT dx dw dbias dh0 pool slots workspace dt b c A_log Dskip z dt_bias ddt "
         "db dc dA_log dD dz ddt_bias q k cos sin pos wq wk qo ko dqo dko dq dk dwq dwk").split()
A = {n: (i + 1) << 40 for i, n in enumerate(NAMES)}


def test_headers_are_exported():
    lib = ctypes.CDLL(gdn.lib_path())
    want = {"gdn_conv.h": ["gdn_conv_bwd", "gdn_conv_fwd", "gdn_conv_fwd_pool", "gdn_conv_workspace_size"],
            "gdn_ssm.h": ["gdn_ssm_bwd", "gdn_ssm_fwd", "gdn_ssm_fwd_recurrent_pool", "gdn_ssm_workspace_size"],
            "gdn_qk_norm.h": ["gdn_qk_norm_bwd", "gdn_qk_norm_fwd", "gdn_qk_norm_workspace_size"]}
    for header, names in want.items():
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
        assert sorted(set(re.findall(r"\b(gdn_\w+)\s*\(", text))) == names
        for name in names:
            assert hasattr(lib, name) and name in gdn.__all__ and callable(getattr(gdn, name))
    for name in ("conv_fwd", "conv_bwd", "conv_fwd_pool", "causal_conv", "ssm_fwd", "ssm_bwd", "ssm_fwd_recurrent_pool",
                 "selective_scan", "qk_norm_fwd", "qk_norm_bwd", "qk_norm"):
        assert name in gdn.__all__ and callable(getattr(gdn, name))


def _args(names, given, **kw):
    a = {n: A[n] for n in names.split()}
    a.update(given)
    a.update(kw)
    return a


_CONV = dict(B=0, T=8, D=32, W=4, stream=None, dtype=1, flags=1, h0=0, cu_seqlens=0)
_SSM = dict(B=0, T=8, D=32, G=2, N=16, stream=None, dtype=1, flags=1, h0=0, cu_seqlens=0)
_NORM = dict(B=1, T=0, Hq=2, Hk=1, d=64, rot=16, P=8, eps=1e-6, stream=None, dtype=1, flags=0)
BIG = dict(workspace_bytes=1 << 38)


def conv(**kw):
    return gdn.gdn_conv_fwd(**_args("x w bias out hT", _CONV, **kw))


def conv_pool(**kw):
    kw = {n: v for n, v in kw.items() if n not in ("h0", "hT")}
    a = _args("x w bias pool slots out", dict(_CONV, nslots=4), **kw)
    a.pop("h0")
    return gdn.gdn_conv_fwd_pool(**a)


def conv_bwd(**kw):
    return gdn.gdn_conv_bwd(**_args("x w bias dout dx dw dbias workspace", dict(_CONV, **BIG, dhT=0, dh0=0), **kw))


_IN = "x dt b c A_log Dskip z dt_bias"


def ssm(**kw):
    return gdn.gdn_ssm_fwd(**_args(_IN + " out hT workspace", dict(_SSM, **BIG), **kw))


def ssm_pool(**kw):
    a = _args(_IN + " pool slots out", dict(_SSM, nslots=4), **kw)
    a.pop("h0")
    return gdn.gdn_ssm_fwd_recurrent_pool(**a)


def ssm_bwd(**kw):
    return gdn.gdn_ssm_bwd(**_args(_IN + " dout dx ddt db dc dA_log dD dz ddt_bias workspace",
                                   dict(_SSM, **BIG, dhT=0, dh0=0), **kw))


def norm(**kw):
    return gdn.gdn_qk_norm_fwd(**_args("q k cos sin pos wq wk qo ko", _NORM, **kw))


def norm_bwd(**kw):
    return gdn.gdn_qk_norm_bwd(**_args("q k cos sin pos wq wk dqo dko dq dk dwq dwk workspace", dict(_NORM, **BIG), **kw))


# the calls that launch nothing without sequences (the backward ones still clear the parameters' gradients)
@pytest.mark.parametrize("call", [conv, conv_pool, ssm, ssm_pool, norm])
def test_nothing_to_do(call):
    assert call() == OK


@pytest.mark.parametrize("call", [conv, conv_pool, conv_bwd, ssm, ssm_pool, ssm_bwd, norm, norm_bwd])
def test_types_and_flags(call):
    for kw in (dict(dtype=2), dict(dtype=-1), dict(flags=4), dict(flags=-1), dict(B=-1), dict(T=-1)):
        assert call(**kw) == INVALID, kw


@pytest.mark.parametrize("call", [conv, conv_pool, conv_bwd])
def test_conv_sizes(call):
    for kw in (dict(D=0), dict(W=0), dict(B=1 << 16, T=1 << 16), dict(B=1 << 15, T=(1 << 15) + 1), dict(D=1 << 20), dict(B=1 << 24, T=1)):
        assert call(**kw) == INVALID, kw
    for W in (1, 5, 100):
        assert call(W=W) == UNSUPPORTED, W


@pytest.mark.parametrize("call", [ssm, ssm_pool, ssm_bwd])
def test_ssm_sizes(call):
    for kw in (dict(D=0), dict(G=0), dict(N=0), dict(D=33), dict(B=1 << 16, T=1 << 16), dict(D=1 << 20),
               dict(B=1 << 24, T=1), dict(B=1 << 20, T=1, D=1 << 10)):
        assert call(**kw) == INVALID, kw
    for N in (8, 24, 128):
        assert call(N=N) == UNSUPPORTED, N


@pytest.mark.parametrize("call", [norm, norm_bwd])
def test_norm_sizes(call):
    for kw in (dict(Hq=0), dict(Hk=0), dict(Hq=65536), dict(d=0), dict(rot=-2), dict(rot=3), dict(rot=66), dict(P=0),
               dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(cos=0), dict(sin=0),
               dict(B=1 << 16, T=1 << 16), dict(B=1 << 15, T=1 << 15, Hq=65535)):
        assert call(**kw) == INVALID, kw
    for d in (16, 48, 96, 512):
        assert call(d=d) == UNSUPPORTED, d
    assert norm(rot=0, P=0, cos=0, sin=0, pos=0) == OK


@pytest.mark.parametrize("call,kw,names", [
    (conv, {}, "x w out hT"), (conv_pool, {}, "x w out pool slots"), (conv_bwd, {}, "x w dout dx dw workspace"),
    (ssm, dict(T=400), "x dt b c A_log out hT workspace"), (ssm_pool, {}, "x dt b c A_log out pool slots"),
    (ssm_bwd, {}, "x dt b c A_log dout dx ddt db dc dA_log workspace"), (norm, dict(T=8), "q k qo ko"),
    (norm_bwd, dict(T=8), "q k dqo dko dq dk workspace")])
def test_missing_and_misaligned_pointers(call, kw, names):
    for n in names.split():
        assert call(**{**kw, "B": 1, n: 0}) == INVALID, n
        assert call(**{**kw, "B": 1, n: A[n] + (2 if n == "slots" else 8)}) == INVALID, n


@pytest.mark.parametrize("call,names", [
    (conv, "bias h0"), (conv_bwd, "bias h0 dhT dbias dh0"), (ssm, "Dskip z dt_bias h0"),
    (ssm_bwd, "Dskip z dt_bias h0 dhT dD dz ddt_bias dh0"), (norm, "cos sin wq wk"), (norm_bwd, "wq wk dwq dwk")])
def test_misaligned_options(call, names):
    for n in names.split():
        assert call(B=1, **{n: A[n] + 8}) == INVALID, n
    if call not in (norm, norm_bwd):
        assert call(B=1, cu_seqlens=A["cu_seqlens"] + 2) == INVALID
    else:
        assert call(T=1, pos=A["pos"] + 2) == INVALID


def test_overlapping_outputs():
    b = 8 * 32 * 2  # bytes of 8 rows of 32 channels
    for call in (conv, ssm):
        assert call(B=1, out=A["x"]) == INVALID
        assert call(B=1, out=A["x"] + b - 16) == INVALID
        assert call(B=1, hT=A["out"] + b - 16) == INVALID
        assert call(B=1, h0=A["hT"] + 16) == INVALID  # a shifted state; h0 == hT alone is in place
    for call in (conv_pool, ssm_pool):
        assert call(B=1, out=A["x"]) == INVALID
        assert call(B=1, out=A["pool"]) == INVALID
        assert call(B=1, pool=A["x"] + b - 16) == INVALID
        assert call(B=1, nslots=-1) == INVALID
    for call in (conv_bwd, ssm_bwd):
        assert call(B=1, dx=A["dout"]) == INVALID
        assert call(B=1, dx=A["x"] + b - 16) == INVALID
        assert call(B=1, dh0=A["h0"], h0=A["h0"]) == INVALID
        assert call(B=1, workspace=A["x"]) == INVALID
    assert ssm_bwd(B=1, db=A["dc"]) == INVALID
    assert ssm_bwd(B=1, dh0=A["dhT"] + 16, dhT=A["dhT"]) == INVALID
    assert conv_bwd(B=1, dh0=A["dhT"], dhT=A["dhT"]) == INVALID
    assert ssm_bwd(B=1, z=0) == INVALID  # a gate's gradient without a gate
    for call in (norm, norm_bwd):
        y = "qo" if call is norm else "dq"
        assert call(T=8, **{y: A["q"]}) == INVALID
        assert call(T=8, **{y: A["k"]}) == INVALID
        assert call(T=8, **{y: A["cos"]}) == INVALID
    assert norm(T=8, qo=A["ko"]) == INVALID


def test_workspaces():
    size = gdn.gdn_conv_workspace_size
    need = size(2, 100, 64, 4, 0, 1)
    assert need > 0 and conv_bwd(B=2, T=100, D=64, workspace_bytes=need - 1) == INVALID
    assert size(0, 100, 64, 4, 0, 1) == 0 and size(1, 1, 0, 4, 0, 1) == INVALID and size(1, 1, 8, 5, 0, 1) == UNSUPPORTED
    # some hundredth of the rows' bytes, however many rows
    assert size(8, 4096, 1280, 4, 0, 1) < 8 * 4096 * 1280 * 2 / 2
    size = gdn.gdn_ssm_workspace_size
    assert size(1, 64, 256, 1, 16, 0, 1) == 0  # too short
    assert size(512, 4096, 1280, 1, 16, 0, 1) == 0  # enough channels and sequences
    for back in (False, True):
        need = size(1, 4096, 1280, 1, 16, 0, 1, back)
        assert need > 0
        call = ssm_bwd if back else ssm
        assert call(B=1, T=4096, D=1280, G=1, workspace_bytes=need - 1) == INVALID
    assert size(1, 4096, 33, 2, 16, 0, 1) == INVALID and size(1, 4096, 32, 2, 8, 0, 1) == UNSUPPORTED
    assert gdn.gdn_qk_norm_workspace_size(0, 5, 1, 1, 64) == 0
    assert gdn.gdn_qk_norm_workspace_size(1, 5, 1, 1, 60) == UNSUPPORTED
    need = gdn.gdn_qk_norm_workspace_size(2, 500, 16, 4, 128)
    assert need > 0 and norm_bwd(B=2, T=500, Hq=16, Hk=4, d=128, workspace_bytes=need - 1) == INVALID


@pytest.mark.parametrize("packed", [0, 1])
def test_workspace_sizes_hold_over_the_range(packed):
    """Never negative for sizes that are taken, and no overflow at the largest."""
    for B, T, D in ((1, 1, 1), (1, 2 ** 30, 1), (300, 3500000 if not packed else 2 ** 30, 4), (2 ** 20, 2, 64)):
        assert gdn.gdn_conv_workspace_size(B, T, D, 4, packed, 0) > 0
        for back in (False, True):
            assert gdn.gdn_ssm_workspace_size(B, T, D, 1, 16, packed, 0, back) >= 0


@pytest.mark.parametrize("D,G,N", [(1280, 1, 16), (1280, 1, 64), (640, 2, 32), (64, 1, 16), (33, 1, 64)])
@pytest.mark.parametrize("T", [3000, 131072, 2 ** 30])
def test_packed_scans_are_cut_however_many_sequences(D, G, N, T):
    """One sequence may be nearly all of the rows: no segment is longer than one and a half of a wave's even shares of
    them (or 64 rows), seen from the states that the workspace holds."""
    waves = {16: 5120, 32: 4096, 64: 2048}[N]  # that the device holds at once
    tiles = G * -(-(D // G) // 64)
    longest = max(64, 1.5 * T * tiles / waves) + 4  # (a multiple of 4 rows)
    for B in (1, 2, 40, 100, 300, 511, 512, 1000, 5000, 60000):
        need = gdn.gdn_ssm_workspace_size(B, T, D, G, N, 1, 1)
        segments = need // (4 * D * (N + 1))  # a state and a sum each; rows / L, and one for each sequence
        assert segments - B >= int(T / longest) > 0, (B, segments)


# ------------------------------------------------- the binding's own checks --

def test_python_checks():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 4)
    bad = [(TypeError, dict(x=x.double())), (ValueError, dict(x=x[0])), (ValueError, dict(w=w.bfloat16())),
           (ValueError, dict(w=w[:7])), (ValueError, dict(bias=torch.zeros(7))), (ValueError, dict(h0=torch.zeros(2, 4, 8))),
           (ValueError, dict(out=torch.zeros(2, 5, 8, dtype=torch.bfloat16))),
           (TypeError, dict(cu_seqlens=torch.zeros(3))), (ValueError, dict(cu_seqlens=torch.zeros(3, dtype=torch.int32))),
           (ValueError, dict())]  # not on a GPU
    for err, kw in bad:
        with pytest.raises(err):
            gdn.conv_fwd(**{"x": x, "w": w, **kw})
    with pytest.raises(ValueError, match="slots"):
        gdn.conv_fwd_pool(x, w, torch.zeros(4, 3, 8), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="pool"):
        gdn.conv_fwd_pool(x, w, torch.zeros(4, 2, 8), torch.zeros(2, dtype=torch.int32))
    k, A_log = torch.zeros(2, 5, 2, 16), torch.zeros(8, 16)
    good = dict(x=x, dt=x, b=k, c=k, A_log=A_log)
    bad = [(ValueError, dict(dt=x[:1])), (ValueError, dict(dt=x.bfloat16())), (ValueError, dict(b=k[0])),
           (ValueError, dict(c=k[:, :, :1])), (ValueError, dict(b=torch.zeros(2, 5, 3, 16))),
           (ValueError, dict(A_log=A_log.double())), (ValueError, dict(D=torch.zeros(9))),
           (ValueError, dict(z=x[:, :4])), (ValueError, dict(dt_bias=torch.zeros(8, 1))),
           (ValueError, dict(h0=torch.zeros(2, 8, 32))), (ValueError, dict())]
    for err, kw in bad:
        with pytest.raises(err):
            gdn.ssm_fwd(**{**good, **kw})
    with pytest.raises(ValueError, match="dout"):
        gdn.ssm_bwd(*good.values(), dout=x[:1])
    q, kk, cos = torch.zeros(2, 5, 4, 64), torch.zeros(2, 5, 2, 64), torch.zeros(9, 16)
    bad = [(ValueError, dict(k=kk[:1])), (TypeError, dict(k=kk.bfloat16())), (ValueError, dict(norm="l1")),
           (ValueError, dict(cos=cos)), (ValueError, dict(cos=cos, sin=cos[:8])), (ValueError, dict(cos=cos[0], sin=cos[0])),
           (ValueError, dict(cos=torch.zeros(9, 33), sin=torch.zeros(9, 33))), (ValueError, dict(wq=torch.zeros(32))),
           (ValueError, dict(cos=cos, sin=cos, pos=torch.zeros(2, 5))),
           (ValueError, dict(q=q[0], k=kk[0], cos=cos, sin=cos)), (ValueError, dict())]
    for err, kw in bad:
        with pytest.raises(err):
            gdn.qk_norm_fwd(**{"q": q, "k": kk, **kw})


def test_python_tables_get_no_gradient():
    torch = pytest.importorskip("torch")
    q, cos = torch.zeros(2, 5, 4, 64), torch.zeros(9, 16, requires_grad=True)
    with pytest.raises(ValueError, match="constant"):
        gdn.qk_norm(q, q, cos, cos)
