"""Pins of the oracle of convolution, selective scan and norms: closed forms,
and its gradients against central differences."""
import numpy as np
import pytest

from oracle import block


def _rng(seed):
    return np.random.default_rng(seed)


def _close(a, b, tol=1e-9):
    a, b = np.asarray(a), np.asarray(b)
    assert a.shape == b.shape and np.all(np.abs(a - b) <= tol * (1 + np.abs(b)))


def _differences(loss, args, name, grad, seed, h=1e-5):
    """Along random directions; a smooth loss' central difference is off by h^2 and by 2^-53 / h."""
    r = _rng(seed)
    for _ in range(4):
        d = r.standard_normal(args[name].shape)
        diff = (loss(**{**args, name: args[name] + h * d}) - loss(**{**args, name: args[name] - h * d})) / (2 * h)
        assert abs(diff - np.sum(grad * d)) <= 1e-7 * (1 + abs(diff)), name


def _conv_case(seed, T=6, D=3, W=4):
    r = _rng(seed)
    return dict(x=r.standard_normal((T, D)), w=r.standard_normal((D, W)), bias=r.standard_normal(D),
                h0=r.standard_normal((W - 1, D)))


def test_convolution_is_a_convolution():
    for W in (2, 3, 4):
        for T in (0, 1, 2, 9):
            c = _conv_case(W, T=T, W=W)
            out, hT, _, _ = block.conv(**c, silu=False)
            line = np.concatenate([c["h0"], c["x"]])
            for d in range(3):
                want = np.convolve(line[:, d], c["w"][d, ::-1], "valid") if T else np.zeros(0)
                _close(out[:, d], want + (c["bias"][d] if T else 0), 1e-13)
            _close(hT, line[len(line) - (W - 1):], 0)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("T", [1, 2, 6])
def test_convolution_gradients(silu, T):
    c = _conv_case(5, T=T)
    r = _rng(6)
    dout, dhT = r.standard_normal(c["x"].shape), r.standard_normal(c["h0"].shape)

    def loss(**a):
        out, hT, _, _ = block.conv(**a, silu=silu)
        return np.sum(out * dout) + np.sum(hT * dhT)

    dx, dw, db, dh0, _ = block.conv_bwd(**c, silu=silu, dout=dout, dhT=dhT)
    for name, g in (("x", dx), ("w", dw), ("bias", db), ("h0", dh0)):
        _differences(loss, c, name, g, 7)


def _ssm_case(seed, T=5, D=4, G=2, N=3):
    r = _rng(seed)
    return dict(x=r.standard_normal((T, D)), dt=r.uniform(0, 1, (T, D)), b=r.standard_normal((T, G, N)),
                c=r.standard_normal((T, G, N)), A_log=r.standard_normal((D, N)), D=r.standard_normal(D),
                z=r.standard_normal((T, D)), dt_bias=r.uniform(0, 0.5, D), h0=r.standard_normal((D, N)))


def test_scan_of_one_token_and_split():
    c = _ssm_case(1, T=1)
    f = block.ssm(**c, soft=True)
    s = np.log1p(np.exp(c["dt"][0] + c["dt_bias"]))
    h = np.exp(-s[:, None] * np.exp(c["A_log"])) * c["h0"] + (s * c["x"][0])[:, None] * c["b"][0][[0, 0, 1, 1]]
    y = np.sum(h * c["c"][0][[0, 0, 1, 1]], -1) + c["D"] * c["x"][0]
    _close(f["hT"], h, 1e-13)
    _close(f["out"][0], y * c["z"][0] / (1 + np.exp(-c["z"][0])), 1e-13)
    c = _ssm_case(2)
    whole = block.ssm(**c, soft=False)
    at = lambda s: {n: c[n][s] if n in ("x", "dt", "b", "c", "z") else c[n] for n in c}  # noqa: E731
    first = block.ssm(**at(slice(0, 2)), soft=False)
    rest = block.ssm(**{**at(slice(2, 5)), "h0": first["hT"]}, soft=False)
    _close(np.concatenate([first["out"], rest["out"]]), whole["out"], 1e-13)
    _close(rest["hT"], whole["hT"], 1e-13)


def test_scan_without_decay_is_a_sum():
    c = _ssm_case(3, G=1)
    c["A_log"][:] = -np.inf
    f = block.ssm(**c, soft=False)
    s = c["dt"] + c["dt_bias"]
    _close(f["hT"], c["h0"] + np.einsum("td,tn->dn", s * c["x"], c["b"][:, 0]), 1e-13)


@pytest.mark.parametrize("soft", [False, True])
@pytest.mark.parametrize("name", ["x", "dt", "b", "c", "A_log", "D", "z", "dt_bias", "h0"])
def test_scan_gradients(soft, name):
    c = _ssm_case(4)
    r = _rng(5)
    dout, dhT = r.standard_normal(c["x"].shape), r.standard_normal(c["h0"].shape)

    def loss(**a):
        f = block.ssm(**a, soft=soft)
        return np.sum(f["out"] * dout) + np.sum(f["hT"] * dhT)

    g = block.ssm_bwd(**c, soft=soft, dout=dout, dhT=dhT)
    _differences(loss, c, name, g["d" + name], 6)
    assert np.all(np.abs(g["d" + name]) <= g["md" + name] * (1 + 1e-12))


def _angles(P, rot):
    a = np.arange(P)[:, None] * 10.0 ** -np.arange(rot // 2)
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_adds_angles(interleaved):
    r = _rng(8)
    y = r.standard_normal((3, 2, 8))
    cos, sin = _angles(30, 6)
    at = np.array([2, 5, 9])
    once = block.rotate(y, cos[at], sin[at], interleaved)
    _close(np.sum(once ** 2, -1), np.sum(y ** 2, -1), 1e-13)
    _close(block.rotate(once, cos[at + 3], sin[at + 3], interleaved),
           block.rotate(y, cos[2 * at + 3], sin[2 * at + 3], interleaved), 1e-13)
    _close(block.rotate(once, cos[at], sin[at], interleaved, back=True), y, 1e-13)
    assert np.array_equal(once[..., 6:], y[..., 6:])


@pytest.mark.parametrize("l2", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_gradients(l2, interleaved):
    r = _rng(9)
    c = dict(x=r.standard_normal((4, 3, 8)), w=r.standard_normal(8))
    cos, sin = _angles(6, 4)
    pos, dy = np.array([0, 5, -1, 3]), r.standard_normal((4, 3, 8))
    how = dict(cos=cos, sin=sin, pos=pos, l2=l2, eps=0.01, interleaved=interleaved)
    y, m = block.norm(**c, **how)
    assert np.all(y[2] == 0) and np.all(np.abs(y) <= m * (1 + 1e-12))
    dx, dw, mdx, mdw = block.norm_bwd(**c, **how, dy=dy)
    assert np.all(np.abs(dx) <= mdx * (1 + 1e-12)) and np.all(np.abs(dw) <= mdw * (1 + 1e-12))

    def loss(**a):
        return np.sum(block.norm(**a, **how)[0] * dy)

    _differences(loss, c, "x", dx, 10)
    _differences(loss, c, "w", dw, 11)


def test_unit_rows():
    x = _rng(12).standard_normal((5, 2, 16))
    y, _ = block.norm(x, None, None, None, None, True, 0.0, False)
    _close(np.sum(y ** 2, -1), np.ones((5, 2)), 1e-13)
    y, _ = block.norm(x, None, None, None, None, False, 0.0, False)
    _close(np.mean(y ** 2, -1), np.ones((5, 2)), 1e-13)
