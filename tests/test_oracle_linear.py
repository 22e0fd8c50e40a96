"""Pins of the linear-attention oracle: closed forms, the quadratic form, and
its gradients against central differences."""
import numpy as np
import pytest

from oracle import linear


def _case(seed, B=2, T=7, H=3, dk=4, dv=5):
    r = np.random.default_rng(seed)
    return dict(q=r.standard_normal((B, T, H, dk)), k=r.standard_normal((B, T, H, dk)),
                v=r.standard_normal((B, T, H, dv)), g=-np.exp(r.standard_normal(H)),
                h0=r.standard_normal((B, H, dk, dv)))


def test_one_token():
    c = _case(0, T=1)
    out, hT = linear.fwd(**c)
    a = np.exp(c["g"])[None, :, None, None]
    S = a * c["h0"] + np.einsum("bhi,bhj->bhij", c["k"][:, 0], c["v"][:, 0])
    assert np.allclose(hT, S, atol=1e-14)
    assert np.allclose(out[:, 0], np.einsum("bhi,bhij->bhj", c["q"][:, 0], S), atol=1e-14)


def test_quadratic_form():
    c = _case(1)
    out, _ = linear.fwd(c["q"], c["k"], c["v"], c["g"])
    i = np.arange(7)
    D = np.where(i[:, None] >= i, np.exp(c["g"][:, None, None] * (i[:, None] - i)), 0.0)
    P = np.einsum("bihd,bjhd->bhij", c["q"], c["k"]) * D
    assert np.allclose(out, np.einsum("bhij,bjhd->bihd", P, c["v"]), atol=1e-13)


def test_split_and_forgetting():
    c = _case(2)
    out, hT = linear.fwd(**c)
    cut = lambda s: {n: c[n][:, s] for n in "qkv"}  # noqa: E731
    o1, h1 = linear.fwd(**cut(slice(0, 3)), g=c["g"], h0=c["h0"])
    o2, h2 = linear.fwd(**cut(slice(3, 7)), g=c["g"], h0=h1)
    assert np.allclose(np.concatenate([o1, o2], 1), out, atol=1e-13) and np.allclose(h2, hT, atol=1e-13)
    with np.errstate(invalid="ignore"):
        out, _ = linear.fwd(c["q"], c["k"], c["v"], np.full(3, -np.inf), c["h0"])
    assert np.allclose(out, np.sum(c["q"] * c["k"], -1, keepdims=True) * c["v"], atol=1e-13)


@pytest.mark.parametrize("name", ["q", "k", "v", "h0"])
def test_gradients_against_differences(name):
    c = _case(3)
    r = np.random.default_rng(4)
    dout, dhT = r.standard_normal(c["v"].shape), r.standard_normal(c["h0"].shape)
    grad = linear.bwd(c["q"], c["k"], c["v"], c["g"], dout, c["h0"], dhT)["d" + name]

    def loss(x):
        out, hT = linear.fwd(**{**c, name: x})
        return np.sum(out * dout) + np.sum(hT * dhT)

    for _ in range(5):
        d = r.standard_normal(c[name].shape)
        # the loss is a polynomial of degree one in each single input: differences are exact up to rounding
        diff = (loss(c[name] + d) - loss(c[name] - d)) / 2
        assert abs(diff - np.sum(grad * d)) <= 1e-11 * np.sum(np.abs(grad * d))


def test_empty_sequence_hands_the_state_on():
    c = _case(5, T=0)
    out, hT = linear.fwd(**c)
    assert out.shape[1] == 0 and np.array_equal(hT, c["h0"])
    r = linear.bwd(c["q"], c["k"], c["v"], c["g"], out, c["h0"], c["h0"])
    assert np.array_equal(r["dh0"], c["h0"])


def test_delta_rule_is_the_package_oracles():
    import oracle

    c = _case(6)
    beta = np.full((2, 7, 3), 0.4)
    g = np.broadcast_to(c["g"], (2, 7, 3)).copy()
    out, hT = linear.delta(c["q"], c["k"], c["v"], g, beta, c["h0"])
    o, h = oracle.fwd_seq(c["q"], c["k"], c["v"], g, beta, c["h0"])
    assert np.allclose(out, o, atol=1e-12) and np.allclose(hT, h, atol=1e-12)
