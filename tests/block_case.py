"""Inputs, oracle runs and tolerances shared by the tests of convolution,
selective scan, and norms with rotation.

Tolerances are counts of roundings, U = 2^-24 each, of the oracle's magnitudes
(the same formulas over absolute values).  The functions' own errors: exp2 and
the reciprocal 1 ulp (2 U), so a sigmoid is within (|x| + 6) U (the exponent's
product with log2(e) moves it by |x| U), a SiLU within (|x| + 8) U, a softplus
within 16 U and, for its argument's sum, |v| U.

  Convolution: W + 1 terms.  Parameters: rows more.
  Scan: with v and s bounded by V, after T tokens the state is within K = 2 (T
    + V + 24) U of the recurrence over absolute values with the square roots of
    its decays: an exponent x = sum s A is off by at most x (T + V + 20) U in
    whatever way its steps are joined, and x exp(-x) <= 0.74 exp(-x/2); the
    products and sums give T U more.  An output takes N + 4 more, and its gate
    |z| + 8; a gradient has two such factors and sums over rows or channels.
  Norm: the sum of squares d/2 (the root halves it) and 8 more, the rotation 4.

bf16 outputs add half a step, 2^-8 of the value.  fp32 outputs are fp32 values
as they are.  TINY is for results near the smallest normal number.
"""
import numpy as np

from oracle import block

U, TINY = 2.0 ** -24, 1e-35
HALF = {"bf16": 2.0 ** -8, "f32": 0.0}


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def within(name, got, want, tol):
    got = f64(got) if hasattr(got, "detach") else got
    assert got.shape == want.shape, (name, got.shape, want.shape)
    bad = ~(np.abs(got - want) <= tol + TINY)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        tol = np.broadcast_to(tol, want.shape)
        raise AssertionError(f"{name}{list(i)}: {got[i]} instead of {want[i]}, {abs(got[i] - want[i]):.3g} off, "
                             f"{tol[i]:.3g} allowed; {bad.sum()} of {bad.size}")


def spans(lens):
    ends = np.cumsum([0] + list(lens)).tolist()
    return list(zip(ends, ends[1:]))


def conv_tol(W, y, rows=0):
    """Roundings of a convolution's output, its SiLU among them."""
    return W + 12 + np.abs(y) + rows


def check_conv(c, out, hT, dtype, silu, which=None):
    """out (rows, D) and hT against the oracle; c: x, w, bias, h0 as float64, lens."""
    for n, (lo, hi) in enumerate(spans(c["lens"])):
        h0 = None if c["h0"] is None else c["h0"][n]
        o, h, y, line = block.conv(c["x"][lo:hi], c["w"], c["bias"], h0, silu)
        m, _, _, _ = block.conv(np.abs(c["x"][lo:hi]), np.abs(c["w"]), None if c["bias"] is None else np.abs(c["bias"]),
                                None if h0 is None else np.abs(h0), False)
        within(f"out[{n}]", out[lo:hi], o, conv_tol(c["w"].shape[1], y) * U * 1.2 * m + HALF[dtype] * np.abs(o))
        within(f"hT[{n}]", hT[n], h, 0)


def check_conv_bwd(c, g, dout, dhT, dtype, silu):
    W, rows = c["w"].shape[1], sum(c["lens"])
    dw, db, mdw, mdb = 0, 0, 0, 0
    for n, (lo, hi) in enumerate(spans(c["lens"])):
        h0 = None if c["h0"] is None else c["h0"][n]
        a = (c["x"][lo:hi], c["w"], c["bias"], h0, silu, dout[lo:hi], None if dhT is None else dhT[n])
        dx, dwn, dbn, dh0, dy = block.conv_bwd(*a)
        _, _, y, line = block.conv(*a[:4], silu)
        my = block.conv(np.abs(a[0]), np.abs(a[1]), None if a[2] is None else np.abs(a[2]),
                        None if h0 is None else np.abs(h0), False)[0]
        # dy's own error: the derivative of SiLU changes by at most 1/2 for y's 1
        mdy = np.abs(a[5]) * (1.1 * (12 + np.abs(y)) + (0.5 * (W + 2) * my if silu else 0))
        ady = np.abs(a[5]) * 1.1
        m = np.zeros(line.shape)
        if dhT is not None:
            m[hi - lo:] += np.abs(dhT[n])
        mw = np.zeros(c["w"].shape)
        for t in range(hi - lo):
            for i in range(W):
                m[t + i] += (mdy[t] + (W + 2) * ady[t]) * np.abs(c["w"][:, i])
                mw[:, i] += (mdy[t] + (rows + 2) * ady[t]) * np.abs(line[t + i])
        m *= U
        within(f"dx[{n}]", g["dx"][lo:hi], dx, m[W - 1:] + HALF[dtype] * np.abs(dx))
        if g["dh0"] is not None:
            within(f"dh0[{n}]", g["dh0"][n], dh0, m[:W - 1] + HALF[dtype] * np.abs(dh0))
        dw, db, mdw = dw + dwn, db + dbn, mdw + mw * U
        mdb = mdb + (mdy + (rows + 2) * ady).sum(0) * U
    within("dw", g["dw"], dw + np.zeros(c["w"].shape), mdw)
    if g["dbias"] is not None:
        within("dbias", g["dbias"], db + np.zeros(c["w"].shape[0]), mdb)


PER_TOKEN = ("x", "dt", "b", "c", "z")


def ssm_sequence(c, n, lo, hi):
    a = {k: None if c[k] is None else c[k][lo:hi] if k in PER_TOKEN else c[k]
         for k in PER_TOKEN + ("A_log", "D", "dt_bias")}
    return {**a, "h0": None if c["h0"] is None else c["h0"][n]}


def ssm_roundings(c, T):
    v = np.abs(c["dt"]).max(initial=0) + (0 if c["dt_bias"] is None else np.abs(c["dt_bias"]).max(initial=0))
    z = 0 if c["z"] is None else np.abs(c["z"]).max(initial=0)
    return 2 * (T + v + 24), z + 8


def check_ssm(c, out, hT, dtype, soft):
    for n, (lo, hi) in enumerate(spans(c["lens"])):
        f = block.ssm(**ssm_sequence(c, n, lo, hi), soft=soft)
        K, Kz = ssm_roundings(c, hi - lo)
        N = c["b"].shape[-1]
        within(f"out[{n}]", out[lo:hi], f["out"], (K + Kz + N + 4) * U * f["mo"] + HALF[dtype] * np.abs(f["out"]))
        within(f"hT[{n}]", hT[n], f["hT"], K * U * f["mh"])


def check_ssm_bwd(c, g, dout, dhT, dtype, soft):
    total = {}
    for n, (lo, hi) in enumerate(spans(c["lens"])):
        w = block.ssm_bwd(**ssm_sequence(c, n, lo, hi), soft=soft, dout=dout[lo:hi],
                          dhT=None if dhT is None else dhT[n])
        K, Kz = ssm_roundings(c, hi - lo)
        N, Dg = c["b"].shape[-1], c["x"].shape[-1] // c["b"].shape[-2]
        K = 2 * K + 2 * Kz + 16
        for k, more in (("dx", N), ("ddt", N + 4), ("db", Dg), ("dc", Dg), ("dz", N)):
            if k in w:
                within(f"{k}[{n}]", g[k][lo:hi], w[k], (K + more) * U * w["m" + k] + HALF[dtype] * np.abs(w[k]))
        if g["dh0"] is not None:
            within(f"dh0[{n}]", g["dh0"][n], w["dh0"], K * U * w["mdh0"])
        for k in ("dA_log", "dD", "ddt_bias"):
            a, b = total.get(k, (0, 0))
            total[k] = a + w[k], b + (K + N + sum(c["lens"])) * U * w["m" + k]
    for k, (a, b) in total.items():
        if g[k] is not None:
            within(k, g[k], a + np.zeros(tuple(g[k].shape)), b)


def check_norm(x, w, cos, sin, pos, l2, eps, interleaved, dtype, y):
    want, m = block.norm(x, w, cos, sin, pos, l2, eps, interleaved)
    within("y", y, want, (x.shape[-1] / 2 + 12) * U * m + HALF[dtype] * np.abs(want))


def check_norm_bwd(x, w, cos, sin, pos, l2, eps, interleaved, dtype, dy, dx, dw):
    want, wantw, m, mw = block.norm_bwd(x, w, cos, sin, pos, l2, eps, interleaved, dy)
    d = x.shape[-1]
    within("dx", dx, want, (2 * d + 32) * U * m + HALF[dtype] * np.abs(want))
    if dw is not None:
        within("dw", dw, wantw, (d / 2 + 16 + x.shape[0] * x.shape[1]) * U * mw)
