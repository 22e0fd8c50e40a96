"""How exact linear attention is, against the FP64 oracle, with inputs in which
each rounding that the kernels leave out would show.

States.  With keys (and queries) that are unit vectors, each token another
one, an element of hT or dh0 is one decayed value, not a sum.  Its roundings,
each of 2^-24 at most: the decay's power, the product with it, and for each
chunk (32 rows; fp32 16) and each segment (64 rows at least) behind it one and
a half (m + (a^n - 1) m: the result's, and the factor's where it is under a
half).  The three bf16 terms of a value are its 24 bits, and adding them up,
the smallest first, is exact.  With two terms 2^-17 would be missing.

Scores.  Tokens come in pairs of equal keys and opposite values, so that what
two of them leave in the output is their decay's difference, some 2^-6 of
either, and what their scores' roundings leave is not.  In one chunk no state
takes part.  With A the same sums over absolute values: the scores' fp32 sums
and decay (d + 4) 2^-24 A, their two bf16 terms 2^-16 A (half a step of half a
step), the sums over two terms a row 2 T 2^-24 A, the output's own rounding
2^-8.  With one term 2^-8 A would be missing.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import gated_deltanet_recurrence_delta_amd as gdn  # noqa: E402
from test_gpu_linear import DT, f64, oracle_of, run_all  # noqa: E402

pytestmark = pytest.mark.gpu

HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def dev(x, dtype="f32"):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 128), (128, 32), (128, 128)])
@pytest.mark.parametrize("T", [1, 31, 32, 64, 100, 512])
def test_states_are_exact_to_24_bits(dtype, dk, dv, T):
    r = np.random.default_rng(T + dk + dv)
    H = 2
    unit = np.zeros((1, T, H, dk))
    for i in range(min(T, dk)):
        unit[:, i * T // dk if T >= dk else i, :, i] = 1
    c = dict(q=dev(unit, dtype), k=dev(unit, dtype), v=dev(r.standard_normal((1, T, H, dv)), dtype),
             dout=dev(r.standard_normal((1, T, H, dv)), dtype), g=dev([-2.0 ** -4, -2.0 ** -8]), h0=None, dhT=None)
    if T == 512:
        assert gdn.gdn_linear_workspace_size(1, T, H, dk, dv, 0, 1) > 0  # a sequence that is cut
    got, ref = run_all(c), oracle_of(c)
    n = 2 + 1.5 * (T // (32 if dtype == "bf16" else 16) + T // 64 + 2)
    for name in ("hT", "dh0"):
        x, want = f64(got[name]), ref[name]
        assert (np.abs(x - want) <= n * 2.0 ** -24 * np.abs(want)).all(), \
            (name, np.nanmax(np.abs(x - want) / np.maximum(np.abs(want), 1e-30)) * 2.0 ** 24)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(32, 32), (32, 128), (64, 64), (128, 128)])
@pytest.mark.parametrize("T", [2, 16, 17, 31, 32])
def test_scores_that_cancel(dtype, dk, dv, T):
    r = np.random.default_rng(T + dk * dv)
    H, pair = 2, np.arange(T) // 2
    sign = np.where(np.arange(T) % 2 == 0, 1.0, -1.0)[None, :, None, None]
    draw = lambda d: r.standard_normal((1, T, H, d))[:, pair]  # noqa: E731
    c = dict(q=dev(draw(dk) / dk ** 0.5, dtype), k=dev(draw(dk) / dk ** 0.5, dtype), v=dev(draw(dv) * sign, dtype),
             dout=dev(draw(dv) * sign, dtype), g=dev([-2.0 ** -6, -2.0 ** -8]), h0=None, dhT=None)
    got, ref, mag = run_all(c), oracle_of(c), oracle_of(c, absolute=True)
    for name in ("out", "dq", "dk", "dv"):
        tol = ((2.0 ** -16 if dtype == "bf16" else 0) + (max(dk, dv) + 4 + 2 * T) * 2.0 ** -24) * mag[name]
        tol = tol + HALF_STEP[dtype] * (np.abs(ref[name]) + tol)
        err = np.abs(f64(got[name]) - ref[name])
        assert (err <= tol).all(), (name, float((err / np.maximum(tol, 1e-30)).max()))
