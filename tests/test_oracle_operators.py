"""Pins of the oracles of the block norms, the int8 linear and the clipping
coefficient (CPU)."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import adamw, block_norm, int8


def _case(seed, M=5, D=6, with_post=True, gates=2):
    rng = np.random.default_rng(seed)
    rows = -(-M // gates) if gates else 0
    return dict(x=rng.standard_normal((M, D)), h=rng.standard_normal((M, D)),
                p=dict(w_post=rng.standard_normal(D) if with_post else None,
                       gate=rng.standard_normal((gates, D)) if gates else None, gate_rows=rows, alpha=0.7,
                       w_offset=0.5),
                w_pre=rng.standard_normal(D), a=rng.standard_normal((M, D)), b=rng.standard_normal((M, D)))


def test_norm_hand_case():
    """One row (3, 4): mean square 12.5, so the norm divides by 12.5^(1/2)."""
    x, w = np.array([[3.0, 4.0]]), np.array([2.0, 1.0])
    y, rstd = block_norm.pre(x, w, eps=0.0)
    assert np.allclose(rstd, 1 / np.sqrt(12.5)) and np.allclose(y, [[6 / np.sqrt(12.5), 4 / np.sqrt(12.5)]])
    f, _ = block_norm.post(np.array([[1.0, 1.0]]), x, w, np.array([[0.5, 2.0]]), 1, alpha=2.0, eps=0.0)
    assert np.allclose(f, [[2 + 0.5 * 6 / np.sqrt(12.5), 2 + 2 * 4 / np.sqrt(12.5)]])


@pytest.mark.parametrize("with_post", [True, False])
@pytest.mark.parametrize("gates", [0, 1, 2, 5])
def test_norm_gradients_equal_differences(with_post, gates):
    """Central differences of <a, x'> + <b, y> in every argument.  Step 1e-5 on
    values of order 1: the difference's own error is of order step^2 = 1e-10."""
    c = _case(3 + gates, with_post=with_post, gates=gates)

    def value(x, h, w_pre, p):
        f, _ = block_norm.post(x, h, **p)
        y, _ = block_norm.pre(f, w_pre, w_offset=p["w_offset"])
        return float(np.sum(c["a"] * f) + np.sum(c["b"] * y))

    f, _ = block_norm.post(c["x"], c["h"], **c["p"])
    g = block_norm.backward(f, c["h"], c["a"], c["b"], c["w_pre"], c["p"]["w_post"], c["p"]["gate"], c["p"]["gate_rows"],
                            c["p"]["alpha"], w_offset=c["p"]["w_offset"])
    args = {"dx": c["x"], "dh": c["h"], "dw_pre": c["w_pre"], "dw_post": c["p"]["w_post"], "dgate": c["p"]["gate"]}
    for name, t in args.items():
        if t is None:
            continue
        diff = np.zeros(t.shape)
        for i in np.ndindex(t.shape):
            keep, step = t[i], 1e-5
            t[i] = keep + step
            up = value(c["x"], c["h"], c["w_pre"], c["p"])
            t[i] = keep - step
            diff[i] = (up - value(c["x"], c["h"], c["w_pre"], c["p"])) / (2 * step)
            t[i] = keep
        assert np.allclose(g[name], diff, rtol=1e-6, atol=1e-7), name


def test_int8_codes_against_rationals():
    """Codes are the nearest integers to the fp32 quotient (ties to even), decided here on exact rationals."""
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((6, 64)) * np.array([1, 1e-3, 50, 1e-30, 1e30, 1]).reshape(6, 1)).astype(np.float32)
    x[5] = np.arange(64) - 31.5           # top 32: s = fl32(32 fl32(1/127))
    x[0, 0] = 127.0 * 2.0 ** 3            # s = 8 exactly: multiples of 4 are ties
    x[0, 1:9] = [4, 12, 20, -4, -12, 28, 36, -20]
    codes, s = int8.quantize(x)
    assert list(codes[0, :9]) == [127, 0, 2, 2, 0, -2, 4, 4, -2]
    for m in range(6):
        for k in range(64):
            q = Fraction(float(np.float32(x[m, k] / s[m])))
            lo = q.numerator // q.denominator
            rest = q - lo
            want = lo + (1 if rest > Fraction(1, 2) or (rest == Fraction(1, 2) and lo % 2) else 0)
            assert codes[m, k] == want
    zero, s0 = int8.quantize(np.zeros((1, 16), np.float32))
    assert not zero.any() and s0[0] == 0


def test_int8_gemm_closed_form():
    a = np.array([[1, -128, 127], [0, 2, 3]], np.int8)
    b = np.array([[5, 6, 7]], np.int8)
    y = int8.gemm(a, np.array([2.0, 0.5], np.float32), b, np.array([4.0], np.float32))
    assert np.array_equal(y, [[8.0 * (5 - 768 + 889)], [2.0 * (12 + 21)]])


def test_clip_coefficient():
    norm, coef = adamw.clip([np.array([3.0]), np.array([[4.0, 0.0]])], 1.0)
    assert norm == 5.0 and coef == 1.0 / (5.0 + 1e-6)
    assert adamw.clip([np.array([0.1])], 1.0)[1] == 1.0
    assert adamw.clip([], 1.0) == (0.0, 1.0)
