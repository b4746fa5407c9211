"""Pins of the MXINT8 and SwiGLU oracle: hand-worked blocks, ties, the format's
extremes, and the gradients against differences."""
import numpy as np
import pytest

from oracle import mxint8 as Q


def block(*v):
    out = np.zeros((1, 32))
    out[0, :len(v)] = v
    return out


def test_hand_worked_block():
    # largest 5: X = 4, a step of 1/16; 0.03125 ties between 0 and 1 (even: 0), 0.09375 between 1 and 2 (2)
    codes, s = Q.quantize(block(5.0, -2.5, 0.0625, 0.03125, 0.09375, -0.03125, 1.0))
    assert s.tolist() == [[129]] and codes[0, :7].tolist() == [80, -40, 1, 0, 2, 0, 16]
    assert Q.dequantize(codes, s)[0, :7].tolist() == [5.0, -2.5, 0.0625, 0.0, 0.125, 0.0, 1.0]


def test_codes_stay_within_127():
    codes, s = Q.quantize(block(7.99, -7.99, 4.0))
    assert s[0, 0] == 129 and codes[0, :3].tolist() == [127, -127, 64]
    assert Q.quantize(block(8.0))[0][0, 0] == 64


@pytest.mark.parametrize("top,byte", [(0.0, 0), (2.0**-149, 0), (2.0**-127, 0), (2.0**-126, 1), (1.0, 127),
                                      (np.nextafter(2.0, 0), 127), (2.0, 128), (float(np.finfo(np.float32).max), 254)])
def test_scale_range(top, byte):
    codes, s = Q.quantize(block(top))
    assert s[0, 0] == byte
    if top >= 2.0**-126:
        assert 64 <= codes[0, 0] <= 127 and abs(Q.dequantize(codes, s)[0, 0] - top) <= top / 64


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_infinite_and_nan_blocks(bad):
    x = np.ones((1, 40))
    x[0, 1] = bad
    codes, s = Q.quantize(x)
    assert s[0].tolist() == [255, 127] and not codes[0, :32].any()
    assert np.isnan(Q.dequantize(codes, s)[0, :32]).all() and (Q.dequantize(codes, s)[0, 32:] == 1).all()


def test_every_value_is_within_half_a_step_but_for_the_largest():
    x = np.random.default_rng(1).standard_normal((20, 75))
    codes, s = Q.quantize(x)
    step = np.repeat(2.0 ** (s.astype(float) - 133), 32, axis=1)[:, :75]
    off = np.abs(Q.dequantize(codes, s) - x) / step
    assert (off[np.abs(codes) < 127] <= 0.5).all() and (off < 1).all()


def test_swiglu_gradients_against_differences():
    r = np.random.default_rng(2)
    g, u, gh, c = r.standard_normal((3, 8)) * 3, r.standard_normal((3, 8)), r.standard_normal((3, 8)), r.standard_normal(3)
    f = lambda g, u, c: (c[:, None] * gh * Q.swiglu(g, u)).sum()  # noqa: E731
    gg, gu, ch, gc = Q.swiglu_backward(g, u, gh, c)
    assert np.allclose(ch, c[:, None] * Q.swiglu(g, u))
    e = 1e-6
    for i in range(3):
        d = np.zeros(3)
        d[i] = e
        assert abs((f(g, u, c + d) - f(g, u, c - d)) / (2 * e) - gc[i]) < 1e-7
        for j in range(8):
            d2 = np.zeros((3, 8))
            d2[i, j] = e
            assert abs((f(g + d2, u, c) - f(g - d2, u, c)) / (2 * e) - gg[i, j]) < 1e-7
            assert abs((f(g, u + d2, c) - f(g, u - d2, c)) / (2 * e) - gu[i, j]) < 1e-7


def test_swiglu_hand_worked():
    assert Q.swiglu(np.array([0.0]), np.array([3.0]))[0] == 0.0
    assert abs(Q.swiglu(np.array([np.log(3.0)]), np.array([4.0]))[0] - 3 * np.log(3.0)) < 1e-12    # s = 3/4
    gg, gu, ch, gc = Q.swiglu_backward(np.array([[0.0]]), np.array([[6.0]]), np.array([[2.0]]), [3.0])
    assert (gg[0, 0], gu[0, 0], ch[0, 0], gc[0]) == (18.0, 0.0, 0.0, 0.0)          # 3 * 2 * 6 * 1/2
