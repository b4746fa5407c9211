"""Pins of the MXFP4 and token-sorting oracle: hand-worked blocks, ties, the
format's extremes and the tile order of the scales."""
import numpy as np
import pytest

from oracle import mxfp4 as X


def block(*v):
    out = np.zeros((1, 32))
    out[0, :len(v)] = v
    return out


def test_hand_worked_block():
    # largest 5.0: exponent 2, scale 2^0; 2.5 ties between 2 and 3 (even code: 2),
    # 5 between 4 and 6 (even code: 4), 0.25 between 0 and 0.5 (0)
    codes, s = X.quantize(block(5.0, 2.5, -0.75, 0.25, 3.5, -1.25, 1.75))
    assert s.tolist() == [[127]]
    assert X.values(codes, s)[0, :7].tolist() == [4.0, 2.0, -1.0, 0.0, 4.0, -1.0, 2.0]


def test_saturation_and_scale_steps():
    codes, s = X.quantize(block(7.99))
    assert s[0, 0] == 127 and X.values(codes, s)[0, 0] == 6.0      # above 6 goes to 6
    codes, s = X.quantize(block(8.0))
    assert s[0, 0] == 128 and X.values(codes, s)[0, 0] == 8.0


@pytest.mark.parametrize("top,byte", [(0.0, 0), (2.0**-149, 0), (2.0**-125, 0), (2.0**-124, 1), (2.0**-126, 0),
                                      (float(np.finfo(np.float32).max), 252)])
def test_scale_range(top, byte):
    _, s = X.quantize(block(top))
    assert s[0, 0] == byte


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_infinite_and_nan_blocks(bad):
    codes, s = X.quantize(block(1.0, bad))
    assert s[0, 0] == 255 and not codes.any() and np.isnan(X.values(codes, s)).all()


def test_every_value_is_its_own_rounding():
    v = np.concatenate([X.VALUES, -X.VALUES, np.zeros(16)])[None]
    v[0, -1] = 6
    assert np.array_equal(X.round_trip(v), v)


def test_tiles_are_a_bijection():
    s = np.arange(130 * 6).reshape(130, 6).astype(np.uint8)
    t = X.tile(s)
    assert t.shape == (2, 2, 512)
    assert np.array_equal(X.untile(t, 130, 192), s)
    assert t[0, 0, 0] == s[0, 0] and t[0, 0, 4] == s[32, 0] and t[0, 0, 16] == s[1, 0] and t[1, 1, 1] == s[128, 5]


def test_pack():
    c = np.arange(32, dtype=np.uint8)[None] % 16
    assert X.pack(c)[0, 0] == 0x10 and np.array_equal(X.unpack(X.pack(c)), c)


def test_sort():
    order, position, offsets = X.sort(np.array([[2, 0], [5, 2], [0, -1]]), 3)
    assert offsets.tolist() == [0, 2, 2, 4]
    assert order.tolist() == [1, 4, 0, 3, -1, -1]
    assert position.tolist() == [[2, 0], [-1, 3], [1, -1]]
