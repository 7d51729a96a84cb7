"""Pins of the routing / packed-row / 4-bit oracle: hand-worked values, differences, invariants."""
import numpy as np
import pytest

from oracle import moe


def test_choice_by_hand():
    l = [0.0, 2.0, 2.0, -np.inf, np.nan, 1.0]
    assert moe.route_choose(l, None, 3, moe.SOFTMAX) == [1, 2, 5]              # a tie goes to the lower index
    assert moe.route_choose(l, None, 5, moe.SOFTMAX) == [1, 2, 5, 0, -1]       # masked ones are never chosen
    assert moe.route_choose(l, [3.0, 0, 0, 9, 9, 0], 2, moe.SOFTMAX) == [0, 1]
    assert moe.route_choose([-np.inf] * 4, None, 2, moe.SIGMOID) == [-1, -1]
    # groups of two: best keys 3, 2, 1; with sigmoid scores the sums of two decide
    l = [3.0, -9.0, 2.0, 2.0, 1.0, 1.0]
    assert moe.route_choose(l, None, 2, moe.SOFTMAX, groups=3, topk_groups=1) == [0, 1]
    assert moe.route_choose(l, None, 2, moe.SIGMOID, groups=3, topk_groups=1) == [2, 3]
    # a group with one unmasked expert competes with that one's key alone
    l = [4.0, -np.inf, -3.0, -3.0]
    assert moe.route_choose(l, None, 1, moe.SIGMOID, groups=2, topk_groups=1) == [0]


@pytest.mark.parametrize("score", [moe.SOFTMAX, moe.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    l = rng.normal(size=12)
    l[4] = -np.inf
    ids = moe.route_choose(l, None, 5, score) + [-1]
    d = rng.normal(size=6)

    def loss(x):
        return float(np.dot(d, moe.route_weights(x, ids, score, renorm, 1.7)))

    got = moe.route_loss_grad(l, ids, d, score, renorm, 1.7)
    for e in range(12):
        if np.isinf(l[e]):
            assert got[e] == 0
            continue
        h = 1e-5
        up, dn = l.copy(), l.copy()
        up[e] += h
        dn[e] -= h
        # central differences: h^2 f''' / 6 and rounding eps / h, both below 1e-9 here
        assert abs((loss(up) - loss(dn)) / (2 * h) - got[e]) < 1e-8


def test_weights_sum():
    l = np.array([1.0, 2.0, 3.0, -np.inf])
    for score in (moe.SOFTMAX, moe.SIGMOID):
        assert abs(moe.route_weights(l, [2, 1, -1], score, True, 2.5).sum() - 2.5) < 1e-12
    assert abs(moe.route_weights(l, [0, 1, 2], moe.SOFTMAX, False).sum() - 1.0) < 1e-12
    assert moe.route_weights([-np.inf] * 3, [-1, -1], moe.SOFTMAX, False).tolist() == [0, 0]


def test_sort_by_hand():
    sizes, pos, rows = moe.sort_rows([[2, 0], [0, -1], [2, 7]], 3)
    assert sizes.tolist() == [2, 0, 2] and rows == 4
    assert pos.tolist() == [[2, 0], [1, -1], [3, -1]]


def test_mx_rounding_by_hand():
    # the midpoints between levels go to the even code, beyond 6 to 6
    v = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -0.26, -0.0])
    assert (moe.mx_round(v) & 7).tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 1, 0]
    assert (moe.mx_round(v) >> 3).tolist() == [0] * 8 + [1, 1]
    assert [moe.mx_scale_byte(a) for a in (0.0, 1.0, 3.9, 4.0, 6.0, np.inf, np.nan)] == \
        [0, 125, 126, 127, 127, 255, 255]
    assert moe.mx_scale_byte(2.0 ** -126) == 0 and moe.mx_scale_byte(2.0 ** -140) == 0


def test_mx_round_trip():
    rng = np.random.default_rng(5)
    x = rng.normal(size=(4, 96))
    codes, byte = moe.mx_quantize(x)
    v = moe.mx_values(codes, byte)
    again = moe.mx_quantize(v)
    # a block whose largest magnitude rounds into 4 .. 6 times its scale keeps its scale and codes
    np.testing.assert_array_equal(moe.mx_values(*again), v)
    step = np.exp2(byte.astype(float) - 127)[..., None]
    err = np.abs(v - x).reshape(4, 3, 32)
    assert (err <= 2 * step).all()          # half of the widest gap, or the cut from below 8 to 6
    np.testing.assert_array_equal(moe.mx_unpack(moe.mx_pack(codes)), codes)
    bad = x.copy()
    bad[1, 40] = np.inf
    codes, byte = moe.mx_quantize(bad)
    assert byte[1].tolist()[1] == 255 and (codes[1, 32:64] & 7 == 0).all()
    assert np.isnan(moe.mx_values(codes, byte)[1, 32:64]).all()
