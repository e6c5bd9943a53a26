"""The oracle of 8-bit rows and of sampling (oracle/head.py) against things other than itself."""
import itertools
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import head as oh


def test_codes_are_the_nearest_values_ties_to_even():
    v = sorted(Fraction(float(x)) for x in oh.VALUES[:127])
    points = [x for a, b in zip(v, v[1:]) for x in (a, (a + b) / 2, (a + b) / 2 + Fraction(1, 1 << 20), (a + b) / 2 - Fraction(1, 1 << 20))]
    for x in points:
        best = min(range(127), key=lambda i: (abs(v[i] - x), i % 2))
        assert oh.to_e4m3(np.array([float(x)]))[0] == best
        assert oh.to_e4m3(np.array([-float(x)]))[0] == best + 128
    x = np.linspace(-448, 448, 20001)
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oh.to_e4m3(x.astype(np.float32)), want)


@pytest.mark.parametrize("top", [448.0, np.nextafter(448.0, 449), 447.0, 1.0, 65504.0, 2.0 ** -24, 3.5, 7.0, 7.00001])
def test_scale_is_the_smallest_that_holds(top):
    e = oh.scale_exponent(top)
    assert top <= 448 * 2.0 ** e and top > 448 * 2.0 ** (e - 1)


def test_rows_stand_for_what_they_hold():
    x = np.random.RandomState(1).randn(5, 300).astype(np.float16).astype(np.float64)
    x[1, 128:256] = 0
    x[2, 5], x[3, 290] = np.inf, np.nan
    c, s = oh.rows8(x)
    v = oh.held(c, s)
    assert c.shape == (5, 384) and s.shape == (5, 3) and s[1, 1] == 127
    for r, b in itertools.product(range(5), range(3)):
        part = v[r, 128 * b:128 * b + 128]
        if (r, b) in ((2, 0), (3, 2)):
            assert np.isnan(part).all() and s[r, b] == 255
            continue
        want = np.zeros(128)
        want[:len(x[r, 128 * b:128 * b + 128])] = x[r, 128 * b:128 * b + 128]
        e = 2.0 ** (int(s[r, b]) - 127)
        assert (np.abs(part - want) <= np.maximum(np.abs(want) / 16, 2.0 ** -10 * e)).all()


def test_product_of_one_hot_rows_is_the_weight():
    w = oh.held(*oh.rows8(np.random.RandomState(2).randn(9, 130)))
    x = oh.held(*oh.rows8(np.eye(130)))
    y, top, mag = oh.linear8(x, w)
    assert np.array_equal(y, w[:, :130].T)
    assert np.array_equal(top, np.abs(y)) and np.array_equal(mag, np.abs(y))


def test_tokens_come_in_proportion_to_their_weights():
    l = [math.log(1), math.log(3), -math.inf, math.log(4)]
    got = [oh.sample(l, i / 800)[0] for i in range(800)]
    assert [got.count(i) for i in range(4)] == [100, 300, 0, 400]
    assert abs(oh.sample(l, 0.9)[1] - math.log(0.5)) < 1e-11


def test_limits_by_hand():
    l = [0.0, 2.0, 1.0, 2.0, -1.0]                    # order: 1, 3, 2, 0, 4
    kept = lambda **kw: sorted(oh.sample(l, 0.5, **kw)[2])  # noqa: E731
    assert kept() == [0, 1, 2, 3, 4]
    assert kept(top_k=1) == [1] and kept(top_k=3) == [1, 2, 3] and kept(top_k=9) == [0, 1, 2, 3, 4]
    assert kept(top_p=0.0) == [1] and kept(top_p=1.0) == [0, 1, 2, 3, 4]
    e = math.e
    share = 2 * e * e / (2 * e * e + e + 1 + 1 / e)       # of the two largest
    assert kept(top_p=np.float32(share - 1e-3)) == [1, 3] and kept(top_p=np.float32(share + 1e-3)) == [1, 2, 3]
    assert kept(top_k=2, top_p=0.5) == [1] and kept(top_k=2, top_p=0.51) == [1, 3]
    assert kept(min_p=1.0) == [1, 3] and kept(min_p=5.0) == [1, 3] and kept(min_p=0.3) == [1, 2, 3]
    assert kept(min_p=0.3, top_k=1) == [1]
    assert oh.sample(l, 0.7, t=0.0)[:2] == (1, 0.0)
    assert oh.sample(l, 1.0, top_k=2)[0] == 3 and oh.sample(l, -1.0, top_k=2)[0] == 1
    for bad in ([math.nan, 0.0], [math.inf, 0.0], [-math.inf] * 2):
        assert oh.sample(bad, 0.5)[0] == -1
    for kw in (dict(t=-1.0), dict(t=math.nan), dict(t=math.inf), dict(top_p=math.nan), dict(min_p=math.nan)):
        assert oh.sample(l, 0.5, **kw)[0] == -1
    assert oh.sample(l, math.nan)[0] == -1 and oh.sample(l, math.nan, t=0.0)[0] == 1
