"""The oracle of the block operators, pinned on the CPU against things other
than itself."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import block as ob


def test_e4m3_table_and_rounding():
    assert ob.E4M3[126] == 448.0 and ob.E4M3[1] == 2.0 ** -9 and ob.E4M3[8] == 2.0 ** -6
    v = ob.E4M3
    assert np.array_equal(ob.to_e4m3(v), np.arange(127))
    mid = (v[1:] + v[:-1]) / 2                      # exact ties go to the even code
    assert np.array_equal(ob.to_e4m3(mid) % 2, np.zeros(126))
    import torch                                    # an independent implementation of the format
    x = np.random.default_rng(0).standard_normal(20000).astype(np.float32) * 60
    x = np.clip(np.concatenate([x, x * 1e-4]), -448, 448)
    assert np.array_equal(ob.to_e4m3(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_codes_are_within_half_a_step_of_exact_rationals(fmt):
    x = np.random.default_rng(1).standard_normal((64, 8)).astype(np.float16)
    c, s = ob.quantise(x, fmt)
    val = ob.from_codes(c, fmt)
    amax = Fraction(float(np.abs(x).max()))
    for xi, vi in zip(x.ravel(), val.ravel()):
        t = Fraction(float(xi)) * Fraction(ob.CODE_MAX[fmt]) / amax
        step = 1.0 if fmt == "int8" else max(2.0 ** -9, 2.0 ** (math.floor(math.log2(max(abs(float(t)), 2.0 ** -6))) - 3))
        assert abs(t - Fraction(float(vi))) <= Fraction(step) / 2 * (1 + Fraction(1, 10 ** 5))
    assert abs(float(s) - float(amax) / ob.CODE_MAX[fmt]) <= 2.0 ** -24 * float(s)
    assert ob.quantise(np.zeros((4, 4), np.float16), fmt)[1] == 0


def test_rope_is_a_rotation_and_inverse_is_its_transpose():
    g = np.random.default_rng(2)
    x, y = g.standard_normal((5, 3, 16)), g.standard_normal((5, 3, 16))
    pos = np.array([0, 1, 7, 1000, 131071])
    for layout in ("half", "interleaved"):
        f, _ = ob.frequencies(12)
        rx, ry = ob.rope(x, pos, f, 1.0, layout), ob.rope(y, pos, f, 1.0, layout, inverse=True)
        assert np.allclose((rx * y).sum(), (x * ry).sum(), rtol=1e-12)
        assert np.allclose((rx ** 2).sum(-1), (x ** 2).sum(-1))
        assert np.array_equal(rx[0], x[0]) and np.array_equal(rx[..., 12:], x[..., 12:])
        # the angle between two positions is what counts
        a = ob.rope(x[:1].repeat(2, 0), [3, 8], f, 1.0, layout)
        b = ob.rope(y[:1].repeat(2, 0), [10, 15], f, 1.0, layout)
        assert np.allclose((a[0] * b[0])[..., :12].sum(), (a[1] * b[1])[..., :12].sum())


def test_scaled_frequencies():
    f0, _ = ob.frequencies(128, 500000.0)
    assert f0[0] == 1.0
    fl, m = ob.frequencies(128, 500000.0, "linear", 4.0)
    assert np.allclose(fl, f0 / 4) and m == 1.0
    fb, _ = ob.frequencies(128, 500000.0, "base", 4.0)
    assert fb[0] == 1.0 and np.isclose(fb[-1], f0[-1] / 4)      # the slowest pair is slowed by the factor
    fp, m = ob.frequencies(128, 500000.0, "parts", 4.0)
    assert fp[0] == 1.0 and np.isclose(fp[-1], f0[-1] / 4) and np.isclose(m, 0.1 * math.log(4) + 1)


def test_cache_does_not_depend_on_how_tokens_arrive():
    g = np.random.default_rng(3)
    k, v = (g.standard_normal((150, 2, 8)).astype(np.float16) for _ in range(2))
    a, b = ob.Cache(4, 1, 2, 8, "int8"), ob.Cache(4, 1, 2, 8, "int8")
    a.put(150, [2, 0, 3], 0, k, v)
    for i in range(150):
        b.put(i + 1, [2, 0, 3], 0, k[i:i + 1], v[i:i + 1])
    for n in ("k_codes", "v_codes", "k_scale", "v_scale"):
        assert np.array_equal(getattr(a, n), getattr(b, n))
    kk, vv = a.read(150, [2, 0, 3], 0, 1)
    assert kk.shape == (150, 8) and np.array_equal(kk[128:], k[128:, 1]) and np.array_equal(vv[128:], v[128:, 1])
    assert np.abs(kk - k[:, 1]).max() <= np.abs(k[:, 1]).max() / 254 * 1.001


def test_attention_rows_against_explicit_sums():
    g = np.random.default_rng(4)
    k, v, q = g.standard_normal((5, 4)), g.standard_normal((5, 4)), g.standard_normal(4)
    o, _, _ = ob.attend(q, k, v, 3, 0.5)
    w = [math.exp(0.5 * sum(q[d] * k[j, d] for d in range(4))) for j in range(3)]
    assert np.allclose(o, [sum(w[j] * v[j, d] for j in range(3)) / sum(w) for d in range(4)])
    assert not ob.attend(q, k, v, 0, 0.5)[0].any()


def test_norm_of_constant_rows():
    y, r = np.full((2, 6), 3.0), np.full((2, 6), -1.0)
    out, _, h = ob.norm_residual(y, r, np.ones(6), np.full(6, 2.0), None, 0.5, 4.0, 0.0, 0.0)
    assert np.allclose(out, -0.5 + 4.0 * 2.0) and np.allclose(h(out), 1.0)
