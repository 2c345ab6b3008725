"""Pins of the 4-bit block format's float64 oracle: brute force over the codes,
the format's bounds, and hand-worked blocks."""

import numpy as np
import pytest

from oracle import q4 as ref

CODES = np.arange(16, dtype=np.uint8)


def test_code_values():
    assert list(ref.code_values(CODES[:8])) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert list(ref.code_values(CODES[8:])) == [0, -0.5, -1, -1.5, -2, -3, -4, -6]


def test_rounding_is_to_the_nearest_code():
    v = np.concatenate([np.linspace(-6, 6, 4801), np.random.default_rng(0).uniform(-6, 6, 4096)])
    grid = ref.code_values(CODES)
    best = np.abs(v[:, None] - grid).min(1)
    got = ref.round_e2m1(v)
    assert np.array_equal(np.abs(ref.code_values(got) - v), best)
    tie = (np.abs(np.abs(v[:, None]) - grid[:8]) == best[:, None]).sum(1) == 2
    assert tie.sum() >= 14 and (got[tie] % 2 == 0).all()
    assert np.array_equal(np.signbit(v), got >= 8)


@pytest.mark.parametrize("v,code", [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6), (-0.0, 8),
                                    (-0.1, 8), (6.0, 7)])
def test_ties(v, code):
    assert ref.round_e2m1(np.array([v]))[0] == code


def test_random_rounding_has_no_bias():
    """Over all 256 bytes the mean of a value's roundings is off by at most 1/512
    of its step, and a code stays what it is."""
    v = np.concatenate([np.linspace(-6, 6, 977), ref.code_values(CODES)])
    n = np.arange(256)
    got = ref.code_values(ref.round_e2m1(np.repeat(v[:, None], 256, 1), np.repeat(n[None], v.size, 0)))
    a = np.abs(v)
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    assert (np.abs(got.mean(1) - v) <= step / 512 + 1e-12).all()
    assert (np.abs(got - v[:, None]) < step[:, None]).all()
    exact = np.isin(v, ref.code_values(CODES))
    assert (got[exact] == v[exact, None]).all()


@pytest.mark.parametrize("amax,e", [(6.0, 0), (6.01, 1), (3.0, -1), (3.01, 0), (1.0, -2), (0.0, -125), (2.0 ** -149, -125),
                                    (3.4028234663852886e38, 126), (2.0 ** -120, -122)])
def test_exponent(amax, e):
    assert ref.exponent(amax) == e


def test_exponent_is_the_smallest():
    for a in 10.0 ** np.random.default_rng(1).uniform(-30, 38, 400):
        e = int(ref.exponent(a))
        assert a <= 6 * 2.0 ** e and a > 6 * 2.0 ** (e - 1)


def test_shapes_and_padding():
    x = np.random.default_rng(2).standard_normal((9, 300))
    codes, scales = ref.quantize(x)
    assert codes.shape == (9, 512) and scales.shape == (16, 16) and ref.pack(codes).shape == (9, 256)
    assert not codes[:, 300:].any() and (scales[:, 9:] == 2).all() and (scales[10:] == 2).all()
    v = ref.values(codes, scales)[:, :300]
    # one rounding: 1/4 of a value (half of 2 to 4, of a step of 1 to 2), or half the smallest code's scale
    s = np.repeat(2.0 ** (scales[:, :9].T.astype(float) - 127), 32, axis=1)[:, :300]
    assert (np.abs(v - x) <= np.maximum(0.25 * np.abs(x), 0.25 * s)).all()


def test_packing_order():
    assert list(ref.pack(np.array([[1, 2, 15, 8]], np.uint8))[0]) == [0x21, 0x8F]


def test_non_finite_blocks():
    x = np.ones((1, 96))
    x[0, 3], x[0, 40] = np.nan, -np.inf
    codes, scales = ref.quantize(x)
    assert list(scales[:3, 0]) == [255, 255, 125] and not codes[0, :64].any() and (codes[0, 64:96] == 6).all()
    v = ref.values(codes, scales)
    assert np.isnan(v[0, :64]).all() and (v[0, 64:96] == 1).all()
