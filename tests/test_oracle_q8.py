"""Pins of the 8-bit block format's float64 oracle: torch's E4M3 conversion on
the CPU, the format's bounds, and hand-worked blocks."""

import numpy as np
import pytest
import torch

from oracle import q8 as ref


def test_rounding_is_torchs_on_every_fp32_pattern_class():
    rng = np.random.default_rng(0)
    grid = np.arange(256, dtype=np.uint8)
    values = torch.from_numpy(grid).view(torch.float8_e4m3fn).double().numpy()
    finite = np.sort(values[np.isfinite(values)])
    mid = (finite[1:] + finite[:-1]) / 2  # every tie
    v = np.concatenate([finite, mid, np.nextafter(mid.astype(np.float32), np.float32(1e9)).astype(np.float64),
                        rng.uniform(-448, 448, 4096).astype(np.float32).astype(np.float64),
                        rng.standard_normal(4096).astype(np.float32).astype(np.float64) * 2.0 ** -7])
    v = v[np.abs(v) <= 448]
    want = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.round_e4m3(v), want)


@pytest.mark.parametrize("amax,e", [(448.0, 0), (449.0, 1), (224.0, -1), (1.75, -8), (1.76, -7), (0.0, -117),
                                    (2.0 ** -149, -117), (3.4028234663852886e38, 120)])
def test_exponent(amax, e):
    assert ref.exponent(amax) == e


def test_exponent_is_the_smallest():
    rng = np.random.default_rng(1)
    for a in 10.0 ** rng.uniform(-30, 38, 200):
        e = ref.exponent(a)
        assert a <= 448 * 2.0 ** e and a > 448 * 2.0 ** (e - 1)


def test_rows_error_is_one_rounding():
    """Each value is off by at most half a step of E4M3: 2^-4 of itself, or
    2^-10 (half the smallest code) of the block's scale."""
    x = np.random.default_rng(2).standard_normal((9, 300))
    codes, scales = ref.quantize_rows(x)
    v = ref.row_values(codes, scales)
    assert codes.shape == (9, 384) and scales.shape == (3, 12)
    assert (scales[:, 9:] == 10).all() and not v[:, 300:].any()
    step = np.repeat(2.0 ** (scales[:, :9].T.astype(float) - 127), 128, axis=1)[:, :300]
    assert (np.abs(v[:, :300] - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * step)).all()


def test_weight_transpose_is_the_same_weight():
    w = np.random.default_rng(3).standard_normal((200, 130))
    codes, scales, codes_t, scales_t = ref.quantize_weight(w)
    assert codes.shape == (200, 256) and codes_t.shape == (130, 256) and scales.shape == (2, 2)
    a, b = ref.weight_values(codes, scales), ref.weight_values(codes_t, scales_t)
    assert np.array_equal(a[:, :130], b[:, :200].T)
    assert not a[:, 130:].any() and not b[:, 200:].any()


def test_non_finite_elements():
    x = np.ones((1, 128))
    x[0, 3], x[0, 5], x[0, 7] = np.nan, np.inf, -np.inf
    codes, scales = ref.quantize_rows(x)
    assert scales[0, 0] == 127 - 8 and np.isnan(codes[0, [3, 5, 7]]).all()
    assert codes[0, 0] == 256.0
