"""The oracle of the 4-bit cache (CPU): units and codes against properties of the
nearest level, and the test inputs' torch form against the oracle."""

import math

import numpy as np
import pytest
import torch

from oracle import kvq4
from tests import kvq4cases as Q


def test_codes_are_nearest_and_ties_even():
    levels = kvq4.MAGNITUDES
    for x in np.linspace(-7.5, 7.5, 1201):
        got = kvq4.code(x, 1.0)
        value = levels[got & 7] * (-1 if got & 8 else 1)
        assert abs(abs(x) - abs(value)) <= min(abs(abs(x) - m) for m in levels) + 1e-12
    # halfway: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6}
    for x, c in ties.items():
        assert kvq4.code(x, 1.0) == c and kvq4.code(-x, 1.0) == c + 8
        assert kvq4.code(x * 2.0 ** -40, 2.0 ** -40) == c


@pytest.mark.parametrize("top,byte", [(0.0, 0), (7.0, 127), (7.0000005, 128), (3.5, 126),
                                      (3.5000002, 127), (1.75, 125), (2.0 ** -126 * 7, 1),
                                      (2.0 ** -140, 0), (3.4e38, 253), (math.inf, 255),
                                      (math.nan, 255)])
def test_key_unit(top, byte):
    g = np.zeros(32, dtype=np.float32)
    g[5] = -np.float32(top)
    assert kvq4.key_unit(g) == byte


@pytest.mark.parametrize("top,unit", [(6.0, 1.0), (0.0, 0.0), (1.0, 0.1669921875), (6e-40, None),
                                      (math.nan, math.nan), (math.inf, math.nan)])
def test_value_unit(top, unit):
    row = np.zeros(64, dtype=np.float32)
    row[63] = top
    got = kvq4.value_unit(row)
    if unit is None:
        unit = float((torch.tensor(np.float32(top)).double() / 6).float().bfloat16())
    assert got == unit or (math.isnan(unit) and math.isnan(got))


def test_no_key_is_off_by_more_than_half_a_step():
    g = np.random.default_rng(1)
    for _ in range(200):
        row = (g.standard_normal(64) * 10.0 ** g.uniform(-3, 3)).astype(np.float32)
        codes, units = kvq4.code_keys(row)
        packed = np.array(codes[0::2]) | (np.array(codes[1::2]) << 4)
        back = kvq4.key_values(packed, np.array(units))
        unit = np.repeat([2.0 ** (u - 127) for u in units], 32)
        size = np.abs(row) / unit
        step = np.where(size < 2, 0.5, np.where(size < 4, 1, 2)) * unit
        assert (np.abs(back - row) <= step / 2).all()


def test_torch_form_of_the_inputs_is_the_oracle():
    g = torch.Generator().manual_seed(2)
    for i, dim in enumerate((32, 96, 160)):
        k = torch.randn((40, dim), generator=g) * 2.0 ** torch.randint(-20, 20, (40, 1), generator=g)
        v = torch.randn((40, dim), generator=g) * 2.0 ** torch.randint(-20, 20, (40, 1), generator=g)
        k[3], v[3] = 0.0, 0.0
        k[4, 7], v[4, 7] = math.inf, math.nan
        k[5] = torch.tensor(kvq4.MAGNITUDES * (dim // 8))
        k[6] = k[5] * 1.25
        v[6] = k[6]
        k[7] *= 2.0 ** -130
        v[7] *= 2.0 ** -130
        c = Q.quantised(k, v)
        for t in range(40):
            codes, units = kvq4.code_keys(k[t].numpy())
            nan = np.repeat(np.array(units) == 255, 32)
            got = np.stack([c["k_codes"][t] & 15, c["k_codes"][t] >> 4], -1).reshape(-1)
            assert np.array_equal(got[~nan], np.array(codes)[~nan]), (dim, t)
            assert c["k_scales"][t, :dim // 32].tolist() == units
            codes, unit = kvq4.code_values(v[t].numpy())
            got = np.stack([c["v_codes"][t] & 15, c["v_codes"][t] >> 4], -1).reshape(-1)
            assert np.array_equal(c["v_scales"][t].numpy(), unit, equal_nan=True), (dim, t)
            if unit > 0:
                assert got.tolist() == codes, (dim, t)


def test_rotation_keeps_lengths_and_turns_by_the_angle():
    g = np.random.default_rng(3)
    x = g.standard_normal((5, 2, 24))
    angle = np.arange(9)[:, None] * (0.3 ** np.arange(8))[None]
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    for pairs in (False, True):
        pos = [0, 3, 8, 9, -1]
        y = kvq4.rotate(x, pos, table, pairs)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[3:], x[3:])
        assert np.array_equal(y[..., 16:], x[..., 16:])
        a, b = (slice(0, 16, 2), slice(1, 16, 2)) if pairs else (slice(0, 8), slice(8, 16))
        z, w = x[1, :, a] + 1j * x[1, :, b], y[1, :, a] + 1j * y[1, :, b]
        assert np.allclose(w, z * np.exp(1j * angle[3]))
