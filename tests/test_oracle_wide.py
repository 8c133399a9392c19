"""Pins of the float64 oracle of the 8-bit blocks and of positions on several axes (CPU)."""

import numpy as np
import pytest
import torch

from oracle import operators as O


def test_e4m3_values():
    all_codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.E4M3, all_codes) and O.E4M3[-1] == 448.0


def test_mxfp8_blocks():
    x = np.zeros((4, 32))
    x[0, :6] = [256.0, 511.0, -300.0, 17.0, 2.0 ** -9, 3 * 2.0 ** -11]     # E = 0
    x[1, 0] = 1.0                                                          # E = -8
    x[2, 0] = np.inf
    codes, scales, v = O.mxfp8_quantize(x)
    assert scales[:, 0].tolist() == [127, 119, 255, 27]
    assert v[0, :6].tolist() == [256.0, 448.0, -288.0, 17.0 - 1, 2.0 ** -9, 2.0 ** -9]    # 17: a tie, to even
    assert v[1, 0] == 1.0 and codes[1, 0] == 0x78 and np.isnan(v[2]).all() and not v[3].any()


@pytest.mark.parametrize("seed", range(3))
def test_mxfp8_against_torch_casts(seed):
    r = np.random.default_rng(seed)
    x = r.normal(size=(50, 64)) * 2.0 ** r.integers(-40, 40, (50, 1))
    codes, scales, v = O.mxfp8_quantize(x)
    E = scales.astype(np.int64) - 127
    scaled = np.clip(np.ldexp(x, -np.repeat(E, 32, -1)), -448, 448)
    top = np.abs(scaled).reshape(50, 2, 32).max(-1)
    assert ((top >= 256) & (top < 512)).all()
    want = torch.from_numpy(scaled.astype(np.float32)).to(torch.float8_e4m3fn)
    # float32 first: double rounding could matter only at distances below 2^-24 of a tie
    assert (want.view(torch.uint8).numpy() == codes).mean() > 0.9999
    assert np.array_equal(O.mxfp8_values(codes, scales), v)
    assert np.isnan(O.mxfp8_values(np.array([[127] * 32], np.uint8), np.array([[127]], np.uint8))).all()
    assert np.isnan(O.mxfp8_values(np.zeros((1, 32), np.uint8), np.array([[247]], np.uint8))).all()


def test_axis_angles():
    r = np.random.default_rng(5)
    tab = r.normal(size=(20, 12))
    pos = np.array([[3, 4], [7, 25]])
    cos, sin = O.axis_angles(tab, pos, [0, 1, 1, 0, 0, 1], 12)
    assert cos[0].tolist() == [tab[3, 0], tab[7, 1], tab[7, 2], tab[3, 3], tab[3, 4], tab[7, 5]]
    assert sin[0].tolist() == [tab[3, 6], tab[7, 7], tab[7, 8], tab[3, 9], tab[3, 10], tab[7, 11]]
    assert np.isnan(cos[1]).tolist() == [False, True, True, False, False, True]      # 25 is outside
    one = O.axis_angles(tab, pos[:1], [0] * 6, 12)
    assert np.array_equal(one[0], O.angles(tab, pos[0], 12)[0])
