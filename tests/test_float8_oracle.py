"""Pins of the oracle's 8-bit floating point and counter-based numbers."""

import numpy as np
import pytest

from oracle import float8


def test_values_of_codes():
    v = float8.table("e4m3")
    assert v[0x7E] == 448 and v[0x01] == 2.0 ** -9 and v[0x38] == 1 and v[0xB8] == -1 and np.isnan(v[0x7F])
    v = float8.table("e5m2")
    assert v[0x7B] == 57344 and v[0x01] == 2.0 ** -16 and v[0x3C] == 1 and np.isinf(v[0x7C]) and np.isnan(v[0x7F])


@pytest.mark.parametrize("fmt,kind", [("e4m3", "float8_e4m3fn"), ("e5m2", "float8_e5m2")])
def test_nearest_against_torch(fmt, kind):
    torch = pytest.importorskip("torch")
    g = np.random.default_rng(1)
    x = g.standard_normal(20000) * 2.0 ** g.integers(-20, 8, 20000)
    x = np.concatenate([x.astype(np.float32), (np.arange(2000) / 64).astype(np.float32), [0.0, -0.0, 448.0, -448.0]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(getattr(torch, kind)).view(torch.uint8).numpy()
    assert (float8.nearest(x.astype(np.float64), fmt) == want).all()


def test_ties_go_to_the_even_code():
    # 17 / 16 lies between 1 and 9 / 8 of e4m3, 19 / 16 between 9 / 8 and 10 / 8
    assert float8.table("e4m3")[float8.nearest(np.array([17 / 16, 19 / 16, -17 / 16]), "e4m3")].tolist() == [1, 1.25, -1]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_exponents(fmt):
    top = float8.largest(fmt)
    for e in (-127, -20, 0, 50):
        peak = top * 2.0 ** e
        assert float8.exponent(peak, fmt) == e
        assert float8.exponent(np.nextafter(peak, np.inf), fmt) == e + 1
    assert float8.exponent(0.0, fmt) == 0 and float8.exponent(2.0 ** -149, fmt) == -127


def test_a_block_that_is_not_finite():
    x = np.ones((2, 200))
    x[1, 150] = np.inf
    codes, scale = float8.quantize(x)
    v = float8.values(codes, scale)
    assert (v[0] == 1).all() and (v[1, :128] == 1).all() and np.isnan(v[1, 128:]).all() and scale[1, 1] == 127


@pytest.mark.parametrize("counter,key,want", [
    # the generator's published known answers
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(counter, key, want):
    assert tuple(float8.philox(counter, key)) == want


def test_kept_share():
    kept = float8.keep(64, 500, 0.3, 12345, 6)
    # 32000 draws: five standard deviations of a share of 0.7
    assert abs(kept.mean() - 0.7) < 5 * (0.21 / kept.size) ** 0.5
    assert (float8.keep(8, 40, 0.3, 12345, 6, row0=2) == kept[2:10, :40]).all()
    assert float8.keep(3, 7, 0.0, 1).all()
