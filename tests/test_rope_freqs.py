"""gdr_rope_freqs: each frequency is the nearest whole number of 2^-64 turns (CPU only)."""
from fractions import Fraction

import pytest

from channelwise_gated_delta_gb300 import _binding

PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923078164, 10 ** 70)


def nearest(radians):
    return round(radians / (2 * PI) * 2 ** 64) % 2 ** 64


def freqs(*a, **k):
    return [int(f) % 2 ** 64 for f in _binding.gdr_rope_freqs(*a, device="cpu", **k)]


def test_given_frequencies():
    given = [1.0, 0.75, 2.0 ** -40, 3.0e-5, 6.25, 0.1, -0.5, 1e6, 0.0]
    assert freqs(18, inv_freq=given) == [nearest(Fraction(f)) for f in given]


@pytest.mark.parametrize("d_rot,base,ratio", [(4, 10000.0, Fraction(1, 100)), (8, 10000, Fraction(1, 10)),
                                              (6, 1000.0, Fraction(1, 10)), (256, 2.0 ** 128, Fraction(1, 2))])
def test_powers(d_rot, base, ratio):
    """Bases whose powers are fractions."""
    assert freqs(d_rot, base=base) == [nearest(ratio ** i) for i in range(d_rot // 2)]


def test_sizes():
    assert freqs(0) == [] and len(freqs(2)) == 1 and len(freqs(128)) == 64
    for n in (1, 3):
        with pytest.raises(ValueError):
            _binding.gdr_rope_freqs(4, inv_freq=[1.0] * n, device="cpu")
