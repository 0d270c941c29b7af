"""The rotation table's steps against exact arithmetic: a frequency's turns per position,
modulo one, to the unit of 2^-64, whatever the frequency's size. (Host only.)"""
from fractions import Fraction

import pytest
import torch

# 1 / (2 pi) to 70 digits.
INV_2PI = Fraction("0.1591549430918953357688837633725143620344596457404564487476673440588968")


@pytest.mark.parametrize("freq", [1.0, 0.7, 1e-4, 1e-30, 1e-300, 0.0, 100.0, 123.456, 1e6, 6.283185307179586, 3.0e10,
                                  -1.0, -1e-4, -7.5, -1e-30, -98765.4321])
def test_steps_are_exact(freq):
    import linear_attention_elu_gb300 as la
    step = int(la.la_rope_table([freq], device="cpu")[0, 0]) % 2 ** 64
    turns = Fraction(freq) * INV_2PI * 2 ** 64
    err = (step - turns) % 2 ** 64
    assert min(err, 2 ** 64 - err) <= 1


def test_frequencies_past_any_use_are_accepted():
    import linear_attention_elu_gb300 as la
    t = la.la_rope_table([1e300, -1.7e308, 2.0 ** 60, -2.0 ** 53], device="cpu")
    assert t.dtype == torch.int64 and t.shape == (4, 2)
