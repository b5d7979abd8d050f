"""CPU checks of the fp64 forms that the dense operators are held to, where they could lose digits."""
from decimal import Decimal, getcontext

import numpy as np

from oracle import dense_oracle as D


def test_sigmoid_keeps_its_digits():
    """1 / (1 + e^-z) in 60 digits: the fp64 form is within a few steps of 2^-52, and within the
    argument's own step times its size, at both ends; beyond e^-708 it underflows to 0."""
    getcontext().prec = 60
    z = np.array([-700, -300, -89, -60, -40, -36, -30, -20.25, -8, -1, -1e-3, 0, 1e-3, 1, 8, 20.25, 36, 60, 700])
    for v, got in zip(z, D.sigmoid(z)):
        want = 1 / (1 + (-Decimal(float(v))).exp())
        assert abs(Decimal(float(got)) / want - 1) <= Decimal(4 * 2.0 ** -52), v
    far = D.sigmoid(np.array([-3e38, -np.inf, 3e38, np.inf]))
    assert np.array_equal(far, [0, 0, 1, 1])
    assert np.isnan(D.sigmoid(np.array([np.nan])))[0]
