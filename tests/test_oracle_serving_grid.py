"""The step of a cache's grid is fl32(hi - lo) fl32(1 / maxq), not the quotient: rows on which the two differ.  CPU only."""
import numpy as np
import pytest

from oracle import serving_ref as o

F = np.float32
# rows (a, -a, a/2): width, a, zero point and codes by the product; by the quotient the zero point is one higher
PINS = [(4, 0.7109375, 7, [14, 0, 11]), (4, 3.359375, 7, [14, 0, 11]), (8, 0.8125, 127, [254, 0, 191]),
        (8, 3.46875, 127, [254, 0, 191])]


@pytest.mark.parametrize("bits,a,zero,codes", PINS)
def test_the_step_is_a_product(bits, a, zero, codes):
    row = np.array([a, -a, a / 2], F)
    maxq = F((1 << bits) - 1)
    s, z, q = o.kv_grid(row, bits)
    assert s == F(F(2 * a) * F(F(1) / maxq)) and z == zero and q.tolist() == codes
    quotient = F(F(2 * a) / maxq)
    assert quotient != s and np.rint(F(F(a) * F(F(1) / quotient))) == zero + 1
