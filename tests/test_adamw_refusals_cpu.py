"""Refusals of txl_adamw_step at the edges of its arguments' ranges, on the host."""
import pytest

import transformer_xl_relative_attn_gb300 as txl
from transformer_xl_relative_attn_gb300 import _lib

A, G = 0x10000, 1 << 30  # fake, aligned device addresses, far apart and never dereferenced
F32, BF = txl.TXL_F32, txl.TXL_BF16


@pytest.fixture(scope="module")
def lib():
    return txl.load()


def addr(i):
    return A + i * G


@pytest.mark.parametrize("eps", [5e-324, 1e-300, 1e-50, 1e-45, 1e-40, 1.17e-38])
def test_eps_below_the_normal_numbers_of_fp32(lib, eps):
    """The update's reciprocal takes such an operand for 0, and a zero gradient's 0 / eps
    would become NaN.  0 and 2^-126 pass (here on to the missing workspace)."""
    t = (_lib.AdamwTensor * 1)(_lib.AdamwTensor(addr(0), addr(1), 100, 0.0, 0))

    def call(e):
        return lib.txl_adamw_step(t, 1, F32, F32, 32, None, addr(2), None, addr(3), None, addr(4), addr(5), 0.9, 0.999, e,
                                  0.0, 0, None, None, 0, None)
    assert call(eps) == -1
    assert call(0.0) == -7 and call(2.0 ** -126) == -7 and call(1e-8) == -7
