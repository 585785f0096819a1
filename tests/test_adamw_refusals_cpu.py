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


@pytest.mark.parametrize("pd,bits", [(F32, 32), (BF, 32), (F32, 8), (BF, 8)])
def test_flat_buffers_of_no_elements_may_be_null(lib, pd, bits):
    """A list of empty tensors has no state: every type and width passes its checks (here on to
    the missing workspace), and buffers that the form does not have are still refused."""
    t = (_lib.AdamwTensor * 2)(_lib.AdamwTensor(None, None, 0, 0.0, 0), _lib.AdamwTensor(None, None, 0, 0.0, 0))

    def call(master=None, ms=None):
        return lib.txl_adamw_step(t, 2, pd, F32, bits, master, None, ms, None, None, addr(4), addr(5), 0.9, 0.999, 1e-8,
                                  0.0, 0, None, None, 0, None)
    assert call() == -7
    assert call(master=addr(2)) == (-7 if pd == BF else -1) and call(ms=addr(3)) == (-7 if bits == 8 else -1)
