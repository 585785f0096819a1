"""Refusals of the gradient norms, on the host, and the size of their workspace."""
import math

import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl
from transformer_xl_relative_attn_gb300 import _lib

A = 0x10000  # fake, aligned device addresses, far from each other and never dereferenced
G = 1 << 30
F32, BF = txl.TXL_F32, txl.TXL_BF16


@pytest.fixture(scope="module")
def lib():
    return txl.load()


def addr(i):
    return A + i * G


def table(*entries):
    t = (_lib.GradTensor * max(1, len(entries)))()
    for i, e in enumerate(entries):
        t[i] = _lib.GradTensor(*e, 0)
    return t


def test_grad_norm_rejects_bad_arguments(lib):
    good = table((addr(0), 100, F32), (None, 0, BF), (addr(1), 300, BF))
    need = lib.txl_grad_norm_workspace_bytes(good, 3)
    assert need > 0 and need % 256 == 0

    def call(t=good, n=3, max_norm=1.0, norm=addr(2), norms=addr(3), ws=addr(4), ws_bytes=need):
        return lib.txl_grad_norm(t, n, max_norm, norm, norms, ws, ws_bytes, None)
    assert call(t=None) == -1 and call(n=0) == -1 and call(n=-1) == -1 and call(norm=None) == -1
    for limit in (-1.0, math.inf, math.nan, 1e-39, 1e39):
        assert call(max_norm=limit) == -1, limit
    assert call(t=table((None, 1, F32)), n=1) == -1 and call(t=table((addr(0), -1, F32)), n=1) == -1
    assert call(t=table((addr(0), 5, 2)), n=1) == -1
    assert call(t=table((addr(0), (1 << 38) + 1, F32)), n=1) == -2
    assert call(t=table(*[(addr(0), 1 << 38, BF)] * 5), n=5) == -2
    assert call(t=table((addr(0) + 8, 100, F32)), n=1) == -3 and call(norm=addr(2) + 2) == -3 and call(norms=addr(3) + 1) == -3
    assert call(ws=None) == -7 and call(ws=addr(4) + 128) == -7 and call(ws_bytes=need - 1) == -7
    twice = table((addr(0), 100, F32), (addr(0) + 384, 300, BF))
    assert call(t=twice, n=2) == -4
    assert call(norm=addr(1)) == -4 and call(norms=addr(2)) == -4 and call(ws=addr(0)) == -4 and call(norms=addr(4) + 16) == -4
    assert call(max_norm=0.0, norm=addr(1) + 4) == -4
    for t, n in ((table((addr(0), -1, F32)), 1), (table((addr(0), 1, 9)), 1), (good, 0), (None, 1)):
        assert lib.txl_grad_norm_workspace_bytes(t, n) == 0
    assert lib.txl_grad_norm_workspace_bytes(table((None, 0, F32)), 1) == 0


def test_binding_refuses_what_it_can_see():
    x = torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        txl.GradNorm([x])
    with pytest.raises(ValueError, match="gradient"):
        txl.GradNorm([])
    with pytest.raises(TypeError, match="dtype"):
        txl.GradNorm([x.half()])
    with pytest.raises(TypeError, match="Tensor"):
        txl.GradNorm([1.0])
