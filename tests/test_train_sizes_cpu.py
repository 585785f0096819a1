"""Sizes of 2^31 and more: refused by the training operators' binding, which hands
sizes to C as 32-bit integers (2^32 + 64 arrived there as 64)."""
import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl
from transformer_xl_relative_attn_gb300 import train

BF = torch.bfloat16
BIG = [2 ** 31, 2 ** 32 + 64, 2 ** 33 + 128]


def meta(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.fixture
def unchecked(monkeypatch):
    """Shapes without memory: the check that a tensor is on a GPU is left out."""
    monkeypatch.setattr(train, "_need", lambda *args, **kw: None)


@pytest.mark.parametrize("d", BIG)
def test_row_length(unchecked, d):
    x, w, s = meta(2, d), meta(d), meta(2, dtype=torch.float32)
    for call in (lambda: txl.layer_norm_fwd(x, w, w), lambda: txl.layer_norm_bwd(x, x, w, s, s)):
        with pytest.raises(txl.TxlError) as e:
            call()
        assert e.value.code == -2
    assert txl.layer_norm_bwd_workspace_bytes(3, d, device=0) == 0


@pytest.mark.parametrize("rows", BIG)
def test_rows(unchecked, rows):
    x, w, s = meta(rows, 8), meta(8), meta(rows, dtype=torch.float32)
    with pytest.raises(txl.TxlError) as e:
        txl.layer_norm_bwd(x, x, w, s, s)
    assert e.value.code == -2
    assert txl.layer_norm_bwd_workspace_bytes(rows, 8, device=0) == 0


@pytest.mark.parametrize("big", BIG)
@pytest.mark.parametrize("axis", range(4))
def test_linear(unchecked, big, axis):
    B, T, K, N = (big if a == axis else 64 for a in range(4))
    for x in (meta(B, T, K), meta(B, K // 64, T, 64)):
        with pytest.raises(txl.TxlError) as e:
            txl.linear_bwd(meta(B, T, N), x, meta(N, K))
        assert e.value.code == -2
        assert txl.linear_bwd_workspace_bytes(x.shape, N, device=0) == 0
