"""Sums over many rows in linear_bwd: how long a chain of additions gets."""
import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_db_of_many_rows_and_columns():
    """39424 columns leave each of the two summing warps per SM one range of all 12288
    rows.  In one chain, 4096 + 2^-13 would be 4096 row after row (half a step is
    2^-12), 12287 times: 3.7e-4 of the sum.  In chains of 1024 rows that are added in turn
    an element passes at most 1024 + 12 additions, and with up to a few ranges some 8 more,
    each of which is off by at most 2^-24 of a partial sum that is at most the sum of magnitudes."""
    rows, N, K = 12288, 154 * 256, 8
    dy = torch.full((1, rows, N), 2.0 ** -13, dtype=BF, device="cuda")
    dy[0, 0] = 4096.0
    dy[0, 1, 1::2] = -1.0
    x, w = torch.ones(1, rows, K, dtype=BF, device="cuda"), torch.ones(N, K, dtype=BF, device="cuda")
    db = txl.linear_bwd(dy, x, w, want=("dw", "db"))["db"].double()
    torch.cuda.synchronize()
    assert txl.sync_status() == 0
    small = (rows - 1) * 2.0 ** -13
    want = torch.full((N,), 4096.0 + small, dtype=torch.float64, device="cuda")
    want[1::2] -= 1.0 + 2.0 ** -13
    assert float((db - want).abs().max()) <= (1024 + 12 + 8) * 2.0 ** -24 * (4096.0 + small + 1.0)
