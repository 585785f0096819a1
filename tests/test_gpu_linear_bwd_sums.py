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


@pytest.mark.parametrize("T,K,N", [(65536, 2048, 2048), (262144, 1024, 1024)])
def test_dw_of_a_long_reduction(T, K, N):
    """dw's accumulators take 1024 rows at a time: 64 additions of 16 products, each off by
    at most 2^-23 of a partial sum (a tensor core may cut off), then the T / 1024 of them are
    added in fp32, as are the parts of a split reduction (32 at most), each addition off by
    2^-24; all of it relative to the sum of magnitudes, which for positive factors is the sum.
    In one accumulator the cut-off bits of T / 16 additions, which all have one sign, would be
    some 1.7e-8 of the result each for half of T / 16: 3.5e-5 at T = 65536."""
    g = torch.Generator(device="cuda").manual_seed(T)

    def n(*s):
        return torch.empty(s, device="cuda").uniform_(0.5, 1.5, generator=g).to(BF)

    dy, x, w = n(1, T, N), n(1, T, K), n(N, K)
    dw = txl.linear_bwd(dy, x, w, want=("dw",))["dw"]
    torch.cuda.synchronize()
    assert txl.sync_status() == 0
    pick = torch.arange(0, N, 61, device="cuda")  # rows of dw from every tile
    ref = torch.zeros(len(pick), K, dtype=torch.float64, device="cuda")
    for t in range(0, T, 16384):
        ref += dy[0, t:t + 16384, pick].double().t() @ x[0, t:t + 16384].double()
    tol = 64 * 2.0 ** -23 + (T / 1024 + 32) * 2.0 ** -24
    err = float(((dw[pick].double() - ref).abs() / ref).max())
    print(f"dw of {T} rows: relative error {err:.3g}, bound {tol:.3g}")
    assert err <= tol
