"""AdamW at the edges of what its checks accept."""
import math

import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.mark.parametrize("max_norm", [1e-300, 1e-50, 1e-40])
def test_max_norm_below_the_range_of_fp32(max_norm):
    """The clip factor max_norm / norm is 0 (or next to it) there, not 1: what is left of a
    step is m's and v's decay and the weights'."""
    n = 1000
    p, g = torch.full((n,), 2.0, device="cuda"), torch.ones(n, device="cuda")
    opt = txl.AdamW([p], [g], lr=0.5, weight_decay=0.1, max_norm=max_norm, eps=1e-8)
    opt.step()
    torch.cuda.synchronize()
    assert abs(float(opt.grad_norm) - math.sqrt(n)) <= 64 * U * math.sqrt(n)
    assert float(opt.exp_avg.abs().max()) <= 1e-40 and not opt.exp_avg_sq.any()
    # lr m / (1 - b1) / eps <= 0.5 * 1e-40 / sqrt(n) / 1e-8; three roundings of up to 2
    assert float((p - 1.9).abs().max()) <= 3 * U * 2 + 1e-30


@pytest.mark.parametrize("max_norm", [1e38, 1e39, 1e300])
def test_max_norm_above_the_range_of_fp32(max_norm):
    p, g = torch.full((1000,), 2.0, device="cuda"), torch.ones(1000, device="cuda")
    opt = txl.AdamW([p], [g], lr=0.5, max_norm=max_norm)
    opt.step()
    assert float((p - 1.5).abs().max()) <= 16 * U * 2 + 1e-8 and int(opt.steps) == 1


@pytest.mark.parametrize("bits", [8, 32])
def test_smallest_eps(bits):
    """2^-126, the smallest one taken: elements whose gradient is 0 stay, the others move by lr."""
    p, g = torch.full((1000,), 2.0, device="cuda"), torch.ones(1000, device="cuda")
    g[::2] = 0.0
    txl.AdamW([p], [g], lr=0.5, eps=2.0 ** -126, state_bits=bits).step()
    assert bool((p[::2] == 2.0).all()) and float((p[1::2] - 1.5).abs().max()) <= 16 * U * 2
    with pytest.raises(txl.TxlError) as e:
        txl.AdamW([p], [g], lr=0.5, eps=1e-40, state_bits=bits).step()
    assert e.value.code == -1


@pytest.mark.parametrize("pd", [F32, BF])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("max_norm", [None, 1.0])
def test_nothing_but_empty_parameters(pd, bits, max_norm):
    p = [torch.empty(0, dtype=pd, device="cuda"), torch.empty(3, 0, dtype=pd, device="cuda")]
    opt = txl.AdamW(p, [torch.empty(0, device="cuda"), torch.empty(3, 0, device="cuda")], lr=0.5, state_bits=bits, max_norm=max_norm)
    opt.step()
    opt.load_state_dict(opt.state_dict())
    opt.step()
    torch.cuda.synchronize()
    assert int(opt.steps) == 2 and (max_norm is None or float(opt.grad_norm) == 0.0)
