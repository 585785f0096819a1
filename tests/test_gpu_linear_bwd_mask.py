"""The ReLU mask of linear_bwd's dx where x or the gradient is not finite."""
import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("B,T,K,N,heads", [(1, 130, 136, 64, False), (2, 65, 192, 72, True), (4, 512, 512, 512, False)])
def test_nan_in_x_and_gradients_that_are_not_finite_under_the_mask(B, T, K, N, heads):
    """What is not above 0 (NaN among it) gets a gradient of exactly 0, also where the product
    is infinite or NaN; what is above 0 gets the product as it is."""
    g = torch.Generator(device="cuda").manual_seed(K)
    x, dy, w = (torch.empty(s, device="cuda").normal_(generator=g).to(BF) for s in ((B, T, K), (B, T, N), (N, K)))
    x[..., 0], x[..., 1], x[..., 2] = float("nan"), -float("nan"), -float("inf")
    x[..., 3], x[..., 4], x[..., 5] = float("inf"), -0.0, 2.0 ** -133  # the last a subnormal bf16
    bad = {0: float("inf"), T // 2: float("nan"), T - 1: -float("inf")}
    for row, value in bad.items():
        dy[:, row, 1] = value
    xin = x.view(B, T, K // 64, 64).transpose(1, 2).contiguous() if heads else x
    dx = txl.linear_bwd(dy, xin, w, relu_in=True, want=("dx",))["dx"]
    torch.cuda.synchronize()
    assert txl.sync_status() == 0
    dx = dx.transpose(1, 2).flatten(2) if heads else dx
    on = x > 0
    assert not on[..., [0, 1, 2, 4]].any() and bool(on[..., [3, 5]].all())
    assert bool((dx[~on] == 0).all())
    for row in bad:
        assert not torch.isfinite(dx[:, row][on[:, row]]).any()
    rest = torch.tensor([t for t in range(T) if t not in bad], device="cuda")
    ref = torch.where(on[:, rest], dy[:, rest].double() @ w.double(), 0.0)
    # one rounding to bf16, and an addition of fp32 per 16 of N products cut off at 2^-23
    acc = (N / 16 + 4) * 2.0 ** -23 * (dy[:, rest].double().abs() @ w.double().abs())
    assert bool(((dx[:, rest].double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + acc) + acc).all())
