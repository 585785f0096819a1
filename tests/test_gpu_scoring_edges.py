"""Scoring operators where their arithmetic is at an edge: infinite hidden states, references far
below the logits that count, clipping by far, long sums of gradients, many tensors.
U = 2^-24, half a step of fp32."""
import math

import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
INF = math.inf


@pytest.mark.parametrize("rows,K,V", [(1, 8, 1), (5, 64, 1), (22, 512, 1000), (300, 64, 100), (300, 72, 257), (3000, 136, 2000), (22, 64, 512)])
def test_an_infinite_hidden_state_leaves_nothing(rows, K, V):
    """x_k = inf and all w_vk below 0: every logit is -inf, with a bias too, whatever part of a tile
    the columns fill.  The other rows' results are those of a call without it."""
    g = torch.Generator(device="cuda").manual_seed(V)
    n = lambda *s: torch.empty(s, device="cuda").normal_(generator=g).to(BF)
    x, w, b = n(rows, K), n(V, K), n(V)
    k = K - 1
    w[:, k] = -w[:, k].abs() - 0.01
    x[:, k] = 0.0
    t = torch.arange(rows, device="cuda") % V
    t[rows // 2] = -1
    hit = torch.arange(rows, device="cuda") % 3 == 0
    y = x.clone()
    y[hit] = 0.0
    y[hit, k] = INF
    for bias in (None, b, torch.cat((b[:1], b))[1:]):
        want, got = txl.linear_logprobs(x, w, t, bias=bias), txl.linear_logprobs(y, w, t, bias=bias)
        assert bool((got["lse"][hit] == -INF).all()) and bool((got["entropy"][hit] == 0).all())
        assert bool((got["logprob"][hit] == torch.where(t < 0, 0.0, -INF)[hit]).all())
        assert all(torch.equal(got[key][~hit], want[key][~hit]) for key in want)
