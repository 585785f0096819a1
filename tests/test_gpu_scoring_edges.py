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


@pytest.mark.parametrize("rows,V", [(19456, 256), (19456, 2048), (300, 2048), (19456, 262144)])
def test_a_run_that_begins_far_below_what_counts(rows, V):
    """The first 32 columns of each half of a tile lie L below all others, whose logits are 0.  Once a
    thread's reference is at those, their terms are 1 and their sums whole numbers, which fp32 holds:
    what is left are the low columns' part q e^-L of S, off by U (3 L / ln 2 + 64 + 60) of itself and
    times L + 1 in the entropy, and the logarithm, quotient and products of the results (6 U ls + 4 U).
    For L from 3 on, as 32 columns of e^3 weigh more than four times the columns of a half tile."""
    low = torch.zeros(V, dtype=torch.bool, device="cuda")
    low[:32] = low[128:160] = True
    L = (3.0 + torch.arange(rows, device="cuda") % 35 * 0.5).double()
    x, w = torch.zeros(rows, 8, device="cuda", dtype=BF), torch.zeros(V, 8, device="cuda", dtype=BF)
    x[:, 0], w[low, 0] = L.to(BF), -1.0
    t = torch.arange(rows, device="cuda") % 100
    got = txl.linear_logprobs(x, w, t)
    q = 64 * (-L).exp()
    s = V - 64 + q
    ls, part = s.log(), q / s * U * (3 * L / math.log(2) + 124)
    given = torch.where(low[t], -L, 0.0)
    ref = {"lse": ls, "entropy": ls + q * L / s, "logprob": given - ls}
    tol = {"lse": part + 6 * U * ls + 4 * U, "entropy": part * (L + 1) + (6 * ls + 4 + q * L / s) * U,
           "logprob": part + U * (L + 7 * ls + 4)}
    for k in ref:
        off = (got[k].double() - ref[k]).abs()
        assert bool((off <= tol[k]).all()), (k, float(off.max()), float((off / tol[k]).max()))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("limit,norm", [(1e-3, 1e38), (1e-6, 2e38), (1e-8, 2e38), (2.0 ** -126, 3e38), (2.0 ** -100, 2.0 ** 27), (1e-30, 1e9)])
def test_clipping_by_a_factor_below_the_range(dtype, limit, norm):
    """max_norm / norm is below 2^-126, the clipped gradients mostly are not: norm and limit are off by
    24 U (as a root half of 4 additions of a thread's, 21 in a CTA, 14 for the pieces, and a square's
    rounding), a quotient and two products by 4 U, besides the type's rounding and that to the type's
    smallest step."""
    g = torch.Generator(device="cuda").manual_seed(3)
    unit = torch.empty(9000, device="cuda", dtype=torch.float64).normal_(generator=g)
    unit[:5] = torch.tensor([0.0, 1e-20, -30.0, 50.0, 1e-3], device="cuda")
    grads = [(p * (norm / unit.norm()).item()).to(dtype) for p in (unit[:4001], unit[4001:])]
    was = [p.double() for p in grads]
    length = torch.cat(was).norm()
    n = txl.GradNorm(grads)
    n.clip(limit)
    assert abs(float(n.norm) / float(length) - 1) <= 24 * U
    half, tiny = torch.finfo(dtype).eps / 2, 2.0 ** -149 if dtype is F32 else 2.0 ** -133
    for p, q in zip(grads, was):
        ref = q * (limit / length)
        e = 28 * U
        assert bool(((p.double() - ref).abs() <= ref.abs() * (e + half * (1 + e)) + tiny).all())


@pytest.mark.parametrize("dtype,value", [(BF, 1.546875), (BF, 1.515625), (F32, 1.406510353088379)])
def test_long_sums_of_alike_gradients(dtype, value):
    """16 GB of one value: the chains of additions do not grow with the gradients (128 of a thread's,
    one for each 16 rounds of its piece, 21 in a CTA, 18 for the pieces; half of it in the norm)."""
    x = torch.full((2 ** 33 if dtype is BF else 2 ** 32,), value, device="cuda", dtype=dtype)
    n = txl.GradNorm([x])
    n.measure()
    want = float(x[0].double()) * math.sqrt(x.numel())
    assert abs(float(n.norm) / want - 1) <= U * ((128 + 27 + 21 + 18) / 2 + 2)
    assert abs(float(n.norms[0]) / want - 1) <= U * ((128 + 27 + 21 + 1216 / 32 + 5) / 2 + 2)


@pytest.mark.parametrize("count", [3000, 5000, 300_000])
def test_many_small_tensors(count):
    """Alike ones: the additions of all tensors' sums do not grow with their number (a thread's chains
    of 64, then one for each chain, 13 in a CTA, 6 of a piece's own)."""
    flat = torch.full((count, 4), 1.406510353088379, device="cuda")
    flat[:, 3] = 0.0
    n = txl.GradNorm(list(flat.unbind(0)))
    n.measure()
    want = float(flat[0, 0].double()) * math.sqrt(3 * count)
    tol = U * ((64 + count / 256 / 64 + 13 + 6) / 2 + 2)
    assert abs(float(n.norm) / want - 1) <= tol
    each = float(flat[0, 0].double()) * math.sqrt(3)
    assert bool(((n.norms.double() / each - 1).abs() <= 8 * U).all())
    first = n.norm.clone(), flat.clone()
    n.clip(want * 2)
    assert torch.equal(n.norm, first[0]) and torch.equal(flat, first[1])
    n.clip(want / 3)
    assert torch.equal(n.norm, first[0])
    assert bool(((flat.double() / (first[1][0, 0].double() / 3) - (flat != 0).double()).abs() <= tol + 4 * U).all())
    assert bool((flat[:, 3] == 0).all()) and bool((flat[:, :3] == flat[0, 0]).all())


def test_alternatives_counted_by_a_numpy_integer():
    np = pytest.importorskip("numpy")
    x, t = torch.randn(5, 300, device="cuda"), torch.zeros(5, dtype=torch.int64, device="cuda")
    want = txl.token_logprobs(x, t, top=3)
    for count in (np.int64(3), np.int32(3)):
        got = txl.token_logprobs(x, t, top=count)
        assert all(torch.equal(got[k], want[k]) for k in want)
    for count in (3.0, "3", None, -1, np.int64(-1)):
        with pytest.raises(ValueError, match="count"):
            txl.token_logprobs(x, t, top=count)
