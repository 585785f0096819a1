"""token_logprobs and token_logprobs_bwd on the GPU against fp64 formulas.

Tolerances, with U = 2^-24 and d = x - m the distance from the row's maximum.  A term
e^d carries the roundings of d, of its product with log2 e and of that constant, each
U |d|, and the exponential's 4 U (2^-22).  A thread adds c terms in two chains, and its
sums pass one rescaling at most (6 U, its exponents being parts of the d above) per batch of
at least 16 terms and per merge of 16 at most:  sum e^d is off by its value times
U (3 A + K), A = sum p |d|, K = c / 2 + 6 (c / 16 + 17) + 6; and sum e^d d by
U (3 B + (K + 1) A), B = sum p d^2.  A natural logarithm is off by at most 1 unit in the
last place, 2 U of its value.  A gradient has the same error per term, one rounding to
its type (half a step, relative), and 2^-120 for values that were flushed to 0."""
import math

import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
INF, NAN = math.inf, math.nan


def make(rows, V, dtype, seed=0, std=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(rows, V, device="cuda").normal_(0.0, std, generator=g).to(dtype)
    t = torch.randint(-1, V, (rows,), device="cuda", generator=g)
    return x, t


def terms(V, dtype):
    """K of the tolerances: c terms per thread are V / 32 at most in a warp's row, V / 128 in a CTA's."""
    c = V / 32 if V * (2 if dtype is BF else 4) <= 8192 else V / 128
    return c / 2 + 6 * (c / 16 + 17) + 6


def formula(x, t):
    """fp64 statistics of rows with probabilities, and what their tolerances are made of."""
    x = x.double()
    m = x.amax(-1, keepdim=True)
    d = x - m
    s = d.exp().sum(-1)
    p = d.exp() / s[..., None]
    pd = torch.where(p > 0, p * d, 0.0)
    A, B = -pd.sum(-1), torch.where(p > 0, pd * d, 0.0).sum(-1)
    ls = s.log()
    xt = d.gather(-1, t.clamp(min=0)[..., None])[..., 0]
    return dict(m=m[..., 0], ls=ls, lse=m[..., 0] + ls, xt=xt, logprob=torch.where(t < 0, 0.0, xt - ls), entropy=ls + A, A=A, B=B, p=p)


def check(x, t, got):
    f, K = formula(x, t), terms(x.shape[-1], x.dtype)
    # (the reference m log2 e is off by 1.45 U |m| <= 47, which each sum carries through 8 roundings)
    off = 8 * U * (1.45 * U * f["m"].abs()).clamp(max=47.0)
    sums = U * (3 * f["A"] + K + 4) + 2 * U * f["ls"] + off
    tol = {"lse": sums + U * (f["m"].abs() + f["lse"].abs()),
           "logprob": torch.where(t < 0, 0.0, sums + U * torch.where(f["xt"] > -INF, f["xt"].abs(), 0.0) + U * f["ls"]),
           "entropy": sums + off + U * (3 * f["B"] + (K + 4) * f["A"]) + f["A"] * U * (3 * f["A"] + K + 4) + U * f["entropy"]}
    for n in tol:
        assert got[n].dtype is F32 and got[n].shape == t.shape, n
        ref = f[n]
        same = torch.where(ref.isinf(), got[n].double() == ref, (got[n].double() - ref).abs() <= tol[n])
        assert bool(same.all()), (n, float(torch.where(same, 0.0, (got[n].double() - ref).abs() / tol[n]).max()))
    return f


def best(x, k):
    """Indexes of the k largest, equal ones by index."""
    return torch.sort(x.double(), dim=-1, descending=True, stable=True)[1][..., :k]


def check_top(x, f, got, k):
    index = best(x, k)
    assert got["top_index"].dtype is torch.int64 and torch.equal(got["top_index"], index)
    ref = x.double().gather(-1, index) - f["lse"][..., None]
    tol = U * (3 * f["A"] + terms(x.shape[-1], x.dtype) + 4 + 3 * f["ls"])[..., None] + 2 * U * torch.where(ref.isinf(), 0.0, ref.abs())
    same = torch.where(ref.isinf(), got["top_logprob"].double() == ref, (got["top_logprob"].double() - ref).abs() <= tol)
    assert bool(same.all())


SIZES = [(1, 1), (3, 2), (9, 7), (40, 8), (5, 9), (17, 31), (64, 33), (1000, 255), (333, 256), (8, 257), (700, 1000), (5, 1024),
         (5, 1025), (6, 2047), (7, 2048), (9, 2049), (3, 2056), (400, 4099), (1, 5000), (2, 16384), (22, 32768), (150, 10007),
         (320, 8200), (1, 131072), (2, 131075), (700, 3000), (1, 300001),
         # many rows: more of them to warps, and to smaller CTAs
         (1300, 700), (1300, 1500), (1250, 3001), (1220, 4096), (4200, 5001)]


@pytest.mark.parametrize("rows,V", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("top", [0, 1, 5, 32])
def test_statistics_and_alternatives(rows, V, dtype, top):
    top = min(top, V)
    x, t = make(rows, V, dtype, seed=rows + V)
    got = txl.token_logprobs(x, t, top=top)
    assert set(got) == {"logprob", "lse", "entropy"} | ({"top_index", "top_logprob"} if top else set())
    f = check(x, t, got)
    if top:
        check_top(x, f, got, top)
    again = txl.token_logprobs(x, t, top=top)
    assert all(torch.equal(got[k], again[k]) for k in got)


def test_peaked_and_flat_rows():
    for dtype in (BF, F32):
        for V in (100, 9000):
            x, t = make(64, V, dtype, seed=1, std=40.0)  # all but one logit far below
            check(x, t, txl.token_logprobs(x, t))
            x = torch.full((3, V), 1.5, device="cuda", dtype=dtype)  # flat: ln V
            t = torch.tensor([0, V - 1, -1], device="cuda")
            got = txl.token_logprobs(x, t, top=4)
            check(x, t, got)
            assert got["top_index"].tolist() == [[0, 1, 2, 3]] * 3
            # an offset common to the row moves the log-sum-exp alone (in fp32: multiples of 1 / 8
            # up to 1100 are exact there; in bf16, whose steps are 4 at 1000, the offset is not)
            x, t = make(16, V, dtype, seed=2)
            x = (x.to(F32) * 8).round() / 8
            far, near = txl.token_logprobs(x - 1000, t), txl.token_logprobs(x, t)
            f = check(x, t, near)
            check(x - 1000, t, far)
            # (each within check()'s tolerance of one and the same value)
            tol = 2 * U * (3 * f["A"] + terms(V, F32) + 4 + 3 * f["ls"] + f["xt"].abs())
            assert bool(((far["logprob"] - near["logprob"]).abs() <= tol).all())
            tol = 2 * U * (3 * f["B"] + (terms(V, F32) + 4 + 3 * f["A"]) * (f["A"] + 1) + 3 * f["ls"] + f["A"])
            assert bool(((far["entropy"] - near["entropy"]).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,V", [(4, 300), (1300, 300), (4, 9000), (500, 9000), (2, 100000)])
def test_rising_and_falling_logits(dtype, rows, V):
    """The sums' reference has to follow the maximum, by steps above and below those it lets pass."""
    i = torch.arange(V, device="cuda", dtype=torch.float64)
    for step, every in ((1.0, 1), (3.0, 64), (4.0, 64), (8.0, 64), (8.0, 1000), (64.0, 3000)):
        x = (torch.floor(i / every) * step).to(dtype).repeat(rows, 1)
        x[1::2] = x[1::2].flip(1)
        x[2:3] -= 300
        t = torch.arange(rows, device="cuda") * 7919 % V
        t[0] = V - 1
        k = min(V, 5)
        got = txl.token_logprobs(x, t, top=k)
        check_top(x, check(x, t, got), got, k)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,V,top", [(320, 1 << 21, 0), (320, (1 << 23) - 3, 3), (3, 1 << 24, 0), (2, (1 << 24) - 5, 5)])
def test_long_rows_of_alike_logits(rows, V, top, dtype):
    """8192 logits of 0, which every thread's first vectors are among, and the others at one distance c
    below: every addition of a thread rounds the same way, so that one chain through its 2^16 elements
    is off by 4e-4.  A term is off by U (3 |c| + 4); a thread's chain is 64 batches of 16 additions at
    most (8 in fp32), and its chains, 6 U each, number V / 2^18 (fp32: V / 2^17) and one for 128 threads;
    then come 16 merges at most.  The rest as in the tolerances above."""
    c, n0 = -(torch.arange(rows, device="cuda") % 190 + 2).double() / 64, 8192
    x = c.to(dtype)[:, None].repeat(1, V)
    x[:, :n0] = 0.0
    t = (torch.arange(rows, device="cuda") * 7919 + 5) % V
    got = txl.token_logprobs(x, t, top=top)
    s = n0 + (V - n0) * c.exp()
    ls, A = s.log(), -(V - n0) * c.exp() * c / s
    n = V / (1 << 18 if dtype is BF else 1 << 17) + 1
    sums = U * (3 * c.abs() + 4 + (1024 if dtype is BF else 512) + 6 * (n + 16)) + 2 * U * ls
    tol = {"lse": sums + U * ls, "entropy": sums + A * (2 * sums + 4 * U) + U * (ls + A), "logprob": sums + U * (c.abs() + ls)}
    ref = {"lse": ls, "entropy": ls + A, "logprob": torch.where(t < n0, 0.0, c) - ls}
    for k in ref:
        assert bool(((got[k].double() - ref[k]).abs() <= tol[k]).all()), k
    if top:
        assert bool((got["top_index"] == torch.arange(top, device="cuda")).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [6, 40, 3000, 40000])
def test_ties_go_to_the_lower_index(dtype, V):
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randint(-2, 3, (50, V), device="cuda", generator=g).to(dtype)
    x[::7, ::2] = 0.0
    x[::7, 1::2] = -0.0  # equal to 0
    x[3] = 1.0
    t = torch.zeros(50, dtype=torch.int64, device="cuda")
    k = min(V, 32)
    got = txl.token_logprobs(x, t, top=k)
    check_top(x, check(x, t, got), got, k)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,V", [(5, 40), (5, 3001), (3, 40003), (400, 5001)])
def test_masked_logits(dtype, rows, V):
    low = torch.finfo(dtype).min
    for fill in (-INF, low):
        x, _ = make(rows, V, dtype, seed=3)
        t = torch.full((rows,), V - 1, device="cuda")
        x[:, : V // 2] = fill
        x[1, 1:] = fill  # one column is left
        x[1, 0] = 2.0
        t[1] = 0
        x[2] = fill      # none is left
        got = txl.token_logprobs(x, t, top=3)
        keep = torch.arange(rows, device="cuda") != 2
        cut = {k: v[keep] for k, v in got.items()}
        check_top(x[keep], check(x[keep], t[keep], cut), cut, 3)
        assert float(got["logprob"][1]) == 0.0 and float(got["entropy"][1]) == 0.0
        if fill == -INF:
            assert got["lse"][2] == -INF and got["logprob"][2] == -INF and got["entropy"][2] == 0.0
            assert got["top_index"][2].tolist() == [0, 1, 2] and got["top_logprob"][2].tolist() == [-INF] * 3
        else:  # equal logits, however low
            assert abs(float(got["entropy"][2]) - math.log(V)) <= 1e-4
            assert abs(float(got["logprob"][2]) + math.log(V)) <= 1e-4
            assert abs(float(got["lse"][2]) / low - 1) <= 4 * U
        # a masked token has no probability; the row's other results stand
        t[0] = 1
        got = txl.token_logprobs(x, t)
        assert got["logprob"][0] <= (-INF if fill == -INF else 0.9 * low) and torch.isfinite(got["lse"][0])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [40, 40003])
def test_rows_that_are_not_finite_stay_alone(dtype, V):
    x, t = make(8, V, dtype, seed=4)
    t[:] = 5
    ref = txl.token_logprobs(x, t, top=4)
    x[2, 7], x[4, V - 1], x[6, 0] = NAN, INF, NAN
    t[6] = -1
    got = txl.token_logprobs(x, t, top=4)
    for r in range(8):
        for k in ("logprob", "lse", "entropy", "top_logprob"):
            if r in (2, 4, 6):
                if k == "logprob" and r == 6:
                    assert got[k][r] == 0.0  # it has no token
                else:
                    assert bool(got[k][r].isnan().all()), (k, r)
            else:
                assert torch.equal(got[k][r], ref[k][r]), (k, r)
    assert [int(got["top_index"][r, 0]) for r in (2, 4, 6)] == [7, V - 1, 0]


@pytest.mark.parametrize("base", [1e5, 1e6, 1.6e7, 1e8, 3e8, 2.0 ** 29 - 32, 2.0 ** 29, 1e9, 1e10, 1e12, 1e30])
@pytest.mark.parametrize("V", [40, 5000])
def test_logits_far_from_zero(base, V):
    """Differences that fp32 still holds there, or none."""
    g = torch.Generator(device="cuda").manual_seed(V)
    for sign in (1, -1):
        x = torch.randint(0, 6, (20, V), device="cuda", generator=g).double()
        x = (sign * (base + x * max(1.0, base * 2.0 ** -23))).float()
        x[3, 1:] = -INF
        t = torch.arange(20, device="cuda")
        got = txl.token_logprobs(x, t, top=3)
        check(x, t, got)
        assert torch.equal(got["top_index"], best(x, 3))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,V", [(6, 40), (1300, 200), (6, 3001), (6, 40000), (700, 5000)])
def test_order_with_many_values_that_are_not_finite(dtype, rows, V):
    x, t = make(rows, V, dtype, seed=11)
    g = torch.Generator(device="cuda").manual_seed(V)
    kind = torch.randint(0, 40, (rows, V), device="cuda", generator=g)
    x = torch.where(kind == 0, NAN, torch.where(kind == 1, INF, torch.where(kind < 5, -INF, x.float()))).to(dtype)
    x[1] = NAN
    x[2, ::2] = INF
    x[3] = -INF
    for k in (1, 4, 9, 32):
        assert torch.equal(txl.token_logprobs(x, t, top=k)["top_index"], best(x, k))


def test_extreme_magnitudes():
    for dtype, big in ((F32, 3.4e38), (BF, 3.3e38)):
        for V in (40, 9001):
            x = torch.zeros(4, V, device="cuda", dtype=dtype)
            x[0, 3], x[1, 3] = big, -big
            x[2, ::2], x[2, 1::2] = big, -big
            x[3] = -big
            x[3, 9] = -INF
            t = torch.tensor([3, 4, 2, 0], device="cuda")
            got = txl.token_logprobs(x, t, top=2)
            n = math.ceil(V / 2)
            want = [0.0, -math.log(V - 1), -math.log(n), -math.log(V - 1)]
            assert all(abs(a - b) <= 1e-5 for a, b in zip(got["logprob"].tolist(), want))
            assert all(abs(a + b) <= 1e-5 for a, b in zip(got["entropy"].tolist(), want))
            assert got["top_index"].tolist() == [[3, 0], [0, 1], [0, 2], [0, 1]]


def test_tokens_that_are_none_or_not_there():
    for V in (50, 9000):
        x, _ = make(6, V, F32, seed=5)
        t = torch.tensor([0, -1, -100, V, 2 ** 40, -2 ** 62], device="cuda")
        got = txl.token_logprobs(x, t)["logprob"]
        assert got[1:3].tolist() == [0.0, 0.0] and got[5] == 0.0 and bool(got[3:5].isnan().all()) and got[0] < 0
        lse, one = torch.logsumexp(x, -1), torch.ones(6, device="cuda")
        dx = txl.token_logprobs_bwd(x, t, lse, dlogprob=one)
        assert bool(dx[3:5].isnan().all()) and bool((dx[[1, 2, 5]] == 0).all()) and bool(torch.isfinite(dx[0]).all())
        one[3:5] = 0.0
        assert bool((txl.token_logprobs_bwd(x, t, lse, dlogprob=one)[3:5] == 0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides_offsets_and_leading_axes(dtype):
    """Slices of a padded buffer, every offset against 16 bytes; 4 axes; what lies between the
    rows is left as it was."""
    for V, wide in ((50, 61), (4100, 4111), (5000, 5001), (40000, 40064)):
        for off in range(9):
            buf, t = make(6, wide + 9, dtype, seed=off)
            x, t = buf[:, off:off + V], t.clamp(max=V - 1)
            got = txl.token_logprobs(x, t, top=3)
            f = check(x, t, got)
            check_top(x, f, got, 3)
            for to in (off, (off + 3) % 9):
                out = torch.full((6, wide + 9), 7.0, device="cuda", dtype=dtype)
                ones = torch.ones(6, device="cuda")
                r = txl.token_logprobs_bwd(x, t, got["lse"], dlogprob=ones, out=out[:, to:to + V])
                assert torch.equal(r, txl.token_logprobs_bwd(x.contiguous(), t, got["lse"], dlogprob=ones))
                assert bool((out[:, :to] == 7).all()) and bool((out[:, to + V:] == 7).all())
    x, t = make(24, 300, dtype, seed=9)
    flat = txl.token_logprobs(x, t, top=2)
    deep = txl.token_logprobs(x.view(2, 3, 4, 300), t.view(2, 3, 4), top=2)
    for k in flat:
        assert deep[k].shape[:3] == (2, 3, 4) and torch.equal(deep[k].flatten(0, 2), flat[k])
    one_row = txl.token_logprobs(x[3], t[3], top=2)  # no leading axis at all
    assert one_row["lse"].shape == () and torch.equal(one_row["top_index"], flat["top_index"][3])
    padded = torch.empty(2, 3, 4, 333, device="cuda", dtype=dtype)
    padded[..., :300] = x.view(2, 3, 4, 300)
    # (not bit by bit: rows that begin elsewhere against 16 bytes are cut into vectors, and so
    # added, in another way)
    got = txl.token_logprobs(padded[..., :300], t.view(2, 3, 4), top=2)
    check_top(x, check(x, t, {k: v.flatten(0, 2) for k, v in got.items()}), {k: v.flatten(0, 2) for k, v in got.items()}, 2)


def gradient64(x, t, lse, g=None, l=None, h=None, H=None):
    d = x.double() - lse.double()[..., None]
    p = d.exp()
    zero = torch.zeros_like(lse, dtype=torch.float64)
    g, l, h = (zero if a is None else a.double() for a in (g, l, h))
    g = torch.where(t < 0, 0.0, g)
    H = zero if H is None else H.double()
    one = torch.nn.functional.one_hot(t.clamp(min=0), x.shape[-1])
    pd, px = torch.where(p > 0, p * d, 0.0), torch.where(p > 0, p * d.abs(), 0.0)
    ref = g[..., None] * (one - p) + l[..., None] * p - h[..., None] * (pd + p * H[..., None])
    size = (g.abs() + l.abs() + (h * H).abs())[..., None]
    near = torch.where(p > 0, d.abs(), 0.0)
    tol = U * ((3 * near + 10) * (size * p + h.abs()[..., None] * px) + 4 * g.abs()[..., None] * one)
    half = torch.finfo(x.dtype).eps / 2
    return ref, half * ref.abs() + (1 + half) * tol + 2.0 ** -120 * (1 + size + h.abs()[..., None])


@pytest.mark.parametrize("rows,V", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradients(rows, V, dtype):
    x, t = make(rows, V, dtype, seed=rows + 2 * V)
    out = txl.token_logprobs(x, t)
    g = torch.Generator(device="cuda").manual_seed(V)
    w = [torch.empty(rows, device="cuda").normal_(generator=g) for _ in range(3)]
    for use in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (1, 1, 1)):
        dl, ds, dh = (a if u else None for a, u in zip(w, use))
        got = txl.token_logprobs_bwd(x, t, out["lse"], dlogprob=dl, dlse=ds, dentropy=dh, entropy=out["entropy"] if dh is not None else None)
        assert got.dtype is dtype and got.shape == x.shape
        ref, tol = gradient64(x, t, out["lse"], dl, ds, dh, out["entropy"])
        err = (got.double() - ref).abs()
        assert bool((err <= tol).all()), (use, float((err / tol).max()))


def test_gradients_are_those_of_the_statistics():
    """Differences of the forward call's own results along random directions.  With h = 2^-5 and
    |v| <= 1 the third derivative's part is below h^2 / 6 times 8 |w| (the statistics'
    third derivatives along such v are below 8 here: each is a sum of at most that many central
    moments of v and x of size 1); fp32 leaves 2e-6 |w| / h."""
    rows, V = 20, 700
    for seed in range(3):
        x, t = make(rows, V, F32, seed=seed, std=1.0)
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = [torch.empty(rows, device="cuda").normal_(generator=g) for _ in range(3)]
        v = torch.empty(rows, V, device="cuda").uniform_(-1, 1, generator=g)
        f = lambda z: (lambda o: w[0] * o["logprob"] + w[1] * o["lse"] + w[2] * o["entropy"])(txl.token_logprobs(z, t)).double()
        h = 2.0 ** -5
        slope = (f(x + h * v) - f(x - h * v)) / (2 * h)
        out = txl.token_logprobs(x, t)
        dx = txl.token_logprobs_bwd(x, t, out["lse"], dlogprob=w[0], dlse=w[1], dentropy=w[2], entropy=out["entropy"])
        size = sum(a.abs().double() for a in w)
        assert bool(((dx.double() * v.double()).sum(1) - slope).abs().le(size * (h * h / 6 * 8 + 2e-6 / h * 10)).all())


def test_gradient_takes_the_place_of_the_logits():
    for dtype in (BF, F32):
        for rows, V in ((9, 300), (130, 9001), (3, 40000)):
            buf, t = make(rows, V + 3, dtype, seed=V)
            x, t = buf[:, 1:V + 1], t.clamp(max=V - 1)
            lse, one = txl.token_logprobs(x, t)["lse"], torch.ones(rows, device="cuda")
            ref, edge = txl.token_logprobs_bwd(x, t, lse, dlogprob=one), buf[:, [0, V + 1, V + 2]].clone()
            was = x._version
            got = txl.token_logprobs_bwd(x, t, lse, dlogprob=one, out=x)
            assert got is x and torch.equal(x, ref) and torch.equal(buf[:, [0, V + 1, V + 2]], edge)
            assert x._version > was


def test_rows_that_nothing_reaches_get_zeros():
    for dtype in (BF, F32):
        for V in (33, 9000):
            x, t = make(6, V, dtype, seed=6)
            t[:] = torch.tensor([1, -1, 2, 3, -1, 0], device="cuda")
            x[1], x[2, 5], x[4] = NAN, INF, -INF
            out = txl.token_logprobs(x, t)
            g = torch.tensor([1.0, 1.0, 0.0, 2.0, 1.0, -1.0], device="cuda")
            dx = txl.token_logprobs_bwd(x, t, out["lse"], dlogprob=g)
            assert bool((dx[[1, 2, 4]] == 0).all()) and bool(torch.isfinite(dx).all())
            zero = torch.zeros_like(g)
            dx = txl.token_logprobs_bwd(x, t, out["lse"], dlogprob=g, dlse=zero, dentropy=zero, entropy=out["entropy"])
            assert bool((dx[[1, 2, 4]] == 0).all()) and bool(torch.isfinite(dx).all())
            # a row of nothing but -inf passes nothing on
            x[3] = -INF
            out = txl.token_logprobs(x, t)
            dx = txl.token_logprobs_bwd(x, t, out["lse"], dlogprob=g, dlse=g, dentropy=g, entropy=out["entropy"])
            assert bool((dx[3] == 0).all()) and bool((dx[4] == 0).all()) and bool(dx[1].isnan().all())
            # masked columns of a row with probabilities get no gradient
            x[5, V // 3:] = -INF
            out = txl.token_logprobs(x, t)
            dx = txl.token_logprobs_bwd(x, t, out["lse"], dlogprob=g, dlse=g, dentropy=g, entropy=out["entropy"])
            assert bool((dx[5, V // 3:] == 0).all()) and bool(torch.isfinite(dx[5]).all())


def test_no_rows():
    x = torch.empty(0, 50, device="cuda")
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    got = txl.token_logprobs(x, t, top=3)
    assert got["lse"].shape == (0,) and got["top_index"].shape == (0, 3)
    assert txl.token_logprobs_bwd(x, t, got["lse"], dlogprob=got["logprob"]).shape == (0, 50)


def test_offsets_beyond_32_bits():
    V, rows = 131072, 32800  # 4.3e9 logits
    x = torch.empty(rows, V, device="cuda", dtype=BF).fill_(-3.0)
    last, t = make(4, V, BF, seed=8)
    x[-4:] = last
    tokens = torch.zeros(rows, dtype=torch.int64, device="cuda")
    tokens[-4:] = t
    got = txl.token_logprobs(x, tokens, top=2)
    cut = {k: v[-4:] for k, v in got.items()}
    check_top(last, check(last, t, cut), cut, 2)
    small = txl.token_logprobs(last, t)["lse"]
    assert float((small - cut["lse"]).abs().max()) <= 1e-4
    ones = torch.ones(rows, device="cuda")
    txl.token_logprobs_bwd(x, tokens, got["lse"], dlogprob=ones, out=x)
    assert torch.equal(x[-4:], txl.token_logprobs_bwd(last, t, cut["lse"].contiguous(), dlogprob=ones[:4]))


def test_streams_and_graphs():
    x, t = make(64, 9001, BF, seed=10)
    one = torch.ones(64, device="cuda")
    ref = txl.token_logprobs(x, t, top=5)
    dref = txl.token_logprobs_bwd(x, t, ref["lse"], dlogprob=one)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for given in (side, side.cuda_stream):
        got = txl.token_logprobs(x, t, top=5, stream=given)
        dx = txl.token_logprobs_bwd(x, t, got["lse"], dlogprob=one, stream=given)
        side.synchronize()
        assert all(torch.equal(ref[k], got[k]) for k in ref) and torch.equal(dref, dx)
    graph = torch.cuda.CUDAGraph()
    outs = {k: torch.zeros_like(v) for k, v in ref.items()}
    grad = torch.zeros_like(x)
    with torch.cuda.graph(graph):
        txl.token_logprobs(x, t, top=5, outs=outs)
        txl.token_logprobs_bwd(x, t, outs["lse"], dlogprob=one, out=grad)
    for seed in (11, 12):
        y, s = make(64, 9001, BF, seed=seed)
        x.copy_(y), t.copy_(s)
        graph.replay()
        ref = txl.token_logprobs(y, s, top=5)
        assert all(torch.equal(ref[k], outs[k]) for k in ref)
        assert torch.equal(grad, txl.token_logprobs_bwd(y, s, ref["lse"], dlogprob=one))


def test_bad_tensors_are_refused():
    x, t = make(4, 64, BF)
    f = torch.zeros(4, device="cuda")
    with pytest.raises(ValueError, match="cpu"):
        txl.token_logprobs(x, t.cpu())
    with pytest.raises(TypeError, match="dtype"):
        txl.token_logprobs(x, t.int())
    with pytest.raises(ValueError, match="shape"):
        txl.token_logprobs(x, t[:3])
    for bad in (x.t(), x[:, ::2], x[:1].expand(4, 64), x.view(2, 2, 64).transpose(0, 1)):
        with pytest.raises(ValueError, match="rows|row"):
            txl.token_logprobs(bad, torch.zeros(bad.shape[:-1], dtype=torch.int64, device="cuda"))
    with pytest.raises(txl.TxlError) as e:
        txl.token_logprobs(x, t, top=33)
    assert e.value.code == -2
    with pytest.raises(txl.TxlError) as e:
        txl.token_logprobs(x[:, :5], t, top=6)
    assert e.value.code == -1
    with pytest.raises(txl.TxlError) as e:  # one row further on
        txl.token_logprobs_bwd(x[:3], t[:3], f[:3], dlogprob=f[:3], out=x[1:])
    assert e.value.code == -4
    outs = {k: f for k in ("logprob", "lse", "entropy")}
    with pytest.raises(txl.TxlError) as e:
        txl.token_logprobs(x, t, outs=outs)
    assert e.value.code == -4


@pytest.mark.parametrize("top,V,code", [(2 ** 30, 64, -1), (2 ** 40, 64, -1), (40, 64, -2), (33, 32, -1)])
def test_counts_beyond_the_limit_are_refused_ahead_of_buffers_for_them(top, V, code):
    x, t = make(1000, V, BF)
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    with pytest.raises(txl.TxlError) as e:
        txl.token_logprobs(x, t, top=top)
    assert e.value.code == code and torch.cuda.memory_stats()["allocation.all.allocated"] == before


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,V", [(1500, 5003), (1521, 5003), (1530, 12288), (1530, 12289), (1530, 24577), (4110, 9000), (4110, 20001)])
def test_many_rows_on_both_sides_of_the_choice_of_threads(rows, V, dtype):
    x, t = make(rows, V, dtype, seed=rows + V)
    got = txl.token_logprobs(x, t)
    check(x, t, got)
    again = txl.token_logprobs(x, t)
    assert all(torch.equal(got[k], again[k]) for k in got)
