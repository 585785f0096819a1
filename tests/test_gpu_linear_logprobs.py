"""linear_logprobs on the GPU against fp64.

Tolerances, U = 2^-24.  A logit is a sum of K products of bf16 numbers (exact in fp32): the
tensor core adds 16 at a time to the accumulator and cuts off what it adds, which loses less
than 2^-21 of the partial sum's size per step (8 U: its addends are aligned to the largest and
cut at least 3 bits below fp32's last), so a logit is off by E = 8 U (K / 16 + 1) S at most,
S = sum |x w| + |bias|.  The statistics are off by no more than the logits' largest error e
(lse and log p twice, entropy by e (1 + the spread of the logits around their mean times 2)),
besides what their own sums bring, as for token_logprobs."""
import math

import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
INF, NAN = math.inf, math.nan


def make(rows, K, V, bias=False, seed=0, std=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s, std=1.0: torch.empty(s, device="cuda").normal_(0.0, std, generator=g).to(BF)
    x, w = n(rows, K), n(V, K, std=std * K ** -0.5)
    return x, w, torch.randint(-1, V, (rows,), device="cuda", generator=g), n(V, std=0.5) if bias else None


def check(x, w, t, b, got):
    V, K = w.shape
    z = x.double() @ w.double().t()
    size = x.double().abs() @ w.double().abs().t()
    if b is not None:
        z, size = z + b.double(), size + torch.where(b.isinf(), 0.0, b.double().abs())
    e = 8 * U * (K / 16 + 1) * size.amax(1) + U * size.amax(1)
    m = z.amax(1, keepdim=True)
    d = z - m
    s = d.exp().sum(1)
    p = d.exp() / s[:, None]
    pd = torch.where(p > 0, p * d, 0.0)
    A, B, ls = -pd.sum(1), torch.where(p > 0, pd * d, 0.0).sum(1), s.log()
    # a thread's chain: half of the columns of its runs, at most 64 per tile and all tiles, in two
    # chains; then 6 roundings a merge of the parts, of which there are at most 2 per 32 columns and CTA
    Kc = min(V, 65536) / 4 + 6 * 60
    sums = U * (3 * A + Kc) + 2 * U * ls
    tol = {"lse": e + sums + 2 * U * (m[:, 0].abs() + ls), "entropy": e * (1 + 2 * A) + sums * (1 + A) + U * (3 * B + (Kc + 4) * A),
           "logprob": 2 * e + sums + U * (d.abs().where(d > -INF, torch.zeros_like(d)).amax(1) + ls)}
    ref = {"lse": m[:, 0] + ls, "entropy": ls + A, "logprob": torch.where(t < 0, 0.0, d.gather(1, t.clamp(min=0)[:, None])[:, 0] - ls)}
    for k in ref:
        assert got[k].dtype is F32 and got[k].shape == t.shape
        same = torch.where(ref[k].isinf(), got[k].double() == ref[k], (got[k].double() - ref[k]).abs() <= tol[k])
        assert bool(same.all()), (k, float(torch.where(same, 0.0, (got[k].double() - ref[k]).abs() / tol[k]).max()))
    # and as near as fp32 arithmetic comes: the tolerances above are for the worst order of things
    for k in ("lse", "entropy"):
        fine = ref[k].isfinite()
        if bool(fine.any()):
            assert float((got[k].double() - ref[k])[fine].norm()) <= 1e-5 * float(ref[k][fine].norm()) + 1e-5 * math.sqrt(len(t)), k


SIZES = [(1, 8, 1), (1, 8, 2), (3, 16, 7), (1, 64, 128), (5, 72, 129), (22, 512, 1000), (127, 64, 255), (128, 128, 256), (129, 200, 257),
         (256, 512, 512), (257, 64, 513), (300, 1000, 100), (999, 520, 1003), (22, 512, 32768), (700, 1024, 5000), (2000, 64, 40),
         (1, 1024, 131072), (130, 64, 100003), (3000, 136, 2000), (5000, 512, 4096), (40, 2048, 300), (64, 8, 50000)]


@pytest.mark.parametrize("rows,K,V", SIZES)
@pytest.mark.parametrize("bias", [False, True])
def test_matches_fp64(rows, K, V, bias):
    x, w, t, b = make(rows, K, V, bias, seed=rows + K + V)
    got = txl.linear_logprobs(x, w, t, bias=b)
    assert txl.sync_status() == 0
    check(x, w, t, b, got)
    again = txl.linear_logprobs(x, w, t, bias=b)
    assert all(torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("rows,V", [(5, 3000), (300, 9000), (40, 70000)])
def test_rising_and_falling_logits(rows, V):
    """The sums' reference has to follow the maximum, by steps above and below those it lets pass
    (whole numbers that bf16 holds: the logits are exact)."""
    i = torch.arange(V, device="cuda", dtype=torch.float64)
    for step, every in ((1.0, 32), (4.0, 64), (16.0, 64), (32.0, 100), (64.0, 500), (512.0, 3000)):
        w = torch.zeros(V, 16, device="cuda", dtype=BF)
        w[:, 0] = (torch.floor(i / every) * step).to(BF)
        w[:, 1] = w[:, 0].flip(0)
        w[:, 2] = -2048.0
        x = torch.zeros(rows, 16, device="cuda", dtype=BF)
        x[::2, 0], x[1::2, 1], x[::3, 2] = 1.0, 1.0, 1.0
        t = torch.arange(rows, device="cuda") * 7919 % V
        check(x, w, t, None, txl.linear_logprobs(x, w, t))


@pytest.mark.parametrize("base", [2.0 ** 10, 2.0 ** 16, 2.0 ** 21, -2.0 ** 21, 2.0 ** 27, 2.0 ** 33, -2.0 ** 90])
def test_logits_far_from_zero(base):
    """One column of x and w makes the offset; the rest are whole numbers, which fp32 still holds
    beside it up to 2^21 (beyond, what is left of them)."""
    g = torch.Generator(device="cuda").manual_seed(3)
    for rows, V in ((5, 300), (300, 5000)):
        w = torch.randint(-1, 2, (V, 32), device="cuda", generator=g).to(BF)
        x = torch.randint(-1, 2, (rows, 32), device="cuda", generator=g).to(BF)
        w[:, 0], x[:, 0] = 1.0, base
        t = torch.arange(rows, device="cuda") % V
        got = txl.linear_logprobs(x, w, t)
        if abs(base) <= 2.0 ** 21:
            check(x, w, t, None, got)
            want = txl.linear_logprobs(torch.cat((torch.zeros_like(x[:, :1]), x[:, 1:]), 1), w, t)
            assert bool(((got["logprob"] - want["logprob"]).abs() <= 1e-5 * (1 + want["logprob"].abs())).all())
        else:
            assert bool(((got["lse"] / base - 1).abs() <= 1e-5).all()) and bool((got["logprob"] <= 0).all())
            assert bool((got["entropy"] >= 0).all()) and bool((got["entropy"] <= math.log(V) + 1e-4).all())


# of 152 SMs each has 128 rows, or two of them 256, and all columns; more tiles than an item takes;
# the most columns there may be, nearly
@pytest.mark.parametrize("rows,V", [(19456, 262144), (19456, 600001), (130, (1 << 24) - 3)])
def test_long_runs_of_alike_logits(rows, V):
    """One logit of 0 and V - 1 at one distance c below it: every addition of a thread rounds the same
    way, so that one chain through a run's columns (65536 of them) is off by up to 9e-4.  A term is off
    by U (3 |c| + 4), a tile's sums are 64 additions at most, a run's one for each of its tiles (2048 at
    most), and 6 U go to each merge: a lane's, of two parts for each of an item's runs (24 rounds of 152
    SMs at most), and a few more; logarithm and results round by U (2 ls + lse).  In the entropy,
    ls - t / s, t / s is -A, and off by twice as much as s."""
    x, w = torch.zeros(rows, 8, device="cuda", dtype=BF), torch.zeros(V, 8, device="cuda", dtype=BF)
    c = -(torch.arange(rows, device="cuda") % 190 + 2).double() / 64
    x[:, 0], w[1:, 0] = c.to(BF), 1.0
    t = torch.arange(rows, device="cuda") % 5 * 1000
    got = txl.linear_logprobs(x, w, t)
    s = 1 + (V - 1) * c.exp()
    ls, A = s.log(), -(V - 1) * c.exp() * c / s
    merges = 2 * min(V / 256, 24 * 152) / 32 + 10
    sums = U * (3 * c.abs() + 4 + 64 + min(V / 256, 2048) + 6 * merges) + 2 * U * ls
    tol = {"lse": sums + U * ls, "entropy": sums + A * (2 * sums + 4 * U) + U * (ls + A), "logprob": sums + U * (c.abs() + ls)}
    ref = {"lse": ls, "entropy": ls + A, "logprob": torch.where(t == 0, 0.0, c) - ls}
    for k in ref:
        assert bool(((got[k].double() - ref[k]).abs() <= tol[k]).all()), k


def test_agrees_with_the_logits_in_memory():
    """One and the same logits: whole numbers, exact in bf16 and in every accumulator."""
    g = torch.Generator(device="cuda").manual_seed(1)
    for rows, K, V in ((256, 64, 1024), (128, 128, 4096)):
        x = torch.randint(-1, 2, (1, rows, K), device="cuda", generator=g).to(BF)
        w = torch.randint(-1, 2, (V, K), device="cuda", generator=g).to(BF)
        t = torch.randint(0, V, (1, rows), device="cuda", generator=g)
        z = txl.linear(x, w)
        assert float(z.abs().max()) <= 128
        a, b = txl.token_logprobs(z, t), txl.linear_logprobs(x, w, t)
        for k in a:
            assert float((a[k] - b[k]).abs().max()) <= 1e-5 * float(a[k].abs().max())


def test_masks_and_rows_that_are_not_finite():
    for rows, K, V in ((6, 64, 300), (300, 64, 300), (6, 64, 20000), (600, 64, 9000)):
        x, w, t, b = make(rows, K, V, True, seed=2)
        t[:] = torch.arange(rows, device="cuda") % (V // 2)
        ref = txl.linear_logprobs(x, w, t, bias=b)
        b[V // 2:] = -INF  # the vocabulary's padding
        got = txl.linear_logprobs(x, w, t, bias=b)
        check(x, w, t, b, got)
        cut = txl.linear_logprobs(x, w[:V // 2].contiguous(), t, bias=b[:V // 2].contiguous())
        for k in cut:
            assert float((cut[k] - got[k]).abs().max()) <= 2e-5, k
        t[1] = V - 1  # a masked token
        assert txl.linear_logprobs(x, w, t, bias=b)["logprob"][1] == -INF
        none = txl.linear_logprobs(x, w, t, bias=torch.full_like(b, -INF))
        assert bool((none["lse"] == -INF).all() and (none["logprob"] == -INF).all() and (none["entropy"] == 0).all())
        y = x.clone()
        y[2, 5], y[4, 0] = NAN, INF
        got = txl.linear_logprobs(y, w, t, bias=b)
        want = txl.linear_logprobs(x, w, t, bias=b)
        for k in got:
            assert bool(got[k][[2, 4]].isnan().all())
            keep = [r for r in range(rows) if r not in (2, 4)]
            assert torch.equal(got[k][keep], want[k][keep])
        del ref


def test_tokens_that_are_none_or_not_there():
    for rows, V in ((6, 200), (600, 5000)):
        x, w, t, _ = make(rows, 64, V, seed=3)
        t[:6] = torch.tensor([0, -1, -100, V, 2 ** 40, V - 1], device="cuda")
        got = txl.linear_logprobs(x, w, t)
        lp = got["logprob"]
        assert lp[1] == 0 and lp[2] == 0 and bool(lp[3:5].isnan().all()) and lp[0] < 0 and lp[5] < 0
        assert bool(torch.isfinite(got["lse"]).all())


def test_columns_behind_the_vocabulary_are_not_counted():
    """V = 130 of a buffer whose further rows would win."""
    w = torch.full((512, 64), 100.0, device="cuda", dtype=BF)
    w[:130] = 0.0
    x = torch.ones(5, 64, device="cuda", dtype=BF)
    t = torch.zeros(5, dtype=torch.int64, device="cuda")
    got = txl.linear_logprobs(x, w[:130], t)
    assert float((got["lse"] - math.log(130)).abs().max()) <= 1e-5


def test_leading_axes_outs_workspace_and_no_rows():
    x, w, t, b = make(24, 128, 777, True, seed=4)
    want = txl.linear_logprobs(x, w, t, bias=b)
    need = txl.linear_logprobs_workspace_bytes(24, 128, 777)
    assert need > 0
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")  # NaN all over
    outs = {k: torch.full((2, 3, 4), NAN, device="cuda") for k in want}
    got = txl.linear_logprobs(x.view(2, 3, 4, 128), w, t.view(2, 3, 4), bias=b, workspace=ws[:need], outs=outs)
    assert got is outs and all(torch.equal(outs[k].flatten(), want[k]) for k in want)
    assert bool((ws[need:] == 255).all())
    with pytest.raises(txl.TxlError) as e:
        txl.linear_logprobs(x, w, t, workspace=ws[:need - 1])
    assert e.value.code == -7
    one = txl.linear_logprobs(x[3], w, t[3], bias=b)
    assert one["lse"].shape == () and abs(float(one["lse"] - want["lse"][3])) <= 1e-4
    none = txl.linear_logprobs(x[:0], w, t[:0])
    assert none["lse"].shape == (0,)


def test_streams_and_graphs():
    x, w, t, b = make(300, 256, 5000, True, seed=5)
    want = txl.linear_logprobs(x, w, t, bias=b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for given in (side, side.cuda_stream):
        got = txl.linear_logprobs(x, w, t, bias=b, stream=given)
        side.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want)
    outs = {k: torch.zeros_like(v) for k, v in want.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        txl.linear_logprobs(x, w, t, bias=b, outs=outs)
    y, _, s, _ = make(300, 256, 5000, seed=6)
    x.copy_(y), t.copy_(s)
    graph.replay()
    want = txl.linear_logprobs(y, w, s, bias=b)
    assert all(torch.equal(outs[k], want[k]) for k in want)
    # two calls at once, a workspace each
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for st in streams:
        with torch.cuda.stream(st):
            got.append([txl.linear_logprobs(x, w, t, bias=b) for _ in range(4)])
    torch.cuda.synchronize()
    assert all(torch.equal(o[k], want[k]) for g in got for o in g for k in want)
    assert txl.sync_status() == 0


def test_bad_tensors_are_refused():
    x, w, t, b = make(4, 64, 100, True)
    for kw in (dict(x=x.float()), dict(w=w.float()), dict(t=t.int()), dict(b=b.float())):
        a = dict(x=x, w=w, t=t, b=b, **{}) | kw
        with pytest.raises(TypeError, match="dtype"):
            txl.linear_logprobs(a["x"], a["w"], a["t"], bias=a["b"])
    for kw in (dict(x=x[:, ::2]), dict(w=w[:, :32]), dict(t=t[:3]), dict(b=b[:99]), dict(w=w[0]), dict(x=x.cpu())):
        a = dict(x=x, w=w, t=t, b=b) | kw
        with pytest.raises(ValueError):
            txl.linear_logprobs(a["x"], a["w"], a["t"], bias=a["b"])
    odd = torch.zeros(4, 60, device="cuda", dtype=BF)
    with pytest.raises(txl.TxlError) as e:
        txl.linear_logprobs(odd, odd, t)
    assert e.value.code == -2
    with pytest.raises(txl.TxlError) as e:
        txl.linear_logprobs(x.view(-1)[4:68].view(1, 64), w, t[:1])
    assert e.value.code == -3
    f = torch.zeros(4, device="cuda")
    with pytest.raises(txl.TxlError) as e:
        txl.linear_logprobs(x, w, t, outs={"logprob": f, "lse": f, "entropy": f})
    assert e.value.code == -4
