"""layer_norm_fwd and layer_norm_bwd on the GPU against fp64 formulas.

Tolerances, per element: the output's one rounding (half a step of its type,
relative) plus the fp32 arithmetic's.  A sum over a row of d elements runs as
chains of at most ceil(d / 32) + 10 additions (32 lanes at least, then a tree), each
rounding by 2^-24 of a partial sum that is at most the sum of magnitudes; the
operations around it add fewer than 16 further roundings of the terms named.
Sums over rows run as chains of at most 192 additions at the sizes tested here."""
import numpy as np
import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def make(rows, d, dtype, add, seed, mean=0.3, lead=None):
    g = torch.Generator().manual_seed(seed)
    shape = (rows, d) if lead is None else (*lead, d)

    def n(*s, std=1.0, at=0.0):
        return torch.empty(s).normal_(at, std, generator=g).to(dtype)

    return dict(x=n(*shape, at=mean), y=n(*shape, std=0.5) if add else None, gamma=n(d, std=0.2, at=1.0),
                beta=n(d, std=0.2), dout=n(*shape), dres=n(*shape))


def to_gpu(t):
    return {k: None if v is None else v.cuda() for k, v in t.items()}


def forward64(t, eps=1e-5):
    z = t["x"].double() + (t["y"].double() if t["y"] is not None else 0.0)
    mean = z.mean(-1, keepdim=True)
    rstd = ((z - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    return z, mean, rstd, (z - mean) * rstd * t["gamma"].double() + t["beta"].double()


def within(got, ref, tol, what):
    err = (got.double().cpu() - ref).abs()
    assert bool((err <= tol).all()), (what, float((err - tol).max()), float((err / tol.clamp(min=1e-300)).max()))


def check_forward(t, eps=1e-5, **kw):
    g = to_gpu(t)
    out, mean, rstd = txl.layer_norm_fwd(g["x"], g["gamma"], g["beta"], y=g["y"], eps=eps, **kw)
    torch.cuda.synchronize()
    z, mu, rs, ref = forward64(t, eps)
    d, dt = t["x"].shape[-1], t["x"].dtype
    k = -(-d // 32) + 26
    size = z.abs() + z.abs().mean(-1, keepdim=True)
    half = torch.finfo(dt).eps / 2
    gam = t["gamma"].double().abs()
    within(mean, mu.squeeze(-1), k * U * z.abs().mean(-1), "mean")
    # var's relative error is at most twice that of (z - mean), whose error is k U size
    spread = (size.square().mean(-1) * rs.squeeze(-1).square()).sqrt()
    within(rstd, rs.squeeze(-1), 2 * k * U * spread * rs.squeeze(-1), "rstd")
    within(out, ref, half * ref.abs() + 2 * k * U * (size * rs * gam * (1 + spread[..., None]) + t["beta"].double().abs()), "out")
    return out, mean, rstd


def check_backward(t, mean, rstd, dres, **kw):
    g = to_gpu(t)
    got = txl.layer_norm_bwd(g["dout"], g["x"], g["gamma"], mean, rstd, y=g["y"], dres=g["dres"] if dres else None, **kw)
    torch.cuda.synchronize()
    z = forward64(t)[0]
    mu, rs = mean.cpu().double()[..., None], rstd.cpu().double()[..., None]
    d, dt = t["x"].shape[-1], t["x"].dtype
    xh, do = (z - mu) * rs, t["dout"].double()
    gg = do * t["gamma"].double()
    s1, s2 = gg.mean(-1, keepdim=True), (gg * xh).mean(-1, keepdim=True)
    ref = rs * (gg - s1 - xh * s2)
    xe = (z.abs() + mu.abs()) * rs  # what xh's rounding is relative to
    k = -(-d // 32) + 26
    tol = k * U * rs * (gg.abs() + gg.abs().mean(-1, keepdim=True) + xe * s2.abs() +
                        (xh.abs() + k * U * xe) * (gg.abs() * xe).mean(-1, keepdim=True))
    if dres:
        ref = ref + t["dres"].double()
        tol = tol + 2 * U * (t["dres"].double().abs() + ref.abs())
    within(got["dx"], ref, torch.finfo(dt).eps / 2 * (ref.abs() + tol) + tol, "dx")
    f = lambda a: a.reshape(-1, d)
    within(got["dgamma"], f(do * xh).sum(0), 192 * U * f(do.abs() * xe).sum(0), "dgamma")
    within(got["dbeta"], f(do).sum(0), 192 * U * f(do.abs()).sum(0), "dbeta")
    return got


SIZES = [(1, 1), (3, 2), (5, 7), (1, 512), (22, 512), (130, 33), (70, 256), (64, 1000), (33, 1001), (128, 1024),
         (17, 1536), (9, 2048), (200, 768), (7, 4100), (3, 8192), (2, 16384), (5, 16383), (2000, 64), (700, 96), (2, 3001),
         # more rows than are few, so that they come through the ring in whole and broken stages, or row by row
         (1100, 3000), (1201, 1024), (1030, 8192), (601, 6001), (1500, 1001), (1025, 8200)]


@pytest.mark.parametrize("rows,d", SIZES)
@pytest.mark.parametrize("dtype,add", [(BF, True), (BF, False), (F32, True), (F32, False)])
def test_forward_and_backward_match_fp64(rows, d, dtype, add):
    t = make(rows, d, dtype, add, seed=rows * 31 + d)
    _, mean, rstd = check_forward(t)
    check_backward(t, mean, rstd, dres=add)
    check_backward(t, mean, rstd, dres=not add)


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 512), (BF, 1000), (BF, 2048), (BF, 514), (BF, 77), (BF, 1539),
                                     (F32, 512), (F32, 1100), (F32, 33), (F32, 2049)])
def test_backward_with_few_rows_and_with_one_more(dtype, d):
    """Up to some number of rows no workspace is needed (the columns are summed by
    CTAs of their own); both sides of it."""
    few = max(r for r in range(1, 1 << 13) if txl.layer_norm_bwd_workspace_bytes(r, d, dtype) == 0)
    assert txl.layer_norm_bwd_workspace_bytes(few + 1, d, dtype) > 0
    for rows in (few, few + 1):
        t = make(rows, d, dtype, True, seed=rows + d)
        _, mean, rstd = check_forward(t)
        got = check_backward(t, mean, rstd, dres=True)
        again = check_backward(t, mean, rstd, dres=True)
        assert all(torch.equal(got[k], again[k]) for k in got)


def test_many_rows_and_a_leading_shape():
    t = make(0, 512, BF, True, seed=5, lead=(3, 700))
    out, mean, rstd = check_forward(t)
    assert out.shape == (3, 700, 512) and mean.shape == rstd.shape == (3, 700)
    check_backward(t, mean, rstd, dres=True)


def test_rows_of_one_value_and_a_large_mean():
    """A constant row has variance 0: xh = 0 and rstd = eps^-1/2; a mean of
    300 standard deviations keeps its variance (two passes over the row)."""
    t = make(40, 640, F32, False, seed=6)
    t["x"][::2] = 3.0
    check_forward(t)
    t = make(64, 777, F32, False, seed=7, mean=300.0)
    check_forward(t)


def test_row_that_is_not_finite_leaves_the_others():
    t = make(9, 300, F32, False, seed=8)
    t["x"][4, 7] = float("inf")
    t["x"][5, 8] = float("nan")
    g = to_gpu(t)
    out, mean, rstd = txl.layer_norm_fwd(g["x"], g["gamma"], g["beta"])
    rows = [0, 1, 2, 3, 6, 7, 8]
    ref = forward64({k: (v[rows] if k in ("x",) else v) for k, v in t.items()})[3]
    assert torch.isnan(out[4]).any() and torch.isnan(out[5]).all()
    assert float((out[rows].cpu().double() - ref).abs().max()) < 1e-5


def test_zero_rows():
    x = torch.empty(0, 512, dtype=BF, device="cuda")
    w = torch.ones(512, dtype=BF, device="cuda")
    out, mean, rstd = txl.layer_norm_fwd(x, w, w)
    assert out.shape == (0, 512) and mean.numel() == 0
    g = txl.layer_norm_bwd(x, x, w, mean, rstd)
    torch.cuda.synchronize()
    assert g["dx"].numel() == 0 and not g["dgamma"].any() and not g["dbeta"].any()


def test_gradients_match_differences():
    """Central differences of sum(out dout) of the fp64 formula, in x, gamma
    and beta.  Step h = 1e-4 with |third derivative| of order 1: the difference
    is within 1e-6; the kernel's fp32 gradient within 2e-5."""
    t = make(3, 13, F32, False, seed=9)
    g = to_gpu(t)
    _, mean, rstd = txl.layer_norm_fwd(g["x"], g["gamma"], g["beta"])
    got = txl.layer_norm_bwd(g["dout"], g["x"], g["gamma"], mean, rstd)
    f = lambda u: float((forward64(u)[3] * t["dout"].double()).sum())
    h = 1e-4
    for name, grad in (("x", "dx"), ("gamma", "dgamma"), ("beta", "dbeta")):
        a = t[name].double()
        num = torch.zeros_like(a)
        for i in np.ndindex(*a.shape):
            up, down = a.clone(), a.clone()
            up[i] += h
            down[i] -= h
            num[i] = (f({**t, name: up}) - f({**t, name: down})) / (2 * h)
        assert float((got[grad].cpu().double() - num).abs().max()) < 3e-5, name


def test_same_bits_again_and_in_a_graph():
    t = to_gpu(make(3000, 520, BF, True, seed=10))
    fwd = lambda: txl.layer_norm_fwd(t["x"], t["gamma"], t["beta"], y=t["y"])
    _, mean, rstd = fwd()
    bwd = lambda: txl.layer_norm_bwd(t["dout"], t["x"], t["gamma"], mean, rstd, y=t["y"])
    ref_f, ref_b = fwd(), bwd()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got_f, got_b = fwd(), bwd()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref_f, got_f))
    assert all(torch.equal(ref_b[k], got_b[k]) for k in ref_b)


def test_given_buffers_another_stream_and_a_workspace():
    t = to_gpu(make(500, 260, F32, True, seed=11))
    ref = txl.layer_norm_fwd(t["x"], t["gamma"], t["beta"], y=t["y"])
    rb = txl.layer_norm_bwd(t["dout"], t["x"], t["gamma"], *ref[1:], y=t["y"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    mine = [torch.empty_like(a) for a in ref]
    got = txl.layer_norm_fwd(t["x"], t["gamma"], t["beta"], y=t["y"], out=mine[0], mean=mine[1], rstd=mine[2], stream=st)
    ws = torch.empty(txl.layer_norm_bwd_workspace_bytes(500, 260, F32), dtype=torch.uint8, device="cuda")
    grads = {k: torch.empty_like(v) for k, v in rb.items()}
    gb = txl.layer_norm_bwd(t["dout"], t["x"], t["gamma"], mine[1], mine[2], y=t["y"], stream=st, workspace=ws, grads=grads)
    st.synchronize()
    assert all(a is b for a, b in zip(got, mine)) and all(torch.equal(a, b) for a, b in zip(got, ref))
    assert all(gb[k] is grads[k] and torch.equal(gb[k], rb[k]) for k in rb)


def test_nothing_behind_the_rows_is_written():
    rows, d = 37, 130
    t = to_gpu(make(rows, d, BF, False, seed=12))
    big = torch.full((rows * d + 512,), 7.0, dtype=BF, device="cuda")
    stat = torch.full((2, 128), 7.0, device="cuda")
    txl.layer_norm_fwd(t["x"], t["gamma"], t["beta"], out=big[:rows * d].view(rows, d), mean=stat[0, :rows],
                       rstd=stat[1, :rows])
    assert bool((big[rows * d:] == 7).all()) and bool((stat[:, rows:] == 7).all())
    grads = {"dx": big[:rows * d].view(rows, d), "dgamma": stat[0, :d] if d <= 128 else torch.empty(d, device="cuda"),
             "dbeta": torch.full((d + 64,), 7.0, device="cuda")[:d]}
    txl.layer_norm_bwd(t["dout"], t["x"], t["gamma"], torch.zeros(rows, device="cuda"),
                       torch.ones(rows, device="cuda"), grads=grads)
    assert bool((big[rows * d:] == 7).all())


def test_workspace_of_many_rows_is_checked():
    """Many rows need a workspace: a given one is used up to its end and not beyond, and a
    smaller one is refused."""
    t = to_gpu(make(3001, 260, F32, True, seed=13))
    need = txl.layer_norm_bwd_workspace_bytes(3001, 260, F32)
    assert need > 0
    _, mean, rstd = txl.layer_norm_fwd(t["x"], t["gamma"], t["beta"], y=t["y"])
    want = txl.layer_norm_bwd(t["dout"], t["x"], t["gamma"], mean, rstd, y=t["y"])
    ws = torch.full((need + 256,), 7, dtype=torch.uint8, device="cuda")
    got = txl.layer_norm_bwd(t["dout"], t["x"], t["gamma"], mean, rstd, y=t["y"], workspace=ws[:need])
    torch.cuda.synchronize()
    assert all(torch.equal(want[k], got[k]) for k in want) and bool((ws[need:] == 7).all())
    with pytest.raises(txl.TxlError) as e:
        txl.layer_norm_bwd(t["dout"], t["x"], t["gamma"], mean, rstd, y=t["y"], workspace=ws[:need - 256])
    assert e.value.code == -7
