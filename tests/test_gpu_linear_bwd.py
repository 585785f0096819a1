"""linear_bwd on the GPU against fp64 products of the same bf16 inputs.

Tolerances, per element: products of bf16 numbers are exact in fp32, so only the
accumulation rounds.  Its error is bounded by (number of additions in a chain)
* 2^-23 (a tensor core may cut off instead of rounding) * the sum of magnitudes:
one addition per 16 terms of a reduction, one per split.  dx adds its rounding to
bf16 (2^-8 relative)."""
import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def make(B, T, K, N, heads, relu, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*s, std=1.0):
        return torch.empty(s, device="cuda").normal_(0.0, std, generator=g)

    x = n(B, T, K)
    if relu:
        x = x.clamp(min=0)
    x = x.to(BF)
    if heads:
        x = x.view(B, T, K // 64, 64).transpose(1, 2).contiguous()
    return n(B, T, N, std=0.5).to(BF), x, n(N, K, std=K ** -0.5).to(BF)


def rows(x):
    x = x.transpose(1, 2).flatten(2) if x.dim() == 4 else x
    return x.flatten(0, 1).double()


def check(dy, x, w, relu, got, want=("dx", "dw", "db")):
    torch.cuda.synchronize()
    assert txl.sync_status() == 0
    d, xr, wr = rows(dy), rows(x), w.double()
    T, N = d.shape

    def within(a, ref, tol, what):
        err = (a.double() - ref).abs()
        assert bool((err <= tol).all()), (what, float((err / tol.clamp(min=1e-300)).max()))

    if "dx" in want:
        mask = (xr > 0).double() if relu else 1.0
        ref = (d @ wr) * mask
        acc = (N / 16 + 4) * 2.0 ** -23 * (d.abs() @ wr.abs())
        within(rows(got["dx"]), ref, 2.0 ** -8 * (ref.abs() + acc) + acc, "dx")
        assert got["dx"].shape == x.shape
    k = (T / 16 + 40) * 2.0 ** -23
    if "dw" in want:
        within(got["dw"], d.t() @ xr, k * (d.abs().t() @ xr.abs()), "dw")
    if "db" in want:
        within(got["db"], d.sum(0), k * d.abs().sum(0), "db")


@pytest.mark.parametrize("B,T,K,N,heads,relu", [
    (1, 1, 8, 8, False, False),         # one row, less than any box
    (1, 1, 512, 2048, False, True),
    (2, 3, 64, 8, True, False),
    (1, 64, 64, 64, False, False),
    (1, 128, 256, 256, False, True),
    (1, 129, 264, 136, False, True),    # one row, one slice, one box over
    (3, 100, 128, 72, True, False),     # batch rows that end inside a step
    (2, 65, 320, 328, True, True),
    (1, 1000, 8, 1000, False, False),
    (1, 777, 1000, 8, False, True),
    (5, 333, 520, 1096, False, True),
    (4, 512, 512, 2048, False, False),
    (22, 512, 2048, 512, False, True),  # base512's second feed-forward layer
    (4, 384, 1024, 1024, True, False),  # o_net of large384
    (1, 20000, 128, 128, False, False),  # a long reduction over few tiles
    (7, 1, 192, 64, True, False),       # single tokens in the heads layout
    (1, 1024, 64, 4104, False, False),  # db without parts and with, and the last columns of a warp
    (1, 1025, 64, 4104, False, False),
    (2, 1024, 512, 2056, False, True),
    (1, 2049, 512, 2056, False, True),
])
def test_gradients_match_fp64(B, T, K, N, heads, relu):
    dy, x, w = make(B, T, K, N, heads, relu, seed=B * T + K + N)
    check(dy, x, w, relu, txl.linear_bwd(dy, x, w, relu_in=relu))


@pytest.mark.parametrize("want", [("dx",), ("dw",), ("dw", "db"), ("dx", "dw")])
def test_part_of_the_gradients(want):
    dy, x, w = make(3, 300, 264, 520, False, True, seed=3)
    got = txl.linear_bwd(dy, x, w, relu_in=True, want=want)
    assert set(got) == set(want)
    check(dy, x, w, True, got, want)


def test_mask_takes_what_is_not_above_zero():
    """Zeros of either sign, negative inputs and NaN stop the gradient."""
    dy, x, w = make(1, 130, 136, 64, False, False, seed=4)
    x[0, :, 0], x[0, :, 1], x[0, :, 2], x[0, :, 3] = 0.0, -0.0, -1.0, 1e-38
    got = txl.linear_bwd(dy, x, w, relu_in=True, want=("dx",))["dx"]
    assert not got[0, :, :3].any() and bool((got[0, :, 3] != 0).any())
    check(dy, x, w, True, {"dx": got}, ("dx",))


def test_a_column_that_is_not_finite_reaches_its_products_only():
    dy, x, w = make(1, 200, 128, 136, False, False, seed=5)
    dy[0, 7, 11] = float("inf")
    got = txl.linear_bwd(dy, x, w)
    torch.cuda.synchronize()
    assert not torch.isfinite(got["dx"][0, 7]).any()
    assert bool(torch.isfinite(got["dx"][0, torch.arange(200) != 7]).all())
    assert not torch.isfinite(got["dw"][11]).any() and not torch.isfinite(got["db"][11])
    keep = torch.arange(136) != 11
    assert bool(torch.isfinite(got["dw"][keep]).all()) and bool(torch.isfinite(got["db"][keep]).all())


def test_gradients_match_differences():
    """Central differences of sum(out dy) in fp64; the function is linear in x
    and in w, so the difference is exact up to fp64."""
    dy, x, w = make(1, 5, 16, 8, False, False, seed=6)
    got = txl.linear_bwd(dy, x, w)
    f = lambda a, b: float(((a @ b.t()) * dy.double()).sum())
    for name, t, grad in (("x", x, "dx"), ("w", w, "dw")):
        for at in range(0, t.numel(), 7):
            up, down = t.double().clone(), t.double().clone()
            up.view(-1)[at] += 1.0
            down.view(-1)[at] -= 1.0
            num = (f(up, w.double()) - f(down, w.double())) / 2 if name == "x" else (f(x.double(), up) - f(x.double(), down)) / 2
            g = float(got[grad].view(-1)[at])
            assert abs(g - num) <= 2.0 ** -8 * abs(num) + 1e-5, (name, at)


def test_linear_and_its_gradients_agree_with_autograd():
    """Two feed-forward layers with a ReLU between, against torch's autograd in fp64
    on the activations the kernels produced."""
    B, T, K, N = 2, 128, 256, 512
    dy, x, w1 = make(B, T, K, N, False, False, seed=7)
    w2 = make(1, 1, N, 256, False, False, seed=8)[2]
    f1 = txl.linear(x, w1, relu=True)
    g = torch.empty(B, T, 256, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(9)).to(BF)
    second = txl.linear_bwd(g, f1, w2, relu_in=True)
    first = txl.linear_bwd(second["dx"], x, w1)
    a, b, c = f1.double().requires_grad_(), w2.double().requires_grad_(), g.double()
    ((a @ b.t()) * c).sum().backward()
    assert float((second["dw"].double() - b.grad).abs().max()) <= 1e-4 * float(b.grad.abs().max())
    masked = a.grad * (f1 > 0)
    assert float((second["dx"].double() - masked).abs().max()) <= 2.0 ** -7 * float(masked.abs().max())
    check(second["dx"], x, w1, False, first)


def test_same_bits_again_and_in_a_graph():
    dy, x, w = make(4, 700, 256, 264, False, True, seed=10)
    run = lambda: txl.linear_bwd(dy, x, w, relu_in=True)
    ref = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(ref[k], got[k]) for k in ref)
    for _ in range(5):
        again = run()
        assert all(torch.equal(ref[k], again[k]) for k in ref)


def test_given_buffers_another_stream_and_a_workspace():
    dy, x, w = make(2, 900, 384, 256, True, False, seed=11)
    ref = txl.linear_bwd(dy, x, w)
    need = txl.linear_bwd_workspace_bytes(x.shape, 256)
    ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device="cuda")
    grads = {k: torch.full_like(v, float("nan")) for k, v in ref.items()}
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = txl.linear_bwd(dy, x, w, stream=st, workspace=ws, grads=grads)
    st.synchronize()
    assert all(got[k] is grads[k] and torch.equal(got[k], ref[k]) for k in ref)


def test_nothing_outside_the_outputs_is_written():
    T, K, N = 77, 72, 88
    dy, x, w = make(1, T, K, N, False, False, seed=12)
    dx = torch.full((T * K + 4096,), 7.0, dtype=BF, device="cuda")
    dw = torch.full((N * K + 4096,), 7.0, device="cuda")
    db = torch.full((N + 256,), 7.0, device="cuda")
    txl.linear_bwd(dy, x, w, grads={"dx": dx[:T * K].view(1, T, K), "dw": dw[:N * K].view(N, K), "db": db[:N]})
    torch.cuda.synchronize()
    assert bool((dx[T * K:] == 7).all()) and bool((dw[N * K:] == 7).all()) and bool((db[N:] == 7).all())


def test_workspace_is_checked():
    """A long reduction over few tiles is split over the GPU's SMs: its parts
    need a workspace, and a missing, small or overlapping one is refused."""
    lib, A, G = txl.load(), 1 << 40, 1 << 30  # addresses that are compared, never dereferenced
    need = lib.txl_linear_bwd_workspace_bytes(0, 1, 100000, 128, 136, 1, 1, 1)
    assert need > 0 and lib.txl_linear_bwd_workspace_bytes(0, 1, 100000, 128, 136, 1, 0, 0) == 0
    call = lambda ws, n: lib.txl_linear_bwd(A, A + G, 0, 1, 100000, 128, A + 2 * G, 136, 0, A + 3 * G, A + 4 * G, A + 5 * G, ws, n, None)
    assert call(None, need) == -7 and call(A + 6 * G, need - 1) == -7 and call(A + 6 * G + 16, need) == -7
    assert call(A + 4 * G, need) == -4
    dy, x, w = make(1, 20000, 128, 136, False, False, seed=13)
    with pytest.raises(txl.TxlError) as e:
        txl.linear_bwd(dy, x, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -7
