"""GradNorm on the GPU against fp64.

Tolerances, U = 2^-24: a sum of squares is made of non-negative terms, each squared with one
rounding and then part of A additions at most, so it is off by U (A + 1) of its value: per
piece of max(16 KB, 1 / 1216 of all, up to a multiple of 4 KB) a thread of 256 adds one 16-byte
vector per 4 KB to its sums, which meet in 8 + 5 + 8 additions; the P pieces in P / 32 + 5 (a
tensor's) or P / 256 + 13 (all).  Its root is off by half of that and one rounding.  A clipped
value has the factor's error, that of its quotient, and a product's (2 U), and one rounding to
its type."""
import math

import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def make(sizes, dtypes, seed=0, std=1e-2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.empty(n, device="cuda").normal_(0.0, std, generator=g).to(dtypes[i % len(dtypes)]) for i, n in enumerate(sizes)]


def relative(grads):
    """Relative error of a norm."""
    total = sum(g.numel() * g.element_size() for g in grads)
    piece = max(4, -(-total // (1216 * 4096)) + 8)  # (8: for a GPU of fewer SMs)
    pieces = total / (piece * 4096) + len(grads)
    return U * ((piece + 21 + pieces / 32 + 14) / 2 + 2)


def reference(grads):
    norms = torch.stack([g.double().norm() for g in grads])
    return norms, norms.norm()


SIZES = {"one": [1], "few": [5, 0, 1, 300], "ragged": [1, 7, 8, 9, 255, 256, 257, 4095, 4096, 4097, 8191, 8192, 8193, 16385, 100003],
         "layer": [196608, 65536, 131072, 512, 131072, 256, 256, 256, 256, 256], "nothing": [0, 0],
         "many": [1 + (37 * i) % 700 for i in range(1100)], "edges": [100] * 32, "more": [100] * 33, "table": [3] * 480, "next": [3] * 481,
         "large": [40_000_001, 12, 9_999_999]}


@pytest.mark.parametrize("name", SIZES)
@pytest.mark.parametrize("dtypes", [(F32,), (BF,), (BF, F32, F32)], ids=["f32", "bf16", "mixed"])
def test_norms_and_clipping(name, dtypes):
    grads = make(SIZES[name], dtypes, seed=len(name))
    was = [g.clone() for g in grads]
    norms, norm = reference(grads)
    tol = relative(grads)
    n = txl.GradNorm(grads)
    n.measure()
    assert n.norm.shape == (1,) and n.norms.shape == (len(grads),) and n.norm.dtype is n.norms.dtype is F32
    assert bool(((n.norms.double() - norms).abs() <= tol * norms).all())
    assert abs(float(n.norm) - float(norm)) <= tol * float(norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, was))
    first = n.norm.clone(), n.norms.clone()
    n.measure()
    assert torch.equal(first[0], n.norm) and torch.equal(first[1], n.norms)
    if not norm > 0:
        n.clip(1.0)
        assert float(n.norm) == 0.0 and bool((n.norms == 0).all())
        return
    n.clip(float(norm) * 1.01)  # nothing to do
    assert all(torch.equal(a, b) for a, b in zip(grads, was)) and torch.equal(first[0], n.norm)
    limit = float(norm) * 0.3
    n.clip(limit)
    assert torch.equal(first[0], n.norm) and torch.equal(first[1], n.norms)  # before the scaling
    factor = limit / norm
    for a, b in zip(grads, was):
        ref, half = b.double() * factor, torch.finfo(b.dtype).eps / 2
        e = tol + 3 * U
        assert bool(((a.double() - ref).abs() <= ref.abs() * (e + half * (1 + e)) + 2.0 ** -133).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [2.0 ** 126, 1e30, 1e25, 2.0 ** 64, 1e-12, 1e-14, 1e-20, 1e-30, 1e-37])
def test_squares_beyond_the_range(dtype, scale):
    grads = [(g.double() * scale).to(dtype) for g in make([5000, 3, 700, 20000], (F32,), seed=3, std=0.01)]
    norms, norm = reference(grads)
    n = txl.GradNorm(grads)
    n.measure()
    assert abs(float(n.norm) / float(norm) - 1) <= relative(grads)
    assert bool(((n.norms.double() / norms - 1).abs() <= relative(grads)).all())
    if 2.0 ** -120 < float(norm):
        n.clip(float(norm) / 2)
        n.measure()
        assert abs(float(n.norm) / float(norm) * 2 - 1) <= (0.01 if dtype is BF or scale < 1e-30 else 1e-5)


def test_a_wide_range_within_and_between_tensors():
    for dtype in (F32, BF):
        a, b, c = make([70000, 5000, 9000], (F32,), seed=4, std=1.0)
        grads = [(a * 1e25).to(dtype), (b * 1e-25).to(dtype), (c * 1e-3).to(dtype), torch.zeros(50, device="cuda", dtype=dtype)]
        grads[0][1000:] = 0.0
        grads[1][7] = 1e-35
        norms, norm = reference(grads)
        n = txl.GradNorm(grads)
        n.measure()
        assert bool(((n.norms.double() - norms).abs() <= relative(grads) * norms).all())
        assert abs(float(n.norm) / float(norm) - 1) <= relative(grads)
    tiny = torch.full((100,), 2.0 ** -149, device="cuda")  # the smallest number of the type
    n = txl.GradNorm([tiny])
    n.measure()
    assert float(n.norm) == 10 * 2.0 ** -149


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norms_that_are_not_finite_change_nothing(bad, dtype):
    for size, at in ((5000, 17), (5001, 5000), (200000, 199999)):
        grads = make([300, size, 40], (dtype,), seed=5)
        grads[1][at] = bad
        was = [g.clone() for g in grads]
        n = txl.GradNorm(grads)
        n.clip(1e-3)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(grads, was))
        assert not math.isfinite(float(n.norm)) and math.isnan(float(n.norm)) == math.isnan(bad)
        assert torch.isfinite(n.norms).tolist() == [True, False, True]
    big = torch.full((4096,), 3e38, device="cuda")  # finite values, whose norm is not
    n = txl.GradNorm([big])
    n.clip(1.0)
    assert math.isinf(float(n.norm)) and bool((big == 3e38).all())


def test_streams_graphs_and_versions():
    grads = make([300000, 1000, 77], (BF, F32), seed=6)
    was = [g.clone() for g in grads]
    n = txl.GradNorm(grads)
    n.clip(0.5)
    ref, ref_norm = [g.clone() for g in grads], n.norm.clone()
    versions = [g._version for g in grads]
    n.measure()
    assert [g._version for g in grads] == versions
    n.clip(0.5)
    assert all(g._version > v for g, v in zip(grads, versions))
    side = torch.cuda.Stream()
    for given in (side, side.cuda_stream):
        for g, w in zip(grads, was):
            g.copy_(w)
        side.wait_stream(torch.cuda.current_stream())
        n.clip(0.5, stream=given)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(grads, ref)) and torch.equal(n.norm, ref_norm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n.clip(0.5)
    for _ in range(2):
        for g, w in zip(grads, was):
            g.copy_(w)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(grads, ref)) and torch.equal(n.norm, ref_norm)
    # two objects over different tensors on two streams at once
    other = make([200000, 5], (F32,), seed=7)
    m = txl.GradNorm(other)
    m.measure()
    want = m.norm.clone()
    for g, w in zip(grads, was):
        g.copy_(w)
    torch.cuda.synchronize()
    m.norm.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    n.clip(0.5, stream=streams[0])
    m.measure(stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(m.norm, want) and torch.equal(n.norm, ref_norm) and all(torch.equal(a, b) for a, b in zip(grads, ref))


def test_the_memory_lives_as_long_as_the_object():
    n = txl.GradNorm(make([1 << 20], (F32,), seed=8))
    n.measure()
    want = n.norm.clone()
    del n.grads[:]
    torch.empty(1 << 20, device="cuda").fill_(9.0)
    n._call(0.0, None)
    assert torch.equal(n.norm, want)


def test_more_than_2_to_32_elements():
    x = torch.full((2 ** 32 + 5,), 0.5, device="cuda", dtype=BF)
    x[-3:] = 4096.0
    n = txl.GradNorm([x, x[:8].clone()])
    n.clip(256.0)
    want = math.sqrt((2 ** 32 + 2) * 0.25 + 3 * 4096.0 ** 2)
    assert abs(float(n.norms[0]) / want - 1) <= relative(n.grads)
    factor = 256.0 / math.sqrt(want ** 2 + 8 * 0.25)
    half = 2.0 ** -8 + 1e-5
    assert abs(float(x[0]) / (0.5 * factor) - 1) <= half and abs(float(x[-1]) / (4096 * factor) - 1) <= half
    assert bool((x[: -3] == x[0]).all()) and bool((x[-3:] == x[-1]).all())


def test_the_library_call_alone():
    """Without norms; a workspace of the size asked for, and nothing written behind it."""
    from transformer_xl_relative_attn_gb300 import _lib

    lib = txl.load()
    grads = make([70000, 0, 33], (BF, F32), seed=12)
    table = (_lib.GradTensor * 3)()
    for i, g in enumerate(grads):
        table[i] = _lib.GradTensor(g.data_ptr(), g.numel(), txl.TXL_BF16 if g.dtype is BF else txl.TXL_F32, 0)
    need = lib.txl_grad_norm_workspace_bytes(table, 3)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    norm = torch.zeros(2, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.txl_grad_norm(table, 3, 0.0, norm.data_ptr(), None, ws.data_ptr(), need, stream) == 0
    want = float(reference(grads)[1])
    assert abs(float(norm[0]) / want - 1) <= relative(grads) and float(norm[1]) == 0.0
    assert bool((ws[need:] == 255).all())
    assert lib.txl_grad_norm(table, 3, want / 2, norm.data_ptr(), None, ws.data_ptr(), need, stream) == 0
    assert abs(float(reference(grads)[1]) / want * 2 - 1) <= 1e-2


def test_bad_tensors_are_refused():
    x = torch.zeros(64, 64, device="cuda")
    for bad, error in (([x.t()[:, :5]], ValueError), ([x, x.cpu()], ValueError), ([x.double()], TypeError), ([x.half()], TypeError),
                       ([], ValueError), ([3.0], TypeError)):
        with pytest.raises(error):
            txl.GradNorm(bad)
    n = txl.GradNorm([x, x])  # twice the same: measured, but not scaled twice
    x.fill_(1.0)
    n.measure()
    assert abs(float(n.norm) - math.sqrt(2) * 64) <= 1e-4
    with pytest.raises(txl.TxlError) as e:
        n.clip(1.0)
    assert e.value.code == -4 and bool((x == 1).all())
    with pytest.raises(txl.TxlError) as e:
        txl.GradNorm([x.view(-1)[1:]]).measure()
    assert e.value.code == -3
    for limit in (0.0, -1.0, math.nan):
        with pytest.raises(ValueError):
            n.clip(limit)
    for limit in (math.inf, 1e-39):
        with pytest.raises(txl.TxlError) as e:
            n.clip(limit)
        assert e.value.code == -1


def test_clipping_before_an_optimizer_step_is_its_own_clipping():
    """GradNorm.clip and then AdamW without a limit: AdamW's step with that limit, to the rounding
    of the clipped gradients."""
    p = make([5000, 300], (F32,), seed=9, std=1.0)
    q = [t.clone() for t in p]
    g = make([5000, 300], (F32,), seed=10, std=1.0)
    h = [t.clone() for t in g]
    one = txl.AdamW(p, g, lr=1e-2, max_norm=1.0)
    two = txl.AdamW(q, h, lr=1e-2)
    one.step()
    n = txl.GradNorm(h)
    n.clip(1.0)
    two.step()
    assert abs(float(n.norm) / float(one.grad_norm) - 1) <= 1e-5
    assert all(float((a - b).abs().max()) <= 1e-6 for a, b in zip(one.states() + p, two.states() + q))
