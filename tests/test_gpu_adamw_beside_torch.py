"""AdamW beside torch's streams, allocator and autograd."""
import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
U = 2.0 ** -24


def busy(big):
    for _ in range(20):  # some 3 ms of the stream it is issued on
        big.fill_(0.0)


@pytest.mark.parametrize("bits", [8, 32])
def test_step_on_a_stream_that_waited_for_nothing(bits):
    """The constructor's fills stand behind other work on the current stream; a step on
    another stream comes after them all the same."""
    n = 1 << 16
    big = torch.empty(1 << 28, device="cuda")
    p, g, st = torch.full((n,), 2.0, dtype=BF, device="cuda"), torch.ones(n, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    busy(big)
    opt = txl.AdamW([p], [g], lr=0.5, state_bits=bits, max_norm=1e6, stream=None)
    opt.step(stream=st)
    with torch.cuda.stream(st):
        opt.step()
    torch.cuda.synchronize()
    # a constant gradient of 1 moves by lr / (1 + 1e-8) a step (codes of 8 bits: block maxima, which
    # are exact up to the scale's rounding): 16 fp32 roundings of what is at most 2, per step
    assert int(opt.steps) == 2 and float((opt.master - 1.0).abs().max()) <= 2 * (16 * U * 2 + 1e-8)
    assert float((p.float() - 1.0).abs().max()) == 0.0
    assert abs(float(opt.grad_norm) - 256.0) <= 64 * U * 256


def test_memory_of_a_dropped_optimizer_waits_for_its_stream():
    """Dropped while a step on another stream is still to run: its memory, and that of a
    parameter that was given other storage, is not handed out before."""
    n = 1 << 22
    big, st = torch.empty(1 << 28, device="cuda"), torch.cuda.Stream()
    p, g = torch.full((n,), 2.0, dtype=BF, device="cuda"), torch.ones(n, device="cuda")
    opt = txl.AdamW([p], [g], lr=0.5)
    old = [t.data_ptr() for t in (opt.master, opt.exp_avg, opt.exp_avg_sq)]
    was = p.data_ptr()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        busy(big)
    opt.step(stream=st)
    p.data = torch.zeros(1, dtype=BF, device="cuda")
    del opt
    fresh = [torch.full((n,), 5.0, device="cuda") for _ in range(6)]
    narrow = [torch.full((n,), 5.0, dtype=BF, device="cuda") for _ in range(3)]
    assert not {t.data_ptr() for t in fresh} & set(old) and was not in {t.data_ptr() for t in narrow}
    torch.cuda.synchronize()
    assert all(bool((t == 5).all()) for t in fresh + narrow)


def test_a_captured_step_on_a_further_stream():
    """A capture on a stream that no step ran on before: nothing outside it is waited for,
    and an eager step on that stream still is ordered."""
    n = 1000
    p, g, st = torch.full((n,), 2.0, device="cuda"), torch.ones(n, device="cuda"), torch.cuda.Stream()
    opt = txl.AdamW([p], [g], lr=0.5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        opt.step()
        opt.step(stream=st)
    assert int(opt.steps) == 0
    graph.replay()
    torch.cuda.synchronize()
    opt.step(stream=st)
    torch.cuda.synchronize()
    assert int(opt.steps) == 3 and float((p - 0.5).abs().max()) <= 3 * (16 * U * 2 + 1e-8)


def test_an_optimizer_made_in_a_capture():
    """Its fills are part of the graph; a step on another stream does not wait for them."""
    n = 1000
    p, g, st = torch.full((n,), 2.0, device="cuda"), torch.ones(n, device="cuda"), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt = txl.AdamW([p], [g], lr=0.5)
        opt.step()
    graph.replay()
    torch.cuda.synchronize()
    assert int(opt.steps) == 1
    opt.step(stream=st)
    torch.cuda.synchronize()
    assert int(opt.steps) == 2 and float((p - 1.0).abs().max()) <= 2 * (16 * U * 2 + 1e-8)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_autograd_notices_a_step(dtype):
    """Between a forward and its backward pass a step changes the values that the gradient is
    made from: autograd has to refuse, as after torch's own in-place operations."""
    p, x = torch.ones(64, dtype=dtype, device="cuda", requires_grad=True), torch.ones(64, dtype=dtype, device="cuda", requires_grad=True)
    opt = txl.AdamW([p], [torch.ones(64, device="cuda")], lr=0.5)
    y = (p * x).sum()
    before = p._version
    opt.step()
    assert p._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    (p * x).sum().backward()
    assert torch.equal(x.grad, p.detach())


def test_parameters_made_in_inference_mode():
    """They have no version counter that counts; steps work on them as before."""
    with torch.inference_mode():
        p = torch.ones(64, device="cuda")
    opt = txl.AdamW([p], [torch.ones(64, device="cuda")], lr=0.5)
    opt.step()
    assert float((p - 0.5).abs().max()) <= 16 * U


def test_made_on_a_side_stream_and_stepped_on_the_default_one():
    n = 1 << 16
    big, st = torch.empty(1 << 28, device="cuda"), torch.cuda.Stream()
    p, g = torch.full((n,), 2.0, dtype=BF, device="cuda"), torch.ones(n, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        busy(big)
        opt = txl.AdamW([p], [g], lr=0.5)
    opt.step()
    opt.step(stream=torch.cuda.default_stream())
    opt.step(stream=0)
    torch.cuda.synchronize()
    assert int(opt.steps) == 3 and float((opt.master - 0.5).abs().max()) <= 3 * (16 * U * 2 + 1e-8)
