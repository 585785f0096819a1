"""AdamW on the GPU: fp32 states against fp64 formulas, 8-bit states bit for
bit against the same fp32 operations in numpy, and what a step must leave alone.

Tolerances, 32-bit states: each step rounds m and v three times at most, by
2^-24 of terms no larger than |m| + |g| and v + g^2; the update u = m / (...)
carries those (half of v's through the root), the root, two products, the quotient
(2 ulp) and the step size: under 16 roundings; p adds one of its own a step."""
import math

import numpy as np
import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
SHAPES = [(300, 7), (1,), (256,), (257,), (3, 5, 8), (0,), (1023,), (8192 * 2 + 5,), (4,)]


def tensors(shapes, dtype, std, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.empty(s).normal_(0.0, std, generator=g).to(dtype).cuda() for s in shapes]


def reference(p, grads_by_step, lr, betas, eps, decay, max_norm=None):
    """fp64 AdamW over lists; returns p, m, v and the sizes that errors are relative to."""
    b1, b2 = betas
    p = [x.double().cpu() for x in p]
    m, v, moved = ([torch.zeros_like(x) for x in p] for _ in range(3))
    peak = [torch.zeros_like(x) for x in p]
    for t, gs in enumerate(grads_by_step, 1):
        gs = [g.double().cpu() for g in gs]
        c = 1.0
        if max_norm is not None:
            norm = math.sqrt(sum(float(g.square().sum()) for g in gs))
            c = min(1.0, max_norm / norm)
        for i, g in enumerate(gs):
            g = g * c
            m[i] = b1 * m[i] + (1 - b1) * g
            v[i] = b2 * v[i] + (1 - b2) * g * g
            peak[i] = torch.maximum(peak[i], g.abs())
            den = (v[i] / (1 - b2 ** t)).sqrt() + eps
            p[i] = p[i] - lr * (decay[i] * p[i] + m[i] / (1 - b1 ** t) / den)
            moved[i] += lr * (decay[i] * p[i].abs() + peak[i] / (1 - b1 ** t) / den)
    return p, m, v, peak, moved


def parts(opt, flat):
    return [flat[a:a + p.numel()].view(p.shape).cpu() for p, a in zip(opt.params, opt.starts)]


@pytest.mark.parametrize("pd", [F32, BF])
@pytest.mark.parametrize("gd", [F32, BF])
@pytest.mark.parametrize("max_norm", [None, 0.25, 1e6])
def test_steps_match_fp64(pd, gd, max_norm):
    p = tensors(SHAPES, pd, 0.5, 1)
    start = [x.clone() for x in p]
    g = [torch.empty_like(x, dtype=gd) for x in p]
    decay = [0.01 * (i % 3) for i in range(len(p))]
    opt = txl.AdamW(p, g, lr=1e-2, weight_decay=decay, max_norm=max_norm)
    seen = []
    for s in range(4):
        seen.append(tensors(SHAPES, gd, 0.1 * (s + 1), 10 + s))
        for a, b in zip(g, seen[-1]):
            a.copy_(b)
        opt.step()
    torch.cuda.synchronize()
    assert int(opt.steps) == 4
    rp, rm, rv, peak, moved = reference(start, seen, 1e-2, (0.9, 0.999), 1e-8, decay, max_norm)
    if max_norm is not None:
        norm = math.sqrt(sum(float(x.double().square().sum()) for x in seen[-1]))
        assert abs(float(opt.grad_norm) - norm) <= 64 * U * norm
    # the clip factor is rounded once, from a norm of under 64 roundings
    k = 4 * 4 + (0 if max_norm is None else 4 * 66)
    for i, (m, v, q) in enumerate(zip(parts(opt, opt.exp_avg), parts(opt, opt.exp_avg_sq),
                                      parts(opt, opt.master) if pd == BF else [x.cpu() for x in p])):
        assert bool(((m.double() - rm[i]).abs() <= k * U * (rm[i].abs() + peak[i]) + 1e-45).all())
        assert bool(((v.double() - rv[i]).abs() <= 2 * k * U * (rv[i] + peak[i] ** 2) + 1e-45).all())
        tol = 4 * U * rp[i].abs() + (k + 16) * 2 * U * moved[i]
        assert bool(((q.double() - rp[i]).abs() <= tol).all()), i
        if pd == BF:
            assert torch.equal(p[i].cpu(), q.to(BF))  # the parameter is its master's rounding


def test_zero_gradients_only_decay():
    p = tensors([(1000,)], F32, 1.0, 2)
    start = p[0].clone()
    opt = txl.AdamW(p, [torch.zeros(1000, device="cuda")], lr=1e-3, weight_decay=0.1, max_norm=1.0)
    opt.step()
    assert torch.allclose(p[0], start * (1 - 1e-4), rtol=2 * U, atol=0) and float(opt.grad_norm) == 0.0


# ---------------------------------------------------------------- 8-bit states
M32 = np.uint64(0xFFFFFFFF)


def mix(h):
    h = h.astype(np.uint64)
    h ^= h >> np.uint64(16)
    h = (h * np.uint64(0x6C8E9CF5)) & M32
    h ^= h >> np.uint64(15)
    h = (h * np.uint64(0x2B7E1517)) & M32
    return h ^ (h >> np.uint64(16))


def round_e4m3(q, r16):
    f = np.float32
    low = q < f(2.0 ** -6)
    t = np.where(low, q + f(2.0 ** -6), q).astype(f)
    b = ((t.view(np.uint32) + (r16.astype(np.uint32) << 4)) & np.uint32(0xFFF00000)).view(f)
    return np.minimum(np.where(low, b - f(2.0 ** -6), b).astype(f), f(448.0))


def quantize(x, r16, keep):
    f = np.float32
    a = np.abs(x).reshape(-1, 256)
    top = a.max(1, keepdims=True)
    fine = top > f(2.0 ** -110)
    inv = (f(1.0) / np.where(fine, top, f(1.0))).astype(f) * f(448.0)
    q = np.where(fine, a * inv, f(0.0)).astype(f).reshape(-1)
    c = round_e4m3(q, r16)
    if keep:
        c = np.where(q > 0, np.maximum(c, f(2.0 ** -9)), c)
    return np.copysign(c, x), np.where(fine, top * f(1.0 / 448.0), f(0.0)).astype(f).reshape(-1)


def step8(state, g, key, b1=0.9, b2=0.999):
    """One step of the 8-bit states of a flat fp32 gradient."""
    f = np.float32
    (mc, ms, vc, vs) = state
    m = (mc.reshape(-1, 256) * ms[:, None]).astype(f).reshape(-1)
    r = (vc.reshape(-1, 256) * vs[:, None]).astype(f).reshape(-1)
    m = (m * f(b1)).astype(f) + (g * f(1 - b1)).astype(f)
    v = ((r * r).astype(f) * f(b2)).astype(f) + ((g * g).astype(f) * f(1 - b2)).astype(f)
    root = np.sqrt(v)
    h = mix((np.arange(g.size, dtype=np.uint64) + np.uint64(key)) & M32)
    return (*quantize(m, h & np.uint64(0xFFFF), False), *quantize(root, h >> np.uint64(16), True)), m, v


def step_key(seed, t):
    return int(mix(np.array([(seed + t * 0x9E3779B1) & 0xFFFFFFFF], dtype=np.uint64))[0])


@pytest.mark.parametrize("pd,gd", [(F32, F32), (BF, F32), (BF, BF)])
def test_8bit_states_are_bit_exact(pd, gd):
    shapes = [s for s in SHAPES if s != (0,)]
    p = tensors(shapes, pd, 0.5, 3)
    g = [torch.empty_like(x, dtype=gd) for x in p]
    opt = txl.AdamW(p, g, lr=1e-3, state_bits=8, seed=77)
    total = opt.exp_avg.numel()
    state = (np.zeros(total, np.float32), np.zeros(total // 256, np.float32)) * 2
    for s in range(3):
        # magnitudes over many octaves, so that codes reach e4m3's subnormals and zero
        for a, b, w in zip(g, tensors(shapes, F32, 1.0, 20 + s), tensors(shapes, F32, 4.0, 30 + s)):
            a.copy_(b * torch.exp(w))
        flat = np.zeros(total, np.float32)
        for a, x in zip(opt.starts, g):
            flat[a:a + x.numel()] = x.float().cpu().numpy().reshape(-1)
        opt.step()
        torch.cuda.synchronize()
        state, _, _ = step8(state, flat, step_key(77, s + 1))
        got = [x.float().cpu().numpy() for x in opt.states()]
        for mine, ref in zip(got, state):
            assert np.array_equal(mine, ref)
    assert (np.abs(state[0]) < 2.0 ** -6).any() and (state[0] == 0).any() and (state[2] == 2.0 ** -9).any()


def test_8bit_update_uses_the_unrounded_moments():
    """The first step moves p by lr g / (|g| + eps) whatever the codes become:
    m / (1 - b1) = g and sqrt(v / (1 - b2)) = |g|.  (Not by lr sign(g): an |g| of
    1e-4 makes eps = 1e-8 a 1e-4 of the quotient, 1e-6 of p, over the tolerance.)"""
    p = tensors([(5000,)], F32, 0.5, 4)
    start = p[0].clone()
    g = tensors([(5000,)], F32, 1.0, 5)
    txl.AdamW(p, g, lr=1e-2, state_bits=8).step()
    want = 1e-2 * g[0].double() / (g[0].double().abs() + 1e-8)
    assert float((start.double() - p[0].double() - want).abs().max()) <= 1e-2 * 16 * U + 2 * U


def test_8bit_moving_average_keeps_its_mean():
    """A constant gradient's v under beta2 = 0.999: v_t = g^2 (1 - b2^t) grows by
    less than a code's step each time, yet the mean over elements follows.  The
    code of an element is off by at most one step (2^-3) of sqrt(v): its error
    in v is under 0.3 with standard deviation under 0.15; the mean of 65536
    elements is within 6 * 0.15 / 256 and the bias E[r^2] - E[r]^2 <= (2^-3)^2/4 a
    step's own spread, carried along by the average."""
    n = 65536
    gen = torch.Generator().manual_seed(6)
    size = torch.empty(n).uniform_(0.3, 1.0, generator=gen).cuda()
    p = [torch.zeros(n, device="cuda")]
    opt = txl.AdamW(p, [size.clone()], lr=0.0, state_bits=8, seed=9)
    for _ in range(200):
        opt.step()
    codes, scale = opt.states()[2:]
    v = (codes.float().view(-1, 256) * scale[:, None]).view(-1).double().square()
    want = size.double().square() * (1 - 0.999 ** 200)
    ratio = float((v / want).mean())
    assert 0.97 < ratio < 1.03, ratio


def test_8bit_non_finite_gradient_stays_in_its_block():
    p = tensors([(1024,)], F32, 0.5, 7)
    g = tensors([(1024,)], F32, 1.0, 8)
    g[0][300] = float("nan")
    g[0][600] = float("inf")
    opt = txl.AdamW(p, g, lr=1e-2, state_bits=8)
    opt.step()
    bad = torch.isfinite(opt.exp_avg_scale).logical_not().cpu().tolist()
    assert bad == [False, True, True, False]
    assert bool(torch.isfinite(p[0][:256]).all()) and bool(torch.isfinite(p[0][768:]).all())
    assert int(torch.isfinite(p[0]).logical_not().sum()) == 2


# ---------------------------------------------------------------- the step as a whole
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("bits", [8, 32])
def test_norm_that_is_not_finite_changes_nothing(bad, bits):
    p = tensors(SHAPES, BF, 0.5, 9)
    g = tensors(SHAPES, F32, 1.0, 10)
    opt = txl.AdamW(p, g, lr=1e-2, state_bits=bits, max_norm=1.0)
    opt.step()
    before = [x.clone() for x in p + opt.states() + [opt.master]]
    g[0][3, 3] = bad
    opt.step()
    assert int(opt.steps) == 1 and not math.isfinite(float(opt.grad_norm))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
               for a, b in zip(before, p + opt.states() + [opt.master]))
    g[0][3, 3] = 0.5
    opt.step()
    assert int(opt.steps) == 2 and math.isfinite(float(opt.grad_norm))


@pytest.mark.parametrize("count", [31, 32, 33, 481, 1000])
def test_many_tensors(count):
    """More tensors than one launch's table holds, of 1 to 700 elements."""
    shapes = [(1 + (37 * i) % 700,) for i in range(count)]
    p, g = tensors(shapes, F32, 1.0, 11), tensors(shapes, F32, 1.0, 12)
    start = [x.clone() for x in p]
    opt = txl.AdamW(p, g, lr=1e-2, weight_decay=0.1, max_norm=3.0)
    opt.step()
    torch.cuda.synchronize()
    norm = math.sqrt(sum(float(x.double().square().sum()) for x in g))
    assert abs(float(opt.grad_norm) - norm) <= 64 * U * norm
    for a, s, x in zip(p, start, g):
        ref = s.double() - 1e-2 * (0.1 * s.double() + torch.sign(x).double())
        # |g| c >= 1e-8 * 2^10 leaves eps under 2^-10 of the root: compare where it is
        m = (x.abs() * (3.0 / norm) > 1e-4)
        assert float(((a.double() - ref).abs() * m).max()) <= 1e-2 * 2e-4


def test_neighbours_are_left_alone():
    """Parameters that are slices of one buffer: what lies between stays."""
    buf = torch.full((4096,), 7.0, device="cuda")
    cuts = [(0, 250), (256, 257), (512, 1029), (2048, 3001)]
    p = [buf[a:b] for a, b in cuts]
    g = [torch.ones_like(x) for x in p]
    opt = txl.AdamW(p, g, lr=0.5)
    opt.step()
    inside = torch.zeros(4096, dtype=torch.bool)
    for a, b in cuts:
        inside[a:b] = True
    assert bool((buf.cpu()[~inside] == 7).all()) and bool((buf.cpu()[inside] != 7).all())


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_step_replays_as_eager_steps(bits):
    def build():
        p, g = tensors(SHAPES, BF, 0.5, 13), tensors(SHAPES, F32, 0.1, 14)
        return p, g, txl.AdamW(p, g, lr=1e-2, state_bits=bits, max_norm=0.5, seed=3)

    p, g, opt = build()
    for k in range(4):
        if k == 2:
            opt.set_lr(1e-3)
        opt.step()
    q, h, rep = build()
    rep.step()  # outside the capture once
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rep.step()
    for k in range(1, 4):
        if k == 2:
            rep.set_lr(1e-3)
        graph.replay()
    torch.cuda.synchronize()
    assert int(rep.steps) == 4
    assert all(torch.equal(a, b) for a, b in zip(p, q))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(opt.states(), rep.states()))


@pytest.mark.parametrize("bits,pd", [(8, BF), (32, F32)])
def test_checkpoint_resume_is_identical(bits, pd):
    p, g = tensors(SHAPES, pd, 0.5, 15), tensors(SHAPES, F32, 0.1, 16)
    opt = txl.AdamW(p, g, lr=1e-2, state_bits=bits)
    opt.step()
    sd, at = opt.state_dict(), [x.clone() for x in p]
    opt.step()
    want = [x.clone() for x in p]
    q = [x.clone() for x in at]
    other = txl.AdamW(q, g, lr=5.0, state_bits=bits)
    other.load_state_dict(sd)
    other.step()
    assert int(other.steps) == 2 and all(torch.equal(a, b) for a, b in zip(want, q))


def test_step_on_another_stream():
    p, g = tensors(SHAPES, F32, 0.5, 17), tensors(SHAPES, F32, 0.1, 18)
    q = [x.clone() for x in p]
    a, b = txl.AdamW(p, g, lr=1e-2, max_norm=0.1), txl.AdamW(q, g, lr=1e-2, max_norm=0.1)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        a.step()
        b.step(stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(p, q))


def test_bound_tensors_are_checked():
    p = torch.zeros(8, 8, device="cuda")
    with pytest.raises(ValueError):
        txl.AdamW([p.t()], [p.clone()], lr=1e-3)          # not contiguous
    with pytest.raises(ValueError):
        txl.AdamW([p], [torch.zeros(8, 7, device="cuda")], lr=1e-3)
    with pytest.raises(TypeError):
        txl.AdamW([p.half()], [p], lr=1e-3)
    with pytest.raises(txl.TxlError) as e:
        txl.AdamW([p, p], [p.clone(), p.clone()], lr=1e-3).step()  # one tensor twice
    assert e.value.code == -4
    with pytest.raises(txl.TxlError) as e:
        txl.AdamW([p], [p], lr=1e-3).step()               # the gradient is the parameter
    assert e.value.code == -4
    flat = torch.zeros(64, device="cuda")
    with pytest.raises(txl.TxlError) as e:
        txl.AdamW([flat[1:9]], [p[0]], lr=1e-3).step()
    assert e.value.code == -3
    shared = torch.ones(8, 8, device="cuda")               # one gradient for two parameters is read twice
    txl.AdamW([p, torch.zeros(8, 8, device="cuda")], [shared, shared], lr=1e-3).step()
    assert float((p + 1e-3).abs().max()) < 1e-8


def test_storage_given_away_stays_valid():
    """A parameter that is given other storage after binding: the step goes to the
    memory that was bound, which is still there."""
    p, g = torch.ones(1 << 20, device="cuda"), torch.ones(1 << 20, device="cuda")
    opt = txl.AdamW([p], [g], lr=1e-2)
    old = p.data_ptr()
    p.data = torch.zeros(1 << 20, device="cuda")
    fresh = torch.full((1 << 20,), 5.0, device="cuda")  # would take the freed memory
    assert fresh.data_ptr() != old
    opt.step()
    torch.cuda.synchronize()
    assert bool((p == 0).all()) and bool((fresh == 5).all())


def test_constructor_stream_is_ordered_with_the_current_one():
    """An optimizer with a stream of its own: it sees what the current stream wrote
    before, and set_lr, state_dict and load_state_dict stand in the order of both."""
    big = torch.empty(1 << 28, device="cuda")

    def busy():
        for _ in range(20):  # some 3 ms of the stream it is issued on
            big.fill_(0.0)

    n = 1 << 16
    p, g = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.ones(n, device="cuda")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    p.fill_(2.0)
    opt = txl.AdamW([p], [g], lr=0.0, stream=st)
    start = opt.state_dict()
    busy()
    opt.set_lr(0.5)
    opt.step()
    with torch.cuda.stream(st):
        busy()
    opt.step()
    sd = opt.state_dict()
    assert bool((start["master"] == 2).all()) and int(start["steps"]) == 0
    # constant gradients: m / (1 - b1^t) = 1 and v / (1 - b2^t) = 1, so each step takes off 0.5
    # (1 + 1e-8 and four fp32 roundings of values up to 2 apart from that)
    assert int(sd["steps"]) == 2 and float((sd["master"] - 1).abs().max()) <= 2 * (0.5 * 8 * 2.0 ** -24 + 2.0 ** -24 * 2)
    busy()
    opt.load_state_dict(start)
    opt.step()
    sd = opt.state_dict()
    # (start's lr of 0 came back)
    assert int(sd["steps"]) == 1 and bool((sd["master"] == 2).all())
