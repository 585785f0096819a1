"""The training operators together, as a training step uses them: the
feed-forward half of a decoder layer and the attention's output block, forward
with the library's kernels, backward through layer_norm_bwd, linear_bwd and
attn_bwd, and an AdamW step on the weights, against torch's autograd in fp64 on
the same values; and every entry point under the bounds-checked library.

Tolerances: every activation and activation gradient is rounded to bf16 (2^-8
relative to its size) once per operator, and sums of n such roundings of either
sign stay below 2^-8 sqrt(n) of the largest term with room; through the chain of
at most six operators the gradients are held to 3e-2 of their largest value, each
operator alone being held to its own bound elsewhere."""
import os
import subprocess
import sys

import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def rnd(*shape, std=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, device="cuda").normal_(0.0, std, generator=g).to(BF)


def near(got, ref, what, tol=3e-2):
    err = float((got.double() - ref).abs().max())
    assert err <= tol * float(ref.abs().max()), (what, err, float(ref.abs().max()))


def layer_norm64(z, g, b, eps=1e-5):
    mu = z.mean(-1, keepdim=True)
    return (z - mu) / ((z - mu).square().mean(-1, keepdim=True) + eps).sqrt() * g + b


def parameters(d, di, seed):
    return {"w1": rnd(di, d, std=d ** -0.5, seed=seed), "b1": rnd(di, std=0.1, seed=seed + 1),
            "w2": rnd(d, di, std=di ** -0.5, seed=seed + 2), "b2": rnd(d, std=0.1, seed=seed + 3),
            "g": (1 + rnd(d, std=0.1, seed=seed + 4).float()).to(BF), "b": rnd(d, std=0.1, seed=seed + 5)}


def feed_forward(p, x):
    """h = LN(x + W2 relu(W1 x + b1) + b2) and what its backward pass needs."""
    f1 = txl.linear(x, p["w1"], bias=p["b1"], relu=True)
    t = txl.linear(f1, p["w2"], bias=p["b2"])
    h, mean, rstd = txl.layer_norm_fwd(x, p["g"], p["b"], y=t)
    return h, (x, f1, t, mean, rstd)


def feed_forward_bwd(p, dh, saved, grads):
    """Fills grads (fp32, by parameter name); returns x's gradient along the branch
    and along the residual."""
    x, f1, t, mean, rstd = saved
    ln = txl.layer_norm_bwd(dh, x, p["g"], mean, rstd, y=t)
    second = txl.linear_bwd(ln["dx"], f1, p["w2"], relu_in=True)
    first = txl.linear_bwd(second["dx"], x, p["w1"])
    for name, v in (("w1", first["dw"]), ("b1", first["db"]), ("w2", second["dw"]), ("b2", second["db"]),
                    ("g", ln["dgamma"]), ("b", ln["dbeta"])):
        grads[name].copy_(v)
    return first["dx"], ln["dx"]


@pytest.mark.parametrize("B,T,d,di", [(2, 128, 256, 512), (3, 256, 512, 2048)])
def test_feed_forward_block_gradients(B, T, d, di):
    p, x, dh = parameters(d, di, 10), rnd(B, T, d, seed=1), rnd(B, T, d, std=0.1, seed=2)
    h, saved = feed_forward(p, x)
    grads = {k: torch.empty(v.shape, device="cuda") for k, v in p.items()}
    branch, residual = feed_forward_bwd(p, dh, saved, grads)
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    xr = x.double().requires_grad_()
    ref = layer_norm64(xr + torch.relu(xr @ q["w1"].t() + q["b1"]) @ q["w2"].t() + q["b2"], q["g"], q["b"])
    near(h, ref.detach(), "h")
    (ref * dh.double()).sum().backward()
    near(branch.double() + residual.double(), xr.grad, "dx")
    for k in p:
        near(grads[k], q[k].grad, k)


def test_attention_output_block_gradients():
    """LN(x + o_net(attention)): linear_bwd's dx in the heads layout is what
    attn_bwd takes as dout."""
    B, H, L, M, dh_ = 2, 4, 128, 64, 64
    d = H * dh_
    q, k, v = rnd(B, H, L, dh_, seed=3), rnd(B, H, M + L, dh_, seed=4), rnd(B, H, M + L, dh_, seed=5)
    r, u, vb = rnd(M + L, H, dh_, seed=6), rnd(H, dh_, std=0.3, seed=7), rnd(H, dh_, std=0.3, seed=8)
    x, w, dout = rnd(B, L, d, seed=9), rnd(d, d, std=d ** -0.5, seed=10), rnd(B, L, d, std=0.1, seed=11)
    g, b = (1 + rnd(d, std=0.1, seed=12).float()).to(BF), rnd(d, std=0.1, seed=13)
    o, lse = txl.attn_fwd_lse(q, k, v, r, u, vb)
    t = txl.linear(o, w)
    h, mean, rstd = txl.layer_norm_fwd(x, g, b, y=t)
    ln = txl.layer_norm_bwd(dout, x, g, mean, rstd, y=t)
    lin = txl.linear_bwd(ln["dx"], o, w, want=("dx", "dw"))
    assert lin["dx"].shape == (B, H, L, dh_)
    got = txl.attn_bwd(q, k, v, r, u, vb, lin["dx"], out=o, lse=lse)
    torch.cuda.synchronize()
    assert txl.sync_status() == 0
    # autograd on the attention output that the kernel produced, then the attention from its dout
    o64, w64 = o.double().requires_grad_(), w.double().requires_grad_()
    z = x.double() + o64.transpose(1, 2).flatten(2) @ w64.t()
    (layer_norm64(z, g.double(), b.double()) * dout.double()).sum().backward()
    near(lin["dx"], o64.grad, "do")
    near(lin["dw"], w64.grad, "dw")
    ref = txl.attn_bwd(q, k, v, r, u, vb, o64.grad.to(BF), tensor_cores=False)
    for n in ("dq", "dk", "dv", "dr", "du", "dvb"):
        near(got[n], ref[n].double(), n)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_training_step_in_a_graph(bits):
    """Forward, backward and AdamW of one block captured once and replayed: the
    same weights, bit for bit, as the eager steps, and the weights that the forward
    kernels read are the masters' rounding."""
    B, T, d, di = 2, 128, 256, 512

    def build():
        p = parameters(d, di, 30)
        grads = {k: torch.empty(v.shape, device="cuda") for k, v in p.items()}
        opt = txl.AdamW(list(p.values()), [grads[k] for k in p], lr=1e-2, weight_decay=0.01, state_bits=bits,
                        max_norm=1.0, seed=4)
        return p, grads, opt

    x, target = rnd(B, T, d, seed=31), rnd(B, T, d, seed=32)

    def step(p, grads, opt):
        h, saved = feed_forward(p, x)
        feed_forward_bwd(p, h - target, saved, grads)
        opt.step()
        return h

    p, grads, opt = build()
    for _ in range(5):
        step(p, grads, opt)
    q, qg, rep = build()
    step(q, qg, rep)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(q, qg, rep)
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    assert txl.sync_status() == 0
    assert int(opt.steps) == int(rep.steps) == 5
    assert all(torch.equal(p[k], q[k]) for k in p)
    assert all(torch.equal(v, opt.master[a:a + v.numel()].view(v.shape).to(BF)) for v, a in zip(p.values(), opt.starts))


def test_calls_on_several_streams_at_once():
    """Two blocks' gradients and an attention forward, each on a stream of its own and all
    at once: what they give one after the other."""
    d, di = 512, 1024
    p = [parameters(d, di, 50), parameters(d, di, 60)]
    x, dh = [rnd(8, 256, d, seed=70 + i) for i in range(2)], [rnd(8, 256, d, std=0.1, seed=72 + i) for i in range(2)]
    q, k, v, r = rnd(4, 8, 256, 64, seed=74), rnd(4, 8, 512, 64, seed=75), rnd(4, 8, 512, 64, seed=76), rnd(512, 8, 64, seed=77)
    u = rnd(8, 64, std=0.3, seed=78)
    saved = [feed_forward(p[i], x[i])[1] for i in range(2)]

    def grads_of(i):
        g = {n: torch.empty(t.shape, device="cuda") for n, t in p[i].items()}
        dx = feed_forward_bwd(p[i], dh[i], saved[i], g)
        return [*g.values(), *(dx if isinstance(dx, (tuple, list)) else (dx,))]

    jobs = [lambda: grads_of(0), lambda: grads_of(1), lambda: [txl.attn_fwd(q, k, v, r, u, u)]]
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        got = []
        for job, st in zip(jobs, streams):
            with torch.cuda.stream(st):
                got.append([job() for _ in range(3)][-1])
        torch.cuda.synchronize()
        assert txl.sync_status() == 0
        for a, b in zip(want, got):
            assert all(torch.equal(s, t) for s, t in zip(a, b))


CHILD = r'''
import sys
import torch
sys.path.insert(0, ROOT)
import transformer_xl_relative_attn_gb300 as txl

assert txl.LIB_PATH.endswith("libtxl_checked.so"), txl.LIB_PATH
assert txl.bounds_status() == (0, 0), "not the bounds-checked build, or stale records"
bf, f32 = torch.bfloat16, torch.float32
g = torch.Generator(device="cuda").manual_seed(1)
n = lambda *s, dt=bf: torch.empty(s, device="cuda").normal_(generator=g).to(dt)
for rows, d, dt in [(1, 1, f32), (37, 520, bf), (9, 1001, f32), (130, 1024, bf), (5, 4099, bf), (3, 16384, f32),
                    (2005, 1024, bf), (1501, 1001, f32), (1300, 4104, bf), (1501, 1001, bf), (1100, 12000, bf)]:
    x, y, w, b, do = n(rows, d, dt=dt), n(rows, d, dt=dt), n(d, dt=dt), n(d, dt=dt), n(rows, d, dt=dt)
    out, mean, rstd = txl.layer_norm_fwd(x, w, b, y=y)
    z = (x.double() + y.double())
    ref = (z - z.mean(1, keepdim=True)) / (z.var(1, keepdim=True, unbiased=False) + 1e-5).sqrt() * w.double() + b.double()
    assert float((out.double() - ref).abs().max()) <= 2 ** -7 * float(ref.abs().max()) + 1e-4
    got = txl.layer_norm_bwd(do, x, w, mean, rstd, y=y, dres=y)
    assert float((got["dbeta"].double() - do.double().sum(0)).abs().max()) <= 1e-4 * rows
for B, T, K, N, heads in [(1, 1, 8, 8, False), (3, 100, 136, 72, False), (2, 130, 192, 320, True), (2, 1500, 512, 520, False)]:
    x, dy, w = n(B, T, K), n(B, T, N), n(N, K)
    xin = x.view(B, T, K // 64, 64).transpose(1, 2).contiguous() if heads else x
    got = txl.linear_bwd(dy, xin, w, relu_in=True)
    ref = dy.double().flatten(0, 1).t() @ x.double().flatten(0, 1)
    assert float((got["dw"].double() - ref).abs().max()) <= 1e-3 * float(ref.abs().max()) + 1e-4
    dx = got["dx"].transpose(1, 2).flatten(2) if heads else got["dx"]
    ref = (dy.double() @ w.double()) * (x > 0)
    assert float((dx.double() - ref).abs().max()) <= 2 ** -7 * float(ref.abs().max())
for bits in (8, 32):
    for dt in (bf, f32):
        p = [n(s, dt=dt) for s in (1, 255, 256, 257, 5000)]
        o = txl.AdamW(p, [n(t.numel(), dt=f32) for t in p], lr=1e-2, state_bits=bits, max_norm=1.0)
        o.step()
        o.step()
        assert all(bool(torch.isfinite(t).all()) for t in p)
torch.cuda.synchronize()
assert txl.sync_status() == 0
st, first = txl.bounds_status()
assert (st, first) == (0, 0), f"bounds violation recorded: status {st}, record {first:#x}"
print("bounds-checked build: training operators in range")
'''


def test_bounds_checked_build_runs_the_training_operators_in_range():
    lib = os.path.join(ROOT, "transformer_xl_relative_attn_gb300", "libtxl_checked.so")
    assert os.path.exists(lib), "libtxl_checked.so missing: run __graft_entry__.build()"
    env = dict(os.environ, TXL_BOUNDS_CHECKED="1")
    r = subprocess.run([sys.executable, "-c", "ROOT = %r\n" % ROOT + CHILD], env=env, cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "in range" in r.stdout
