"""Log probabilities, their gradient, gradient norms and clipping as a training step and a
scoring run use them: a feed-forward block and an output layer, whose gradients go through
token_logprobs_bwd and linear_bwd and are clipped ahead of AdamW, against torch's autograd in
fp64 on the same values; the same step in a graph; linear_logprobs beside them; several
streams at once.

Tolerances: every activation and activation gradient is rounded to bf16 (2^-8 relative to its
size) once per operator, and through the chain of at most six operators gradients are held to
3e-2 of their largest value, each operator alone being held to its own bound elsewhere.  The
logits' rounding alone moves a row's lse by 2^-8 of its largest logit at most."""
import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rnd(*shape, std=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, device="cuda").normal_(0.0, std, generator=g).to(BF)


def near(got, ref, what, tol=3e-2):
    err = float((got.double() - ref).abs().max())
    assert err <= tol * float(ref.abs().max()), (what, err, float(ref.abs().max()))


def parameters(d, di, V, seed):
    return {"w1": rnd(di, d, std=d ** -0.5, seed=seed), "w2": rnd(d, di, std=di ** -0.5, seed=seed + 1),
            "g": (1 + rnd(d, std=0.1, seed=seed + 2).float()).to(BF), "b": rnd(d, std=0.1, seed=seed + 3),
            "out": rnd(V, d, std=2 * d ** -0.5, seed=seed + 4)}


def hidden(p, x):
    f = txl.linear(x, p["w1"], relu=True)
    t = txl.linear(f, p["w2"])
    h, mean, rstd = txl.layer_norm_fwd(x, p["g"], p["b"], y=t)
    return h, (f, t, mean, rstd)


def step(p, grads, x, tokens, weight, norm, opt, limit):
    """One training step: loss = sum of -weight log p; returns the statistics."""
    h, (f, t, mean, rstd) = hidden(p, x)
    z = txl.linear(h, p["out"])
    stats = txl.token_logprobs(z, tokens)
    dz = txl.token_logprobs_bwd(z, tokens, stats["lse"], dlogprob=weight, out=z)  # the logits' place
    head = txl.linear_bwd(dz, h, p["out"], want=("dx", "dw"))
    ln = txl.layer_norm_bwd(head["dx"], x, p["g"], mean, rstd, y=t)
    second = txl.linear_bwd(ln["dx"], f, p["w2"], relu_in=True, want=("dx", "dw"))
    first = txl.linear_bwd(second["dx"], x, p["w1"], want=("dw",))
    for k, v in (("w1", first["dw"]), ("w2", second["dw"]), ("g", ln["dgamma"]), ("b", ln["dbeta"]), ("out", head["dw"])):
        grads[k].copy_(v)
    norm.clip(limit)
    opt.step()
    return stats


def build(d, di, V, seed=30, lr=1e-2):
    p = parameters(d, di, V, seed)
    grads = {k: torch.zeros(v.shape, device="cuda") for k, v in p.items()}
    return p, grads, txl.GradNorm([grads[k] for k in p]), txl.AdamW(list(p.values()), [grads[k] for k in p], lr=lr, seed=4)


def reference(p, x, tokens, weight):
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    z = x.double() + torch.relu(x.double() @ q["w1"].t()) @ q["w2"].t()
    mu = z.mean(-1, keepdim=True)
    h = (z - mu) / ((z - mu).square().mean(-1, keepdim=True) + 1e-5).sqrt() * q["g"] + q["b"]
    logp = torch.log_softmax(h @ q["out"].t(), -1)
    given = torch.where(tokens < 0, 0.0, logp.gather(-1, tokens.clamp(min=0)[..., None])[..., 0])
    (given * weight.double()).sum().backward()
    return given.detach(), {k: v.grad for k, v in q.items()}


@pytest.mark.parametrize("B,T,d,di,V", [(1, 128, 256, 256, 512), (2, 256, 256, 512, 2048)])
def test_a_step_has_the_gradients_of_its_loss(B, T, d, di, V):
    x = rnd(B, T, d, seed=1)
    g = torch.Generator(device="cuda").manual_seed(2)
    tokens = torch.randint(-V // 8, V, (B, T), device="cuda", generator=g).clamp(min=-1)
    weight = torch.where(tokens < 0, 0.0, -1.0 / int((tokens >= 0).sum()))
    p, grads, norm, opt = build(d, di, V)
    given, ref = reference(p, x, tokens, weight)
    total = torch.cat([v.flatten() for v in ref.values()]).norm()
    stats = step(p, grads, x, tokens, weight, norm, opt, 1e9)  # (nothing to clip)
    assert txl.sync_status() == 0
    near(stats["logprob"], given, "logprob")
    for k in ref:
        near(grads[k], ref[k], k)
    assert abs(float(norm.norm) / float(total) - 1) <= 3e-2
    for v, k in zip(norm.norms, p):
        assert abs(float(v) - float(ref[k].norm())) <= 3e-2 * float(ref[k].norm())
    p, grads, norm, opt = build(d, di, V)
    step(p, grads, x, tokens, weight, norm, opt, float(total) / 4)
    for k in ref:
        near(grads[k], ref[k] * (float(total) / 4) / float(norm.norm), k)


def test_the_step_in_a_graph():
    """Captured once and replayed: the weights of the eager steps, bit for bit."""
    B, T, d, di, V = 1, 128, 256, 256, 1024
    x, tokens = rnd(B, T, d, seed=5), torch.arange(T, device="cuda").view(1, T) * 7 % V
    tokens[0, ::9] = -1
    weight = torch.full((B, T), -1.0 / T, device="cuda")
    p, grads, norm, opt = build(d, di, V)
    losses = []
    for _ in range(5):
        losses.append(float((step(p, grads, x, tokens, weight, norm, opt, 0.5)["logprob"] * weight).sum()))
    q, qg, qn, qo = build(d, di, V)
    step(q, qg, x, tokens, weight, qn, qo, 0.5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stats = step(q, qg, x, tokens, weight, qn, qo, 0.5)
    for i in range(1, 5):
        graph.replay()
        assert float((stats["logprob"] * weight).sum()) == losses[i]
    torch.cuda.synchronize()
    assert txl.sync_status() == 0
    assert torch.equal(norm.norm, qn.norm) and torch.equal(norm.norms, qn.norms)
    assert all(torch.equal(p[k], q[k]) for k in p)


def test_scoring_agrees_with_the_training_pass():
    """linear_logprobs of the same hidden states: the logits' rounding to bf16 apart."""
    B, T, d, di, V = 2, 128, 256, 512, 4096
    x, tokens = rnd(B, T, d, seed=6), torch.arange(B * T, device="cuda").view(B, T) * 11 % V
    p = parameters(d, di, V, 40)
    h, _ = hidden(p, x)
    z = txl.linear(h, p["out"])
    a = txl.token_logprobs(z, tokens, top=4)
    b = txl.linear_logprobs(h, p["out"], tokens)
    step_ = 2.0 ** -8 * z.float().abs().amax(-1)
    assert bool(((a["lse"] - b["lse"]).abs() <= step_).all()) and bool(((a["logprob"] - b["logprob"]).abs() <= 2 * step_).all())
    # the alternatives' probabilities, of which the best is at least the token's
    assert bool((a["top_logprob"][..., 0] >= a["logprob"]).all()) and bool((a["top_logprob"].diff(dim=-1) <= 0).all())
    assert torch.equal(a["top_index"][..., 0], z.argmax(-1)) or bool((z.gather(-1, a["top_index"][..., :1])[..., 0] == z.amax(-1)).all())


def test_several_streams_at_once():
    x, w = rnd(300, 256, seed=7), rnd(5000, 256, std=0.1, seed=8)
    z = rnd(300, 5000, std=2.0, seed=9)
    tokens = torch.arange(300, device="cuda") * 13 % 5000
    one = torch.ones(300, device="cuda")
    lse = txl.token_logprobs(z, tokens)["lse"]
    grads = [rnd(n, std=1e-2, seed=10 + i) for i, n in enumerate((100000, 77, 5000))]
    norm = txl.GradNorm(grads)
    jobs = [lambda: list(txl.token_logprobs(z, tokens, top=7).values()),
            lambda: [txl.token_logprobs_bwd(z, tokens, lse, dlogprob=one)],
            lambda: list(txl.linear_logprobs(x, w, tokens).values()),
            lambda: (norm.measure(), [norm.norm.clone(), norm.norms.clone()])[1]]
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
