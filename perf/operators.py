"""The operators of a decoder layer's training step, as cases to be measured:
LayerNorm forward with its row statistics and backward, the gradients of a
Linear layer, and an AdamW step over many tensors.

`run` computes a case with the library's kernels where `own` is true, and in
plain torch operations (fp32 arithmetic, rounded once at the end) where it is
false; `exact` computes it in fp64 from the formulas.  Sizes are those of the
workloads base512 (d = 512, 22 x 512 rows), large384 (d = 1024, 16 x 384 rows),
seg128 and longmem3200, of their feed-forward layers (4 d), and ragged ones."""
import math

import torch

own = False

#: Elements that share one scale in 8-bit optimizer states; the tensors of a
#: flat state start at multiples of it.
BLOCK = 256
E4M3 = torch.float8_e4m3fn


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _layers(n, d, di):
    """Parameter sizes of n decoder layers: w_qkv, w_o, w1, b1, w2, b2 and two
    LayerNorms' gamma and beta."""
    return [3 * d * d, d * d, di * d, di, d * di, d, d, d, d, d] * n


def listed():
    return [
        # one new token of each of base512's 22 streams: the smallest call
        dict(name="ln_fwd_token", op="ln_fwd", rows=22, d=512, dtype="bf16", add=True),
        # pre-norm layers normalise the whole memory: longmem3200, 8 x 3200 rows
        dict(name="ln_fwd_longmem", op="ln_fwd", rows=25600, d=1024, dtype="bf16", add=False),
        # one stream's segment of seg128
        dict(name="ln_bwd_segment", op="ln_bwd", rows=128, d=512, dtype="bf16", add=True, dres=False),
        # post-norm layer of base512: z = x + y, the gradient over a whole segment
        dict(name="ln_bwd_base512", op="ln_bwd", rows=11264, d=512, dtype="bf16", add=True, dres=False),
        # odd row length and count, fp32, with the residual path's gradient (pre-norm)
        dict(name="ln_bwd_odd", op="ln_bwd", rows=9001, d=1001, dtype="f32", add=False, dres=True),
        # first feed-forward layer over one stream's segment of seg128
        dict(name="linear_bwd_segment", op="linear_bwd", B=1, T=128, K=512, N=2048, heads=False, relu=False),
        # a ragged batch and widths that fill no tile
        dict(name="linear_bwd_ragged", op="linear_bwd", B=3, T=333, K=520, N=1096, heads=False, relu=True),
        # o_net of large384: its input is an attention output in the heads layout
        dict(name="linear_bwd_onet384", op="linear_bwd", B=16, T=384, K=1024, N=1024, heads=True, relu=False),
        # second feed-forward layer of base512: its input came out of a ReLU
        dict(name="linear_bwd_ff512", op="linear_bwd", B=22, T=512, K=2048, N=512, heads=False, relu=True),
        # the parameters of one narrow layer, fp32
        dict(name="adamw_layer", op="adamw", layers=1, d=256, di=512, param="f32", grad="f32", bits=32, clip=False),
        # base512's 12 layers: bf16 weights with an fp32 master copy, clipped gradients
        dict(name="adamw_base512", op="adamw", layers=12, d=512, di=2048, param="bf16", grad="f32", bits=32, clip=True),
        # large384's 18 layers with 8-bit states
        dict(name="adamw_large384_8bit", op="adamw", layers=18, d=1024, di=4096, param="bf16", grad="f32", bits=8,
             clip=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "linear_bwd", "adamw"])
    if op in ("ln_fwd", "ln_bwd"):
        d = rng.choice([256, 512, 1024, 2048]) if rng.random() < 0.4 else _log(rng, 8, 6000)
        rows = min(_log(rng, 1, 40000), max(1, (26 << 20) // d))
        c = dict(op=op, rows=rows, d=d, dtype=rng.choice(["bf16", "bf16", "f32"]), add=rng.random() < 0.5)
        return c if op == "ln_fwd" else dict(c, dres=rng.random() < 0.5)
    if op == "linear_bwd":
        heads = rng.random() < 0.3
        K = 64 * rng.randint(1, 24) if heads else 8 * _log(rng, 8, 256)
        N = 8 * _log(rng, 8, 256)
        B = rng.randint(1, 24)
        T = max(1, min(_log(rng, 1, 1024), int(11e9 / (2.0 * B * K * N))))
        return dict(op=op, B=B, T=T, K=K, N=N, heads=heads, relu=not heads and rng.random() < 0.5)
    d = 8 * _log(rng, 8, 64) + rng.randint(0, 1)
    return dict(op=op, layers=rng.randint(1, 12), d=d, di=rng.randint(1, 4) * d, param=rng.choice(["bf16", "f32"]),
                grad=rng.choice(["f32", "bf16"]), bits=rng.choice([32, 8]), clip=rng.random() < 0.5)


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _size(name):
    return 2 if name == "bf16" else 4


def work(c):
    if c["op"] == "ln_fwd":
        n, e = c["rows"] * c["d"], _size(c["dtype"])
        return {"bytes": n * e * (2 + c["add"]) + 2 * c["d"] * e + 8 * c["rows"], "flops": 8 * n}
    if c["op"] == "ln_bwd":
        n, e = c["rows"] * c["d"], _size(c["dtype"])
        return {"bytes": n * e * (3 + c["add"] + c["dres"]) + c["d"] * (e + 8) + 8 * c["rows"], "flops": 15 * n}
    if c["op"] == "linear_bwd":
        t, k, n = c["B"] * c["T"], c["K"], c["N"]
        return {"bytes": 2 * (t * n + 2 * t * k + n * k) + 4 * (n * k + n), "flops": 4.0 * t * k * n}
    n = sum(_layers(c["layers"], c["d"], c["di"]))
    # the bf16 parameter is written, its master (or the fp32 parameter) read and written
    weights = 8 + (2 if c["param"] == "bf16" else 0)
    states = 16 if c["bits"] == 32 else 4 + 16.0 / BLOCK
    return {"bytes": n * (weights + states + _size(c["grad"])), "flops": 16.0 * n}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
LR, BETAS, EPS, DECAY, MAX_NORM, STEPS, SEED = 1e-3, (0.9, 0.999), 1e-8, 0.01, 0.25, 100, 1234


def _starts(sizes):
    """Where each tensor of a flat state starts, and the state's length."""
    at, starts = 0, []
    for n in sizes:
        starts.append(at)
        at += -(-n // BLOCK) * BLOCK
    return starts, at


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.empty(shape, device="cuda").normal_(mean, std, generator=g).to(dtype)

    s = {"case": c}
    if c["op"] in ("ln_fwd", "ln_bwd"):
        dt, rows, d = _type(c["dtype"]), c["rows"], c["d"]
        s.update(x=normal(rows, d, mean=0.2, dtype=dt), gamma=normal(d, std=0.1, mean=1.0, dtype=dt),
                 beta=normal(d, std=0.1, dtype=dt), y=normal(rows, d, std=0.5, dtype=dt) if c["add"] else None)
        if c["op"] == "ln_bwd":
            s.update(dout=normal(rows, d, std=1e-2, dtype=dt),
                     dres=normal(rows, d, std=1e-2, dtype=dt) if c["dres"] else None)
            z = s["x"].double() + (s["y"].double() if c["add"] else 0.0)  # what a forward pass left behind
            mean = z.mean(1)
            s.update(mean=mean.float(), rstd=(z.var(1, unbiased=False) + 1e-5).rsqrt().float())
        return s
    if c["op"] == "linear_bwd":
        B, T, K, N = c["B"], c["T"], c["K"], c["N"]
        x = normal(B, T, K)
        if c["relu"]:
            x = x.clamp(min=0.0)
        x = x.to(torch.bfloat16)
        if c["heads"]:
            x = x.view(B, T, K // 64, 64).transpose(1, 2).contiguous()
        s.update(x=x, w=normal(N, K, std=0.02, dtype=torch.bfloat16),
                 dy=normal(B, T, N, std=1e-2, dtype=torch.bfloat16))
        return s
    sizes = _layers(c["layers"], c["d"], c["di"])
    starts, total = _starts(sizes)
    at, n = torch.tensor(starts, device="cuda"), torch.tensor(sizes, device="cuda")
    width = torch.tensor(starts[1:] + [total], device="cuda") - at
    tensor = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), width)
    real = torch.arange(total, device="cuda") - at[tensor] < n[tensor]
    # matrices decay, vectors do not
    decay = [DECAY if k > c["di"] else 0.0 for k in sizes]

    def flat(std, mean=0.0):
        return torch.where(real, normal(total, std=std, mean=mean), 0.0)

    # gradients differ from tensor to tensor and from row to row
    size = torch.exp(normal(total // BLOCK)).repeat_interleave(BLOCK)
    p, grad = flat(0.02), flat(1e-3).mul_(size).to(_type(c["grad"]))
    m, v = flat(3e-4).mul_(size), flat(1e-3).mul_(size).square_()
    del size, tensor
    steps = torch.full((1,), STEPS, dtype=torch.int64, device="cuda")
    param = p.to(_type(c["param"]))
    cut = [(a, a + k) for a, k in zip(starts, sizes)]
    states = [m, v]
    if c["bits"] == 8:
        states = _quantize(m, 0) + _quantize(v.sqrt(), 0, keep=True)
    s.update(param=param, steps=steps)
    if own:
        from transformer_xl_relative_attn_gb300 import AdamW

        opt = AdamW([param[a:b] for a, b in cut], [grad[a:b] for a, b in cut], lr=LR, betas=BETAS, eps=EPS,
                    weight_decay=decay, state_bits=c["bits"], max_norm=MAX_NORM if c["clip"] else None, seed=SEED)
        opt.steps.copy_(steps)
        if c["param"] == "bf16":
            opt.master.copy_(p)
        for mine, given in zip(opt.states(), states):
            mine.copy_(given)
        s.update(opt=opt, grads=grad)
        return s
    s.update(grad=grad, master=p if c["param"] == "bf16" else None, states=states, t=STEPS,
             decay=torch.repeat_interleave(torch.tensor(decay, device="cuda"), width),
             index=torch.arange(total, device="cuda") if c["bits"] == 8 else None)
    return s


# --------------------------------------------------------------------------
# 8-bit states: per block one scale amax / 448 and e4m3 codes of x / scale,
# rounded up or down at random so that the mean is kept
# --------------------------------------------------------------------------
M32 = 0xFFFFFFFF


def _mix(h):
    """A hash of 32 bits, of an integer or of an int64 tensor."""
    h = h ^ (h >> 16)
    h = (h * 0x6C8E9CF5) & M32
    h = h ^ (h >> 15)
    h = (h * 0x2B7E1517) & M32
    return h ^ (h >> 16)


def _key(t):
    return _mix((SEED + t * 0x9E3779B1) & M32)


def _round_e4m3(q, r16):
    """q >= 0 to a neighbouring e4m3 value: up with the probability of the
    fraction, by 16 random bits."""
    low = q < 2.0 ** -6  # e4m3's subnormals: steps of 2^-9, as of the numbers from 2^-6 on
    b = torch.where(low, q + 2.0 ** -6, q).view(torch.int32) + (r16 << 4)
    q = (b & ~0xFFFFF).view(torch.float32)
    return torch.where(low, q - 2.0 ** -6, q).clamp(max=448.0)


def _quantize(x, r16, keep=False):
    """[codes, scales] of a flat fp32 state; keep: what is not zero stays so."""
    a = x.abs().view(-1, BLOCK)
    amax = a.amax(1, keepdim=True)
    fine = (amax > 2.0 ** -110) & (amax < math.inf)
    q = torch.where(fine, a * (448.0 / amax), 0.0).view(-1)
    r16 = torch.as_tensor(r16, device=x.device, dtype=torch.int32)
    code = _round_e4m3(q, r16)
    if keep:
        code = torch.where((q > 0) & (code == 0), 2.0 ** -9, code)
    scale = torch.where(amax > 2.0 ** -110, amax / 448.0, torch.where(amax == amax, 0.0, amax)).view(-1)
    return [torch.where(x < 0, -code, code).to(E4M3), scale]


def _values(codes, scale):
    return (codes.float().view(-1, BLOCK) * scale[:, None]).view(-1)


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    return {"ln_fwd": _ln_fwd, "ln_bwd": _ln_bwd, "linear_bwd": _linear_bwd, "adamw": _adamw}[s["case"]["op"]](s)


def _ln_fwd(s):
    if own:
        from transformer_xl_relative_attn_gb300 import layer_norm_fwd

        out, mean, rstd = layer_norm_fwd(s["x"], s["gamma"], s["beta"], y=s["y"])
        return {"out": out, "mean": mean, "rstd": rstd}
    z = s["x"].float()
    if s["y"] is not None:
        z = z + s["y"].float()
    mean = z.mean(1, keepdim=True)
    c = z - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5)
    out = c * rstd * s["gamma"].float() + s["beta"].float()
    return {"out": out.to(s["x"].dtype), "mean": mean.view(-1), "rstd": rstd.view(-1)}


def _ln_bwd(s):
    if own:
        from transformer_xl_relative_attn_gb300 import layer_norm_bwd

        return layer_norm_bwd(s["dout"], s["x"], s["gamma"], s["mean"], s["rstd"], y=s["y"], dres=s["dres"])
    z = s["x"].float()
    if s["y"] is not None:
        z = z + s["y"].float()
    xh = (z - s["mean"][:, None]) * s["rstd"][:, None]
    do = s["dout"].float()
    g = do * s["gamma"].float()
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["x"].dtype), "dgamma": (do * xh).sum(0), "dbeta": do.sum(0)}


def _rows(x):
    """[B, T, K] or heads [B, K / 64, T, 64] as [B T, K]."""
    return (x.transpose(1, 2).flatten(2) if x.dim() == 4 else x).flatten(0, 1)


def _linear_bwd(s):
    if own:
        from transformer_xl_relative_attn_gb300 import linear_bwd

        return linear_bwd(s["dy"], s["x"], s["w"], relu_in=s["case"]["relu"])
    x, dy, w = _rows(s["x"]).float(), _rows(s["dy"]).float(), s["w"].float()
    dx = dy @ w
    if s["case"]["relu"]:
        dx = torch.where(x > 0, dx, 0.0)
    dx = dx.to(torch.bfloat16)
    if s["x"].dim() == 4:
        B, H, T, e = s["x"].shape
        dx = dx.view(B, T, H, e).transpose(1, 2).contiguous()
    return {"dx": dx.view(s["x"].shape), "dw": dy.t() @ x, "db": dy.sum(0)}


def _adamw(s):
    c = s["case"]
    if own:
        opt = s["opt"]
        opt.step()
        out = {"param": s["param"], "master": opt.master if c["param"] == "bf16" else None, "steps": opt.steps,
               "norm": opt.grad_norm if c["clip"] else None}
        states = opt.states()
    else:
        s["t"] += 1
        s["steps"].add_(1)
        t, (b1, b2) = s["t"], BETAS
        g, norm = s["grad"].float(), None
        if c["clip"]:
            norm = torch.sqrt(g.double().square().sum().view(1))
            g = g * torch.where(norm > MAX_NORM, MAX_NORM / norm, 1.0).float()
            norm = norm.float()
        if c["bits"] == 8:
            r = _values(*s["states"][2:])
            m, v = _values(*s["states"][:2]), r * r
        else:
            m, v = s["states"]
        m = m * b1 + g * (1 - b1)
        v = v * b2 + g * g * (1 - b2)
        p = s["param"] if s["master"] is None else s["master"]
        root = torch.sqrt(v)
        u = m / (root * (1 / math.sqrt(1 - b2 ** t)) + EPS)
        p.sub_(p * (s["decay"] * LR) + u * (LR / (1 - b1 ** t)))
        if s["master"] is not None:
            s["param"].copy_(p)
        if c["bits"] == 8:
            h = _mix((s["index"] + _key(t)) & M32)
            new = _quantize(m, h & 0xFFFF) + _quantize(root, h >> 16, keep=True)
        else:
            new = [m, v]
        for old, x in zip(s["states"], new):
            old.copy_(x)
        out = {"param": s["param"], "master": s["master"], "steps": s["steps"], "norm": norm}
        states = s["states"]
    names = ("exp_avg", "exp_avg_scale", "exp_avg_sq_root", "exp_avg_sq_scale") if c["bits"] == 8 else ("exp_avg", "exp_avg_sq")
    out.update(zip(names, states))
    return out


# --------------------------------------------------------------------------
# the same in fp64, from the formulas
# --------------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] in ("ln_fwd", "ln_bwd"):
        z = s["x"].double() if s["y"] is None else s["x"].double() + s["y"].double()
        if c["op"] == "ln_fwd":
            var, mean = torch.var_mean(z, 1, unbiased=False)
            rstd = (var + 1e-5) ** -0.5
            out = torch.addcmul(s["beta"].double(), (z - mean[:, None]) * rstd[:, None], s["gamma"].double())
            return {"out": out, "mean": mean, "rstd": rstd}
        mean, rstd, do = s["mean"].double(), s["rstd"].double(), s["dout"].double()
        xh = (z - mean[:, None]) * rstd[:, None]
        g = do * s["gamma"].double()
        along = (torch.einsum("rd,rd->r", g, xh) / c["d"])[:, None]
        dx = (g - g.sum(1, keepdim=True) / c["d"] - xh * along) * rstd[:, None]
        if s["dres"] is not None:
            dx += s["dres"].double()
        return {"dx": dx, "dgamma": torch.einsum("rd,rd->d", do, xh), "dbeta": do.sum(0)}
    if c["op"] == "linear_bwd":
        x, dy, w = s["x"].double(), s["dy"].double(), s["w"].double()
        if c["heads"]:
            dx = torch.einsum("btn,nhe->bhte", dy, w.view(c["N"], -1, 64))
            dw = torch.einsum("btn,bhte->nhe", dy, x).reshape(c["N"], c["K"])
        else:
            dx, dw = torch.einsum("btn,nk->btk", dy, w), torch.einsum("btn,btk->nk", dy, x)
        if c["relu"]:
            dx = dx * (x > 0)
        return {"dx": dx, "dw": dw, "db": dy.sum((0, 1))}
    g, t = s["grad"].double(), STEPS + 1
    norm = g.norm().view(1)
    if c["clip"]:
        g = g * (MAX_NORM / norm).clamp(max=1.0)
    eight = c["bits"] == 8
    if eight:
        m, v = [(x.double().view(-1, BLOCK) * k.double()[:, None]).view(-1) for x, k in (s["states"][:2], s["states"][2:])]
        v = v ** 2
    else:
        m, v = (x.double() for x in s["states"])
    m, v = torch.lerp(g, m, BETAS[0]), torch.lerp(g * g, v, BETAS[1])
    p = (s["param"] if s["master"] is None else s["master"]).double()
    p = p * (1 - LR * s["decay"].double()) - LR * (m / (1 - BETAS[0] ** t)) / ((v / (1 - BETAS[1] ** t)) ** 0.5 + EPS)
    out = {"param": p, "master": p if c["param"] == "bf16" else None, "steps": None, "norm": norm if c["clip"] else None}
    if eight:  # the codes are rounded at random from fp32 values: they have none in 64 bits
        top = [x.abs().view(-1, BLOCK).amax(1) / 448.0 for x in (m, v ** 0.5)]
        out.update(exp_avg=None, exp_avg_scale=top[0], exp_avg_sq_root=None, exp_avg_sq_scale=top[1])
    else:
        out.update(exp_avg=m, exp_avg_sq=v)
    return out
