"""What a decoder needs behind its last layer, as cases to be measured: log
probabilities of given tokens from logits (with each row's log-sum-exp, entropy
and best alternatives), their gradient, the same log probabilities straight from
hidden states and the output weights, and the norms of many gradients with
clipping.

`run` computes a case with the library's kernels where `own` is true, and in
plain torch operations (fp32 arithmetic, sums of squares in fp64, rounded once at
the end) where it is false; `exact` computes it in fp64 from the formulas.  Row
counts and widths are those of the workloads base512 (d = 512, 22 x 512 rows) and
seg128; vocabularies are generic, from single bytes to 131072 tokens."""
import math

import torch

own = False

BLOCK = 256  # the tensors of a flat gradient buffer start at multiples of it


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decoding step of base512's 22 streams, with the 8 best alternatives
        dict(name="logprobs_token", op="logprobs", rows=22, V=32768, dtype="bf16", top=8, masked=0),
        # byte-level model, a whole base512 segment: short rows
        dict(name="logprobs_bytes", op="logprobs", rows=11264, V=256, dtype="bf16", top=3, masked=0),
        # an odd vocabulary in fp32 whose last columns are padding, with alternatives
        dict(name="logprobs_odd", op="logprobs", rows=1001, V=50021, dtype="f32", top=5, masked=21),
        # the training forward pass of a base512 segment
        dict(name="logprobs_base512", op="logprobs", rows=11264, V=32768, dtype="bf16", top=0, masked=0),
        # gradient of one stream's segment of seg128
        dict(name="bwd_segment", op="bwd", rows=128, V=32768, dtype="bf16", more=False),
        # odd sizes in fp32, with gradients of the log-sum-exp and of the entropy
        dict(name="bwd_odd", op="bwd", rows=999, V=10007, dtype="f32", more=True),
        # gradient of a base512 segment
        dict(name="bwd_base512", op="bwd", rows=11264, V=32768, dtype="bf16", more=False),
        # scoring one token of each of base512's 22 streams: the output weights are read once
        dict(name="head_token", op="head", rows=22, K=512, V=32768, bias=False),
        # ragged rows, width and vocabulary, with a bias
        dict(name="head_ragged", op="head", rows=999, K=520, V=10007, bias=True),
        # scoring a base512 segment
        dict(name="head_base512", op="head", rows=11264, K=512, V=32768, bias=False),
        # norms of one narrow layer's gradients, fp32
        dict(name="norm_layer", op="norm", layers=1, d=256, di=512, grad="f32", clip=False),
        # base512's 12 layers: bf16 gradients of the matrices, fp32 ones of the vectors, clipped
        dict(name="clip_base512", op="norm", layers=12, d=512, di=2048, grad="mixed", clip=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "bwd", "head", "norm"])
    if op == "norm":
        d = 8 * _log(rng, 8, 64) + rng.randint(0, 1)
        return dict(op=op, layers=rng.randint(1, 12), d=d, di=rng.randint(1, 4) * d,
                    grad=rng.choice(["f32", "bf16", "mixed"]), clip=rng.random() < 0.5)
    V = rng.choice([256, 32768, 65536, 131072]) if rng.random() < 0.4 else _log(rng, 32, 131072)
    rows = max(1, min(_log(rng, 1, 12000), (320 << 20) // V))
    if op == "head":
        K = 8 * _log(rng, 8, 128)
        rows = max(1, min(rows, int(180e9 / (2.0 * K * V))))
        return dict(op=op, rows=rows, K=K, V=V, bias=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if dtype == "f32":
        rows = max(1, rows // 2)
    if op == "bwd":
        return dict(op=op, rows=rows, V=V, dtype=dtype, more=rng.random() < 0.4)
    # alternatives of many rows are sorted for in the plain form: fewer rows there
    top = rng.choice([0, 0, 1, 5, 8, 20, 32])
    if top:
        rows = max(1, min(rows, (40 << 20) // V))
    return dict(op=op, rows=rows, V=V, dtype=dtype, top=top, masked=rng.choice([0, 0, V // 20]))


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _size(name):
    return 2 if name == "bf16" else 4


def _layers(c):
    """(matrix?, elements) of each gradient: w_qkv, w_o, w1, b1, w2, b2 and two
    LayerNorms' gamma and beta, per layer."""
    d, di = c["d"], c["di"]
    return [(True, 3 * d * d), (True, d * d), (True, di * d), (False, di), (True, d * di), (False, d), (False, d),
            (False, d), (False, d), (False, d)] * c["layers"]


def _bf16(c, matrix):
    return c["grad"] == "bf16" or (c["grad"] == "mixed" and matrix)


def work(c):
    if c["op"] == "logprobs":
        n = c["rows"] * c["V"]
        return {"bytes": n * _size(c["dtype"]) + c["rows"] * (20 + 12 * c["top"]), "flops": 6.0 * n}
    if c["op"] == "bwd":
        n = c["rows"] * c["V"]
        return {"bytes": 2 * n * _size(c["dtype"]) + c["rows"] * (28 if c["more"] else 16), "flops": (8.0 if c["more"] else 4.0) * n}
    if c["op"] == "head":
        rows, K, V = c["rows"], c["K"], c["V"]
        return {"bytes": 2 * (rows * K + V * K + (V if c["bias"] else 0)) + 20 * rows, "flops": 2.0 * rows * K * V + 6.0 * rows * V}
    sizes = _layers(c)
    n = sum(k for _, k in sizes)
    each = sum(k * (2 if _bf16(c, m) else 4) for m, k in sizes)
    return {"bytes": each * (2 if c["clip"] else 1) + 4 * (len(sizes) + 1), "flops": (3.0 if c["clip"] else 2.0) * n}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
MAX_NORM = 0.25


def _flat(g, sizes):
    """A flat fp32 gradient buffer of tensors of these sizes, and (start, end) of each."""
    cut, at = [], 0
    for n in sizes:
        cut.append((at, at + n))
        at += -(-n // BLOCK) * BLOCK
    x = torch.empty(at, device="cuda").normal_(0.0, 1e-3, generator=g)
    # sizes differ from block to block, as those of gradients from row to row
    x.view(-1, BLOCK).mul_(torch.empty(at // BLOCK, 1, device="cuda").normal_(generator=g).exp_())
    for (_, end), (start, _) in zip(cut, cut[1:] + [(at, at)]):
        x[end:start] = 0.0
    return x, cut


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.empty(shape, device="cuda").normal_(mean, std, generator=g).to(dtype)

    s = {"case": c}
    if c["op"] == "norm":
        sizes = _layers(c)
        half = [k for m, k in sizes if _bf16(c, m)]
        full = [k for m, k in sizes if not _bf16(c, m)]
        grads, parts = {}, []
        for name, ks, dt in (("grad16", half, torch.bfloat16), ("grad32", full, torch.float32)):
            if ks:
                x, cut = _flat(g, ks)
                grads[name] = x = x.to(dt)
                parts += [x[a:b] for a, b in cut]
        # blocks of 256 to tensors, for the norm of each
        blocks = torch.tensor([-(-k // BLOCK) for k in half + full], device="cuda")
        of = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), blocks)
        s.update(grads=grads, of=of, n=len(sizes), max_norm=MAX_NORM)
        if own:
            from transformer_xl_relative_attn_gb300 import GradNorm

            s["norm"] = GradNorm(parts)
        return s
    rows, V = c["rows"], c["V"]
    tokens = torch.randint(0, V, (rows,), device="cuda", generator=g)
    if c["op"] == "head":
        s.update(x=normal(rows, c["K"], dtype=torch.bfloat16),
                 w=normal(V, c["K"], std=2.0 * c["K"] ** -0.5, dtype=torch.bfloat16),
                 bias=normal(V, std=0.5, dtype=torch.bfloat16) if c["bias"] else None)
    else:
        logits = normal(rows, V, std=2.5)
        # the model gives most tokens more than their share
        logits.scatter_add_(1, tokens[:, None], normal(rows, 1, std=4.0, mean=6.0))
        if c.get("masked"):  # columns that pad the vocabulary
            logits[:, V - c["masked"]:] = -math.inf
            tokens %= V - c["masked"]
        s["logits"] = logits.to(_type(c["dtype"]))
    # one row in sixteen is padding, which has no token
    s["tokens"] = torch.where(torch.rand(rows, device="cuda", generator=g) < 1 / 16, -1, tokens)
    if c["op"] == "bwd":
        x = s["logits"].float()  # what a forward pass left behind
        s["lse"] = torch.logsumexp(x, 1)
        p = torch.exp(x - s["lse"][:, None])
        s["entropy"] = s["lse"] - (p * x).sum(1)
        if c["more"]:  # a weight per token, a penalty on the log-sum-exp and an entropy bonus
            s.update(dlogprob=normal(rows, std=1.0 / rows), dlse=s["lse"] * (2e-4 / rows),
                     dentropy=torch.full((rows,), -1e-2 / rows, device="cuda"))
        else:  # the mean of -log p
            s.update(dlogprob=torch.full((rows,), -1.0 / rows, device="cuda"), dlse=None, dentropy=None)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    return {"logprobs": _logprobs, "bwd": _bwd, "head": _head, "norm": _norm}[s["case"]["op"]](s)


def _of_logits(x, tokens):
    """log p of the tokens (0 where there is none), log-sum-exp and entropy of fp32 logits."""
    m = x.amax(1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    s = e.sum(1)
    log_s = torch.log(s)
    entropy = log_s - torch.where(e > 0, e * d, 0.0).sum(1) / s
    given = d.gather(1, tokens.clamp(min=0)[:, None])[:, 0] - log_s
    return {"logprob": torch.where(tokens < 0, 0.0, given), "lse": m[:, 0] + log_s, "entropy": entropy}


def _logprobs(s):
    top = s["case"]["top"]
    if own:
        from transformer_xl_relative_attn_gb300 import token_logprobs

        return token_logprobs(s["logits"], s["tokens"], top=top)
    x = s["logits"].float()
    out = _of_logits(x, s["tokens"])
    if top:  # stable: of equal logits the lowest index comes first
        value, index = torch.sort(x, dim=1, descending=True, stable=True)
        out.update(top_index=index[:, :top].contiguous(), top_logprob=value[:, :top] - out["lse"][:, None])
    return out


def _bwd(s):
    if own:
        from transformer_xl_relative_attn_gb300 import token_logprobs_bwd

        return token_logprobs_bwd(s["logits"], s["tokens"], s["lse"], dlogprob=s["dlogprob"], dlse=s["dlse"],
                                  dentropy=s["dentropy"], entropy=s["entropy"] if s["dentropy"] is not None else None)
    d = s["logits"].float() - s["lse"][:, None]
    p = torch.exp(d)
    g = torch.where(s["tokens"] < 0, 0.0, s["dlogprob"])
    a = -g if s["dlse"] is None else s["dlse"] - g
    dx = a[:, None] * p
    if s["dentropy"] is not None:
        dx = dx - s["dentropy"][:, None] * torch.where(p > 0, p * (d + s["entropy"][:, None]), 0.0)
    dx.scatter_add_(1, s["tokens"].clamp(min=0)[:, None], g[:, None])
    return dx.to(s["logits"].dtype)


def _head(s):
    if own:
        from transformer_xl_relative_attn_gb300 import linear_logprobs

        return linear_logprobs(s["x"], s["w"], s["tokens"], bias=s["bias"])
    x = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        x = x + s["bias"].float()
    return _of_logits(x, s["tokens"])


def _norm(s):
    clip = s["case"]["clip"]
    if clip:  # a limit that follows the norms: every pass has something to clip
        s["max_norm"] *= 0.9999
    if own:
        n = s["norm"]
        n.clip(s["max_norm"]) if clip else n.measure()
        return {"norm": n.norm, "norms": n.norms, "grads": s["grads"] if clip else None}
    blocks = torch.cat([x.double().view(-1, BLOCK).square().sum(1) for x in s["grads"].values()])
    squares = torch.zeros(s["n"], dtype=torch.float64, device="cuda").index_add_(0, s["of"], blocks)
    norm = squares.sum().sqrt().view(1)
    if clip:
        factor = torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0).float()
        [x.copy_(x.float() * factor) for x in s["grads"].values()]
    return {"norm": norm.float(), "norms": squares.sqrt().float(), "grads": s["grads"] if clip else None}


# --------------------------------------------------------------------------
# the same in fp64, from the formulas
# --------------------------------------------------------------------------
def _rows64(x, tokens, top=0):
    """Of fp64 logits, some rows: log p, lse and entropy, and the best `top`."""
    logp = torch.log_softmax(x, 1)
    p = logp.exp()
    valid = tokens >= 0
    out = {"logprob": torch.where(valid, logp[torch.arange(len(x), device="cuda"), tokens * valid], 0.0),
           "lse": torch.logsumexp(x, 1), "entropy": -torch.special.xlogy(p, p).sum(1)}
    if top:
        index = torch.argsort(-x, dim=1, stable=True)[:, :top]
        out.update(top_index=index, top_logprob=torch.take_along_dim(logp, index, 1))
    return out


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm":
        names = list(s["grads"])
        sums = [(s["grads"][k].double() ** 2).view(-1, BLOCK).sum(1) for k in names]
        squares = torch.zeros(s["n"], dtype=torch.float64, device="cuda").scatter_add_(0, s["of"], torch.cat(sums))
        norm = torch.linalg.vector_norm(torch.cat([s["grads"][k].double() for k in names])).view(1)
        factor = (s["max_norm"] * 0.9999 / norm).clamp(max=1.0)
        grads = {k: s["grads"][k].double() * factor for k in names} if c["clip"] else None
        return {"norm": norm, "norms": squares ** 0.5, "grads": grads}
    step = max(1, (64 << 20) // c["V"])  # rows at a time
    if c["op"] == "bwd":
        parts = []
        for r in range(0, c["rows"], step):
            x, t = s["logits"][r:r + step].double(), s["tokens"][r:r + step]
            cut = lambda k: s[k][r:r + step].double()[:, None]  # noqa: E731
            q = (x - cut("lse")).exp()
            one = torch.nn.functional.one_hot(t.clamp(min=0), c["V"])
            dx = cut("dlogprob") * (t >= 0)[:, None] * (one - q)
            if c["more"]:
                dx = dx + cut("dlse") * q - cut("dentropy") * (torch.special.xlogy(q, q) + q * cut("entropy"))
            parts.append(dx)
        return torch.cat(parts)
    parts = []
    for r in range(0, c["rows"], step):
        t = s["tokens"][r:r + step]
        if c["op"] == "head":
            x = torch.einsum("rk,vk->rv", s["x"][r:r + step].double(), s["w"].double())
            x = x if s["bias"] is None else x + s["bias"].double()
        else:
            x = s["logits"][r:r + step].double()
        parts.append(_rows64(x, t, c.get("top", 0)))
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
