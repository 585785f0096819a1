"""Log probabilities and gradient norms under the bounds-checked build, in a child process with
TXL_BOUNDS_CHECKED=1: each type, row path and tile at parity with fp64 and nothing recorded
out of range.

Tolerances: fp32 statistics to 1e-4 of 1 + their size (chains of under 1000 roundings of 2^-24
of terms of one sign); bf16 gradients to their rounding, 2^-7 of the largest value leaving as
much for the arithmetic."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import sys
import torch
sys.path.insert(0, ROOT)
import transformer_xl_relative_attn_gb300 as txl

assert txl.LIB_PATH.endswith("libtxl_checked.so"), txl.LIB_PATH
assert txl.bounds_status() == (0, 0), "not the bounds-checked build, or stale records"
bf, f32 = torch.bfloat16, torch.float32
g = torch.Generator(device="cuda").manual_seed(3)
n = lambda *s, dt=bf, std=1.0: torch.empty(s, device="cuda").normal_(0.0, std, generator=g).to(dt)


def within(got, ref, tol, what):
    assert bool(((got.double() - ref).abs() <= tol).all()), what


# rows that a warp, a CTA and a cluster takes, at every offset against 16 bytes
for rows, V in [(1, 1), (5, 7), (40, 33), (300, 256), (20, 511), (9, 1000), (8, 2047), (6, 2500), (400, 4099), (22, 32768), (2, 131075)]:
    for dt in (bf, f32):
        buf = n(rows, V + 9, dt=dt, std=2.5)
        for off in (0, 1, 3):
            x = buf[:, off:off + V]
            t = torch.randint(-1, V, (rows,), device="cuda", generator=g)
            for top in (0, 1, 8, 32):
                k = min(top, V)
                got = txl.token_logprobs(x, t, top=k)
                logp = torch.log_softmax(x.double(), -1)
                what = (rows, V, dt, off, k)
                lse = torch.logsumexp(x.double(), -1)
                within(got["lse"], lse, 1e-4 * (1 + lse.abs()), what)
                within(got["entropy"], -(logp.exp() * logp).sum(-1), 1e-3, what)
                if k:
                    assert torch.equal(got["top_index"], torch.sort(x.double(), dim=-1, descending=True, stable=True)[1][:, :k]), what
            one = torch.ones(rows, device="cuda")
            out = torch.zeros(rows, V + 5, device="cuda", dtype=dt)
            for extra in ({}, dict(dlse=one, dentropy=one, entropy=got["entropy"])):
                dx = txl.token_logprobs_bwd(x, t, got["lse"], dlogprob=one, out=out[:, 2:2 + V], **extra)
                if not extra:
                    ref = torch.nn.functional.one_hot(t.clamp(min=0), V) - logp.exp()
                    ref = torch.where((t < 0)[:, None], 0.0, ref)
                    within(dx, ref, 2.0 ** -7 if dt is bf else 1e-4, what + ("dx",))
                txl.token_logprobs_bwd(x, t, got["lse"], dlogprob=one, out=x, **extra)
                x.copy_(n(rows, V, dt=dt, std=2.5))
        # ties, masks and rows that are not finite
        x = torch.zeros(rows, V, device="cuda", dtype=dt)
        x[0] = -float("inf")
        x[-1, V // 2] = float("nan")
        txl.token_logprobs(x, t, top=min(V, 20))

# every tile, with and without a bias that lies on 16 bytes
for rows, K, V in [(1, 8, 1), (22, 512, 1000), (127, 72, 255), (129, 200, 257), (300, 64, 100), (999, 520, 1003), (700, 1024, 5000),
                   (2000, 64, 40), (130, 64, 30011), (20, 64, 40000), (520, 64, 14000), (3000, 136, 2000)]:
    x, w, wide = n(rows, K), n(V, K, std=2.0 * K ** -0.5), n(V + 8)
    t = torch.randint(-1, V, (rows,), device="cuda", generator=g)
    for b in (None, wide[:V], wide[1:V + 1]):
        z = x.double() @ w.double().t() + (0.0 if b is None else b.double())
        got = txl.linear_logprobs(x, w, t, bias=b)
        lse = torch.logsumexp(z, -1)
        within(got["lse"], lse, 1e-4 * (1 + lse.abs()), (rows, K, V))
        logp = torch.log_softmax(z, -1)
        within(got["logprob"], torch.where(t < 0, 0.0, logp.gather(1, t.clamp(min=0)[:, None])[:, 0]), 1e-3, (rows, K, V))

for sizes in ((1, 255, 256, 257, 0, 5000, 100001), tuple(1 + (37 * i) % 700 for i in range(500)), tuple(range(100))):
    for scale in (1.0, 1e25, 1e-25):
        p = [n(s, dt=bf if i % 3 else f32, std=scale) for i, s in enumerate(sizes)]
        ref = torch.cat([t.double() for t in p]).norm()
        o = txl.GradNorm(p)
        o.measure()
        assert abs(float(o.norm) / float(ref) - 1) < 1e-4
        o.clip(float(ref) / 3)
        o.measure()
        assert abs(3 * float(o.norm) / float(ref) - 1) < 1e-2
torch.cuda.synchronize()
assert txl.sync_status() == 0
st, first = txl.bounds_status()
assert (st, first) == (0, 0), f"bounds violation recorded: status {st}, record {first:#x}"
print("bounds-checked build: scoring in range")
'''


def test_scoring_variants_in_range():
    lib = os.path.join(ROOT, "transformer_xl_relative_attn_gb300", "libtxl_checked.so")
    assert os.path.exists(lib), "libtxl_checked.so missing: run __graft_entry__.build()"
    env = dict(os.environ, TXL_BOUNDS_CHECKED="1")
    r = subprocess.run([sys.executable, "-c", "ROOT = %r\n" % ROOT + CHILD], env=env, cwd=ROOT, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "in range" in r.stdout
