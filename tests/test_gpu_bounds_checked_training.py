"""The training operators' variants under the bounds-checked build, in a child
process with TXL_BOUNDS_CHECKED=1: each type, row path and part of the gradients at
parity with fp64 and nothing recorded out of range.

Tolerances: bf16 outputs are rounded once (2^-8 relative; 2^-7 of the largest value
leaves as much for the fp32 arithmetic); fp32 sums of n terms of either sign, n up to
12000, are held to 1e-4 of the sum of magnitudes (chains of under 1200 roundings of
2^-24 give 7e-5)."""
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
g = torch.Generator(device="cuda").manual_seed(2)
n = lambda *s, dt=bf: torch.empty(s, device="cuda").normal_(generator=g).to(dt)


def within(got, ref, tol, what):
    assert bool(((got.double() - ref).abs() <= tol).all()), what


# rows that are few, that come one by one and through the ring (whole and broken stages), of each width and type
for rows, d in [(0, 512), (1, 1), (40, 64), (129, 129), (130, 1024), (5, 4099), (3, 16384), (3001, 24), (3001, 64),
                (2500, 100), (2005, 512), (2005, 1024), (1501, 1001), (1501, 2050), (1300, 4104), (1100, 8192), (1100, 12000)]:
    for dt in (bf, f32):
        x, y, w, b, do, res = n(rows, d, dt=dt), n(rows, d, dt=dt), n(d, dt=dt), n(d, dt=dt), n(rows, d, dt=dt), n(rows, d, dt=dt)
        for yy, rr in ((None, None), (y, None), (None, res)):
            out, mean, rstd = txl.layer_norm_fwd(x, w, b, y=yy)
            got = txl.layer_norm_bwd(do, x, w, mean, rstd, y=yy, dres=rr)
            z = x.double() + (yy.double() if yy is not None else 0.0)
            xh = (z - mean.double()[:, None]) * rstd.double()[:, None]
            gg = do.double() * w.double()
            dx = rstd.double()[:, None] * (gg - gg.mean(1, keepdim=True) - xh * (gg * xh).mean(1, keepdim=True))
            dx = dx if rr is None else dx + rr.double()
            what = (rows, d, dt, yy is None, rr is None)
            if rows and d > 1:
                ref = xh * w.double() + b.double()
                within(out, ref, 2.0 ** -7 * float(ref.abs().max()), what + ("out",))
                within(got["dx"], dx, 2.0 ** -7 * float(dx.abs().max()), what + ("dx",))
            within(got["dbeta"], do.double().sum(0), 1e-4 * do.double().abs().sum(0), what + ("dbeta",))
            size = do.double().abs() * (z.abs() + mean.double().abs()[:, None]) * rstd.double()[:, None]
            within(got["dgamma"], (do.double() * xh).sum(0), 1e-4 * size.sum(0), what + ("dgamma",))

# pairs and single CTAs, split and whole, with and without a mask, each part of the gradients
for B, T, K, N, heads in [(1, 1, 8, 8, False), (3, 100, 136, 72, False), (2, 130, 192, 320, True), (1, 2049, 512, 520, False),
                          (4, 384, 1024, 1024, True), (1, 12000, 128, 136, False)]:
    x, dy, w = n(B, T, K), n(B, T, N), n(N, K)
    xin = x.view(B, T, K // 64, 64).transpose(1, 2).contiguous() if heads else x
    d2, x2 = dy.double().flatten(0, 1), x.double().flatten(0, 1)
    for want in (("dx", "dw", "db"), ("dx",), ("dw",), ("dw", "db"), ("dx", "dw")):
        for relu in (False, True):
            got = txl.linear_bwd(dy, xin, w, relu_in=relu, want=want)
            what = (B, T, K, N, heads, relu, want)
            if "dx" in want:
                dx = got["dx"].transpose(1, 2).flatten(2) if heads else got["dx"]
                ref = (d2 @ w.double()) * ((x2 > 0) if relu else 1.0)
                within(dx.flatten(0, 1), ref, 2.0 ** -7 * float(ref.abs().max()), what + ("dx",))
            if "dw" in want:
                within(got["dw"], d2.t() @ x2, 1e-4 * (d2.abs().t() @ x2.abs()), what + ("dw",))
            if "db" in want:
                within(got["db"], d2.sum(0), 1e-4 * d2.abs().sum(0), what + ("db",))

# every type of parameter, gradient and state; more tensors than one launch's table
for sizes in ((1, 255, 256, 257, 0, 5000), tuple(1 + (37 * i) % 700 for i in range(500))):
    for bits in (8, 32):
        for pd in (bf, f32):
            for gd in (bf, f32):
                for clip in (None, 1.0):
                    p = [n(s, dt=pd) for s in sizes]
                    was = [t.clone() for t in p]
                    o = txl.AdamW(p, [n(s, dt=gd) for s in sizes], lr=1e-2, state_bits=bits, max_norm=clip)
                    o.step()
                    for t, s in zip(p, was):  # by lr at most (and the rounding of bf16)
                        within(t, s.double(), 1.01e-2 + 2.0 ** -8 * s.double().abs(), (len(sizes), bits, pd, gd, clip))
torch.cuda.synchronize()
assert txl.sync_status() == 0
st, first = txl.bounds_status()
assert (st, first) == (0, 0), f"bounds violation recorded: status {st}, record {first:#x}"
print("bounds-checked build: training variants in range")
'''


def test_training_variants_in_range():
    lib = os.path.join(ROOT, "transformer_xl_relative_attn_gb300", "libtxl_checked.so")
    assert os.path.exists(lib), "libtxl_checked.so missing: run __graft_entry__.build()"
    env = dict(os.environ, TXL_BOUNDS_CHECKED="1")
    r = subprocess.run([sys.executable, "-c", "ROOT = %r\n" % ROOT + CHILD], env=env, cwd=ROOT, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "in range" in r.stdout
