"""Refusals of the training operators, on the host: every bad argument is
answered before anything is launched, and the binding refuses what the C calls
could not see."""
import ctypes
import math

import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl
from transformer_xl_relative_attn_gb300 import _lib

A = 0x10000  # fake, aligned device addresses, far from each other and never dereferenced
G = 1 << 30
F32, BF = txl.TXL_F32, txl.TXL_BF16


@pytest.fixture(scope="module")
def lib():
    return txl.load()


def addr(i):
    return A + i * G


def test_layer_norm_fwd_rejects_bad_arguments(lib):
    def call(x=addr(0), y=0, gamma=addr(1), beta=addr(2), rows=64, d=500, eps=1e-5, out=addr(3), mean=addr(4),
             rstd=addr(5), dtype=BF):
        return lib.txl_layer_norm_fwd(x, y, gamma, beta, rows, d, ctypes.c_float(eps), out, mean, rstd, dtype, None)
    for name in ("x", "gamma", "beta", "out", "mean", "rstd"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: addr(7) + 8}) == -3, name
    assert call(rows=-1) == -1 and call(d=0) == -1 and call(dtype=2) == -1
    assert call(eps=-1.0) == -1 and call(eps=math.nan) == -1
    assert call(d=16385) == -2 and call(rows=1 << 31, d=2) == -2 and call(rows=1 << 30, d=2048) == -2
    assert call(out=addr(0)) == -4 and call(y=addr(3)) == -4            # out over x, over y
    assert call(mean=addr(4), rstd=addr(4) + 16) == -4                    # the statistics overlap
    assert call(rows=0, x=None, out=None, mean=None, rstd=None) == 0      # nothing to do


def test_layer_norm_bwd_rejects_bad_arguments(lib):
    need = lib.txl_layer_norm_bwd_workspace_bytes(2000, 500, BF)
    assert need > 0

    def call(dout=addr(0), x=addr(1), y=0, gamma=addr(2), mean=addr(3), rstd=addr(4), dres=0, rows=2000, d=500,
             dx=addr(5), dgamma=addr(6), dbeta=addr(7), dtype=BF, ws=addr(8), ws_bytes=need):
        return lib.txl_layer_norm_bwd(dout, x, y, gamma, mean, rstd, dres, rows, d, dx, dgamma, dbeta, dtype, ws,
                                      ws_bytes, None)
    for name in ("dout", "x", "gamma", "mean", "rstd", "dx", "dgamma", "dbeta"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: addr(9) + 4}) == -3, name
    assert call(rows=-1) == -1 and call(d=-5) == -1 and call(dtype=9) == -1
    assert call(d=16385) == -2
    assert call(ws=None) == -7 and call(ws=addr(8) + 16) == -7 and call(ws_bytes=need - 1) == -7
    assert call(dx=addr(0)) == -4 and call(dres=addr(5)) == -4
    assert call(dgamma=addr(7) + 16) == -4 and call(ws=addr(5)) == -4
    assert lib.txl_layer_norm_bwd_workspace_bytes(64, 20000, BF) == 0
    assert lib.txl_layer_norm_bwd_workspace_bytes(-1, 500, BF) == 0


def test_linear_bwd_rejects_bad_arguments(lib):
    def call(dy=addr(0), x=addr(1), layout=0, B=2, T=100, K=128, w=addr(2), N=136, relu=0, dx=addr(3), dw=addr(4),
             db=addr(5), ws=addr(6), ws_bytes=1 << 28):
        return lib.txl_linear_bwd(dy, x, layout, B, T, K, w, N, relu, dx, dw, db, ws, ws_bytes, None)
    for name in ("dy", "x", "w"):
        assert call(**{name: None}) == -1, name
    assert call(dx=None, dw=None, db=None) == -1 and call(dw=None) == -1      # nothing, or db without dw
    for name in ("dy", "x", "w", "dx", "dw", "db"):
        assert call(**{name: addr(9) + 8}) == -3, name
    assert call(layout=2) == -1 and call(B=0) == -1 and call(T=-1) == -1 and call(K=0) == -1 and call(N=-8) == -1
    assert call(K=132) == -2 and call(N=100) == -2 and call(layout=1, K=72) == -2
    assert call(B=1 << 20, T=1 << 10) == -2 and call(K=1 << 21) == -2
    assert call(dx=addr(1)) == -4 and call(dw=addr(4), db=addr(4) + 64) == -4 and call(dw=addr(2)) == -4
    assert lib.txl_linear_bwd_workspace_bytes(0, 2, 100, 132, 136, 1, 1, 1) == 0
    for want in ((0, 0, 0), (0, 0, 1), (1, 0, 0)):                           # no row is reduced over
        assert lib.txl_linear_bwd_workspace_bytes(0, 2, 5000, 128, 136, *want) == 0, want


def table(*entries):
    t = (_lib.AdamwTensor * max(1, len(entries)))()
    for i, e in enumerate(entries):
        t[i] = _lib.AdamwTensor(*e, 0.0, 0)
    return t


def test_adamw_state_layout(lib):
    t = table((addr(0), addr(1), 1), (addr(2), addr(3), 0), (addr(4), addr(5), 257))
    assert lib.txl_adamw_state_elements(t, 3) == 256 + 0 + 512
    assert lib.txl_adamw_state_elements(t, 0) == -1 and lib.txl_adamw_state_elements(None, 1) == -1
    assert lib.txl_adamw_state_elements(table((addr(0), addr(1), -1)), 1) == -1
    assert lib.txl_adamw_state_elements(table((addr(0), addr(1), 1 << 39)), 1) == -1
    assert lib.txl_adamw_workspace_bytes(table((addr(0), addr(1), -1)), 1) == 0


def test_adamw_rejects_bad_arguments(lib):
    good = table((addr(0), addr(1), 100), (addr(2), addr(3), 300))
    need = lib.txl_adamw_workspace_bytes(good, 2)

    def call(t=good, n=2, pd=BF, gd=F32, bits=8, master=addr(10), m=addr(11), ms=addr(12), v=addr(13), vs=addr(14),
             steps=addr(15), lr=addr(16), b1=0.9, b2=0.999, eps=1e-8, max_norm=1.0, norm=addr(17), ws=addr(18),
             ws_bytes=need):
        return lib.txl_adamw_step(t, n, pd, gd, bits, master, m, ms, v, vs, steps, lr, b1, b2, eps, max_norm, 0, norm,
                                  ws, ws_bytes, None)
    assert call(pd=2) == -1 and call(gd=-1) == -1 and call(bits=16) == -1
    assert call(b1=1.0) == -1 and call(b2=-0.1) == -1 and call(b1=math.nan) == -1
    assert call(eps=-1e-8) == -1 and call(eps=math.inf) == -1
    assert call(max_norm=-1.0) == -1 and call(max_norm=math.inf) == -1 and call(max_norm=math.nan) == -1
    assert call(n=0) == -1 and call(t=None) == -1
    assert call(steps=None) == -1 and call(lr=None) == -1 and call(m=None) == -1 and call(v=None) == -1
    assert call(master=None) == -1 and call(pd=F32) == -1               # bf16 needs a master, fp32 has none
    assert call(ms=None) == -1 and call(bits=32) == -1                  # 8 bits need scales, 32 have none
    assert call(t=table((None, addr(1), 100), (addr(2), addr(3), 300))) == -1
    assert call(t=table((addr(0), None, 100), (addr(2), addr(3), 300))) == -1
    for name in ("master", "m", "ms", "v", "vs"):
        assert call(**{name: addr(20) + 8}) == -3, name
    assert call(steps=addr(15) + 4) == -3 and call(lr=addr(16) + 2) == -3 and call(norm=addr(17) + 1) == -3
    assert call(t=table((addr(0) + 2, addr(1), 100), (addr(2), addr(3), 300))) == -3
    assert call(ws=None) == -7 and call(ws=addr(18) + 128) == -7 and call(ws_bytes=need - 1) == -7
    assert call(t=table((addr(0), addr(1), 100), (addr(0) + 192, addr(3), 300))) == -4   # parameters overlap
    assert call(t=table((addr(0), addr(0) + 64, 100), (addr(2), addr(3), 300))) == -4    # gradient in a parameter
    assert call(m=addr(13)) == -4 and call(steps=addr(10)) == -4 and call(lr=addr(17)) == -4
    assert call(ws=addr(1)) == -4                                       # workspace over a gradient


def test_binding_refuses_what_it_can_see():
    x, w = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA"):
        txl.layer_norm_fwd(x, w, w)
    with pytest.raises(TypeError, match="dtype"):
        txl.layer_norm_fwd(x.double(), w, w)
    with pytest.raises(ValueError):
        txl.layer_norm_fwd(torch.zeros(4, 0), w, w)
    with pytest.raises(ValueError, match="CUDA"):
        txl.layer_norm_bwd(x, x, w, w, w)
    b = torch.zeros(1, 4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        txl.linear_bwd(b, b, torch.zeros(8, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="want"):
        txl.linear_bwd(b, b, torch.zeros(8, 8, dtype=torch.bfloat16), want=("dz",))
    with pytest.raises(ValueError, match="x must be"):
        txl.linear_bwd(b, b[0], torch.zeros(8, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        txl.AdamW([x], [x], lr=1e-3)
    with pytest.raises(ValueError, match="gradient"):
        txl.AdamW([x], [], lr=1e-3)
    with pytest.raises(ValueError, match="state_bits"):
        txl.AdamW([x], [x], lr=1e-3, state_bits=4)
    with pytest.raises(ValueError, match="max_norm"):
        txl.AdamW([x], [x], lr=1e-3, max_norm=0.0)
    with pytest.raises(ValueError, match="weight_decay"):
        txl.AdamW([x], [x], lr=1e-3, weight_decay=[0.1, 0.2])
    with pytest.raises(TypeError, match="dtype"):
        txl.layer_norm_bwd_workspace_bytes(4, 8, torch.float16, device=0)
