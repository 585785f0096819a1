"""Refusals of the token log probabilities, on the host: every bad argument is answered
before anything is launched."""
import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl
from transformer_xl_relative_attn_gb300 import logprobs

A = 0x10000  # fake, aligned device addresses, far from each other and never dereferenced
G = 1 << 30
F32, BF = txl.TXL_F32, txl.TXL_BF16


@pytest.fixture(scope="module")
def lib():
    return txl.load()


def addr(i):
    return A + i * G


def test_token_logprobs_rejects_bad_arguments(lib):
    def call(x=addr(0), ld=500, t=addr(1), rows=64, V=500, top=4, lp=addr(2), lse=addr(3), ent=addr(4), ti=addr(5),
             tl=addr(6), dtype=BF):
        return lib.txl_token_logprobs(x, ld, t, rows, V, top, lp, lse, ent, ti, tl, dtype, None)
    for name in ("x", "t", "lp", "lse", "ent", "ti", "tl"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: addr(8) + 1}) == -3, name
    assert call(t=addr(1) + 4) == -3 and call(ti=addr(5) + 4) == -3 and call(lse=addr(3) + 2) == -3
    assert call(x=addr(0) + 2, dtype=F32) == -3
    assert call(top=0) == -1                                             # alternatives that are not asked for
    assert call(rows=-1) == -1 and call(V=0) == -1 and call(dtype=2) == -1 and call(top=-1) == -1
    assert call(ld=499) == -1 and call(V=3, top=4) == -1
    assert call(top=33) == -2 and call(V=(1 << 24) + 1, ld=1 << 31) == -2
    assert call(rows=1 << 31, ld=512) == -2 and call(rows=1 << 20, ld=(1 << 20) + 1) == -2
    assert call(lp=addr(3)) == -4 and call(lse=addr(1) + 8) == -4 and call(ent=addr(0) + 64) == -4
    assert call(ti=addr(6)) == -4 and call(tl=addr(0) + 63 * 1000) == -4
    assert call(rows=0, x=None, t=None, lp=None, lse=None, ent=None) == 0  # nothing to do


def test_token_logprobs_bwd_rejects_bad_arguments(lib):
    def call(x=addr(0), ld=500, t=addr(1), lse=addr(2), ent=addr(3), g=addr(4), dl=addr(5), dh=addr(6), rows=64, V=500,
             dx=addr(7), ldd=500, dtype=BF):
        return lib.txl_token_logprobs_bwd(x, ld, t, lse, ent, g, dl, dh, rows, V, dx, ldd, dtype, None)
    for name in ("x", "t", "lse", "dx", "ent"):
        assert call(**{name: None}) == -1, name
    for name in ("x", "t", "lse", "dx", "ent", "g", "dl", "dh"):
        assert call(**{name: addr(9) + 1}) == -3, name
    assert call(g=None, dl=None, dh=None, ent=None) == -1               # nothing to take the gradient of
    assert call(dh=None) == -1                                           # an entropy without its gradient
    assert call(rows=-1) == -1 and call(V=0) == -1 and call(ld=499) == -1 and call(ldd=499) == -1 and call(dtype=7) == -1
    assert call(rows=1 << 20, ldd=(1 << 20) + 1) == -2
    assert call(dx=addr(0), ldd=501) == -4 and call(dx=addr(0) + 2) == -4 and call(dx=addr(2)) == -4
    assert call(g=addr(7) + 64) == -4


def test_binding_refuses_what_it_can_see():
    x, t = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    f = torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        txl.token_logprobs(x, t)
    with pytest.raises(ValueError, match="CUDA"):
        txl.token_logprobs_bwd(x, t, f, dlogprob=f)
    for bad in (x.double(), x.half()):
        with pytest.raises(TypeError, match="dtype"):
            txl.token_logprobs(bad, t)
    for bad in (torch.zeros(4, 0), torch.tensor(1.0), None):
        with pytest.raises(ValueError, match="logits"):
            txl.token_logprobs(bad, t)


def test_distance_of_rows():
    x = torch.zeros(4, 6, 10)
    assert logprobs._rows(x, "x") == (24, 10, 10)
    assert logprobs._rows(x[..., :7], "x") == (24, 7, 10)
    assert logprobs._rows(x[:, 2, 1:4], "x") == (4, 3, 60)
    assert logprobs._rows(x[1, 1, 2:5], "x") == (1, 3, 3)
    assert logprobs._rows(x[:, :1, :9], "x") == (4, 9, 60)
    assert logprobs._rows(x[..., :1], "x") == (24, 1, 10)
    assert logprobs._rows(torch.zeros(0, 5), "x") == (0, 5, 5)
    for bad in (x[:, :5, :9], x[..., ::2], x.transpose(0, 1)[..., :9], x[0, :1].expand(6, 10), x[0].t()):
        with pytest.raises(ValueError):
            logprobs._rows(bad, "x")


@pytest.mark.parametrize("axis", range(2))
@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32 + 64])
def test_sizes_of_2_to_31(monkeypatch, axis, big):
    monkeypatch.setattr(logprobs, "_need", lambda *args, **kw: None)
    monkeypatch.setattr(logprobs, "_on_gpu", lambda *args, **kw: None)
    x = torch.empty((big, 2) if axis == 0 else (2, big), dtype=torch.bfloat16, device="meta")
    t, f = torch.empty(x.shape[0], dtype=torch.int64, device="meta"), torch.empty(x.shape[0], device="meta")
    for call in (lambda: txl.token_logprobs(x, t), lambda: txl.token_logprobs_bwd(x, t, f, dlogprob=f)):
        with pytest.raises(txl.TxlError) as e:
            call()
        assert e.value.code == -2


def test_linear_logprobs_rejects_bad_arguments(lib):
    need = lib.txl_linear_logprobs_workspace_bytes(100, 64, 500)
    assert need > 0

    def call(x=addr(0), w=addr(1), b=addr(2), t=addr(3), rows=100, K=64, V=500, lp=addr(4), lse=addr(5), ent=addr(6),
             ws=addr(7), ws_bytes=need):
        return lib.txl_linear_logprobs(x, w, b, t, rows, K, V, lp, lse, ent, ws, ws_bytes, None)
    for name in ("x", "w", "t", "lp", "lse", "ent"):
        assert call(**{name: None}) == -1, name
    for name in ("x", "w"):
        assert call(**{name: addr(8) + 8}) == -3, name
    for name in ("b", "t", "lp", "lse", "ent"):
        assert call(**{name: addr(8) + 1}) == -3, name
    assert call(rows=-1) == -1 and call(K=0) == -1 and call(V=0) == -1
    assert call(K=60) == -2 and call(K=(1 << 20) + 8) == -2 and call(V=(1 << 24) + 1) == -2
    assert call(rows=(1 << 28) + 1) == -2 and call(rows=1 << 27, V=1 << 14) == -2
    assert call(ws=None) == -7 and call(ws=addr(7) + 128) == -7 and call(ws_bytes=need - 1) == -7
    assert call(lp=addr(5)) == -4 and call(lse=addr(1) + 64) == -4 and call(ws=addr(0)) == -4 and call(ent=addr(7) + 16) == -4
    assert call(rows=0, x=None, w=None, t=None, ws=None) == 0
    for rows, K, V in ((0, 64, 500), (-1, 64, 500), (100, 60, 500), (100, 64, 0)):
        assert lib.txl_linear_logprobs_workspace_bytes(rows, K, V) == 0


def test_linear_binding_refuses_what_it_can_see():
    x, w, t = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(9, 8, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        txl.linear_logprobs(x, w, t)
    with pytest.raises(ValueError, match="w must be"):
        txl.linear_logprobs(x, w[0], t)
    with pytest.raises(ValueError, match="last axis"):
        txl.linear_logprobs(x[:, :0], w, t)
    assert txl.linear_logprobs_workspace_bytes(2 ** 31, 64, 64, device=0) == 0
