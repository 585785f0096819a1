"""8-bit moments follow gradients whose sizes change within a block: what random
rounding is for.

The first element of each block has a large gradient that never changes, so it holds
the block's scale; the others double their gradient after 50 of 150 steps, and their
moments move by far less than a code's step at a time (sqrt(v) by 0.1 % of the new level).

What random rounding gives.  m: rounding keeps the mean and the recursion is linear, so
the mean of m / exact is 1; a code's step is 2^-3 of the value at most, a rounding's
variance under 2^-8 of its square, and beta1 = 0.9 carries them on to 2^-8 / (1 - 0.81), a
deviation of 0.15: six of those over the root of 65280 elements are 0.0035.
v: each rounding adds its variance to the mean of root^2, never takes any off.  A root that
moves by D between codes d apart is moved on with probability D / d, with variance below
D d; added up along the way to the final root R that is at most R d <= 2^-3 R^2, with 2^-8 for
the first step: the mean of v / exact is between 1 and 1.13, and its noise under
6 * 0.25 / 255 = 0.006."""
import numpy as np
import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl
import test_gpu_adamw as plain

N, BEFORE, STEPS = 65536, 50, 150
PINNED = np.arange(N) % 256 == 0


def gradients(t):
    size = np.random.default_rng(6).uniform(0.2, 0.6, N).astype(np.float32)
    return np.where(PINNED, np.float32(4.0), size * np.float32(1.0 if t < BEFORE else 2.0)).astype(np.float32)


def exact():
    m, v = np.zeros(N), np.zeros(N)
    for t in range(STEPS):
        g = gradients(t).astype(np.float64)
        m, v = 0.9 * m + 0.1 * g, 0.999 * v + 0.001 * g * g
    return m, v


def ratios(m_codes, m_scale, v_codes, v_scale):
    """Means of m / exact and v / exact over the elements that do not hold a scale."""
    m = (m_codes.reshape(-1, 256).astype(np.float64) * m_scale[:, None]).reshape(-1)
    root = (v_codes.reshape(-1, 256).astype(np.float64) * v_scale[:, None]).reshape(-1)
    em, ev = exact()
    return float((m / em)[~PINNED].mean()), float((root * root / ev)[~PINNED].mean())


def follows(m, v):
    return abs(m - 1.0) <= 0.005 and 1.0 - 0.007 <= v <= 1.13 + 0.007


def test_rounding_to_the_nearest_code_does_not_follow(monkeypatch):
    """The same steps in numpy with the random bits fixed at one half, and at zero (down)."""
    random = (np.zeros(N, np.float32), np.zeros(N // 256, np.float32)) * 2
    for t in range(STEPS):
        random, _, _ = plain.step8(random, gradients(t), plain.step_key(9, t + 1))
    assert follows(*ratios(*random))
    for bits in (0x80008000, 0):
        monkeypatch.setattr(plain, "mix", lambda h: np.full(h.shape, bits, np.uint64))
        state = (np.zeros(N, np.float32), np.zeros(N // 256, np.float32)) * 2
        for t in range(STEPS):
            state, _, _ = plain.step8(state, gradients(t), 0)
        m, v = ratios(*state)
        assert m < 0.9 and v < 0.5 and not follows(m, v)


@pytest.mark.gpu
def test_moments_follow_a_change_within_a_block():
    p, g = [torch.zeros(N, device="cuda")], [torch.zeros(N, device="cuda")]
    opt = txl.AdamW(p, g, lr=0.0, state_bits=8, seed=9)
    for t in range(STEPS):
        if t in (0, BEFORE):
            g[0].copy_(torch.from_numpy(gradients(t)))
        opt.step()
    got = ratios(*(s.float().cpu().numpy() for s in opt.states()))
    assert follows(*got), got
