"""The gated activation where the gate closes: sigmoid(y) down to fp32's
subnormal numbers, past the argument at which exp(-y) overflows."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

SILU, GELU = 0, 1
INT8, E4M3 = 0, 1


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp4_quantization_amd as F
    return torch, F


def act64(g, act):
    """f(g), f'(g), and the size of the terms of f' / sigma."""
    y, dy = g, np.ones_like(g)
    if act == GELU:
        c = 2 * math.sqrt(2 / math.pi)
        y, dy = c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g ** 2)
    s = 1 / (1 + np.exp(-y))
    return g * s, s + g * s * (1 - s) * dy, 1 + np.abs(g * dy)


def close(got, want, unit):
    """One rounding to bf16 (2^-8, or half of its smallest subnormal), fp32
    arithmetic (the rounding of an argument of up to 152 scaled by the exponential:
    152 * 2^-24 * 4 < 2^-14.7, and a few roundings), and sigma's own
    subnormal step of 2^-149, two of them, on terms of the size `unit`."""
    tol = (2.0 ** -8 + 2.0 ** -14) * np.abs(want) + 2.0 ** -134 + 2.0 ** -148 * unit
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), float(np.max(np.abs(got - want) / tol))


@pytest.mark.parametrize("act", [SILU, GELU])
@pytest.mark.parametrize("size", [1.0, 1e3, 1e30])
def test_closing_gate(env, act, size):
    torch, F = env
    lo, hi = (-104.0, -56.0) if act == SILU else (-10.75, -8.5)
    width = 256
    g = np.linspace(lo, hi, width)
    u = size * (1 + np.arange(width) % 7) * np.where(np.arange(width) % 2, 1.0, -1.0)
    gu = torch.from_numpy(np.r_[g, u][None].astype(np.float32)).to(torch.bfloat16).cuda()
    h = torch.empty((1, width), dtype=torch.bfloat16, device="cuda")
    F.ufp4_gated_act(gu, act, h)
    x = gu.double().cpu().numpy()
    g, u = x[:, :width], x[:, width:]
    f, _, _ = act64(g, act)
    close(h.double().cpu().numpy(), f * u, np.abs(g * u))
    dh = torch.from_numpy((1 + np.arange(width) % 3)[None].astype(np.float32)).to(torch.bfloat16).cuda()
    d = dh.double().cpu().numpy()
    for fmt in (INT8, E4M3):
        c = F.alloc_checkpoint(1, width, fmt, halves=2)
        again, dgu = torch.empty_like(h), torch.empty_like(gu)
        F.ufp4_gated_act(gu, act, h, c)
        F.ufp4_gated_act_backward(dh, c, act, dgu, again)
        kept = torch.empty((1, 2 * width), device="cuda")
        F.ufp4_checkpoint_load(F.Checkpoint(c.codes, c.scales, fmt), kept)  # (width is whole blocks: one matrix)
        x = kept.double().cpu().numpy()
        g, u = x[:, :width], x[:, width:]
        f, slope, terms = act64(g, act)
        out = dgu.double().cpu().numpy()
        close(again.double().cpu().numpy(), f * u, np.abs(g * u))
        close(out[:, width:], d * f, np.abs(d * g))
        close(out[:, :width], d * u * slope, np.abs(d * u) * terms)
