"""A lost block of the gated activation's checkpoint (its scale is NaN) shows
in every gradient that depends on it, and in no other."""
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


@pytest.mark.parametrize("act", [SILU, GELU])
@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("half", [0, 1])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_lost_block(env, act, fmt, half, bad):
    torch, F = env
    rng = np.random.default_rng(8 * act + 4 * fmt + half)
    rows, width = 3, 72
    x = rng.standard_normal((rows, 2 * width)).astype(np.float32)
    x[1, half * width + 40] = bad
    gu = torch.from_numpy(x).to(torch.bfloat16).cuda()
    c = F.alloc_checkpoint(rows, width, fmt, halves=2)
    new = lambda cols: torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    h, again, dgu = new(width), new(width), new(2 * width)
    F.ufp4_gated_act(gu, act, h, c)
    F.ufp4_gated_act_backward(torch.ones_like(h), c, act, dgu, again)
    lost = np.zeros((rows, width), bool)
    lost[1, 32:64] = True
    # dg = dh u f'(g) and h = f(g) u depend on both halves, du = dh f(g) on the gate
    got = torch.isnan(dgu).cpu().numpy()
    assert np.array_equal(got[:, :width], lost)
    assert np.array_equal(got[:, width:], lost if half == 0 else np.zeros_like(lost))
    assert np.array_equal(torch.isnan(again).cpu().numpy(), lost)
