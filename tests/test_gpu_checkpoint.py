"""8-bit checkpoints and the gated activation that uses them, against plain
implementations in 64 bits."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

INT8, E4M3 = 0, 1
SILU, GELU = 0, 1


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp4_quantization_amd as F
    return torch, F


def f64_to_bf16_up(v):
    """Smallest bf16 >= v (v > 0, in bf16's normal range), as float64."""
    m, e = np.frexp(v)
    return np.ldexp(np.ceil(m * 256), e - 8)


def plain_save(x, fmt):
    """(scales, kept values) in float64 of a float64 matrix of bf16 values."""
    rows, cols = x.shape
    nb = -(-cols // 32)
    b = np.zeros((rows, nb * 32))
    b[:, :cols] = x
    b = b.reshape(rows, nb, 32)
    Q = 127.0 if fmt == INT8 else 448.0
    with np.errstate(all="ignore"):
        amax = np.abs(b).max(2)
        s = np.maximum(f64_to_bf16_up(np.where(np.isfinite(amax), amax, 1.0) / Q), 2.0 ** -100)
        s = np.where(np.isfinite(amax), s, np.nan)
        q = b / s[..., None]
        if fmt == INT8:
            q = np.rint(q)
        else:
            p = np.ldexp(1.0, np.maximum(np.frexp(q)[1] - 1, -6) - 3)
            q = np.rint(q / p) * p
        v = q * s[..., None]
    return s, v.reshape(rows, nb * 32)[:, :cols]


def bf16(torch, a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


def save_load(env, x, fmt):
    torch, F = env
    c = F.alloc_checkpoint(*x.shape, fmt)
    F.ufp4_checkpoint_save(x, c)
    out = torch.empty(x.shape, dtype=torch.float32, device="cuda")
    F.ufp4_checkpoint_load(c, out)
    return c, out


def same(got, want):
    got, want = got.double().cpu().numpy(), np.asarray(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    # codes times scales are exact in fp32
    assert np.array_equal(got[ok], want[ok])


@pytest.mark.parametrize("fmt", [INT8, E4M3])
def test_every_quotient(env, fmt):
    """Every significand of the block's maximum against every significand of
    a value at every exponent below it that can matter: all ties included."""
    torch, F = env
    sig = 1.0 + np.arange(128) / 128.0
    vals = np.concatenate([np.ldexp(sig, -e) for e in range(0, 20)])
    vals = np.concatenate([vals, -vals])
    rows = []
    for m in sig:
        v = vals[np.abs(vals) <= m]
        v = np.concatenate([v, np.zeros(-v.size % 31)]).reshape(-1, 31)
        rows.append(np.concatenate([np.full((v.shape[0], 1), m), v], 1).reshape(-1))
    width = max(r.size for r in rows)
    x = np.zeros((128, -(-width // 32) * 32))
    for i, r in enumerate(rows):
        x[i, :r.size] = r
    for scale in (1.0, 2.0 ** -60, 2.0 ** 90):
        xb = bf16(torch, x * scale).cuda()
        s, want = plain_save(x * scale, fmt)
        c, out = save_load(env, xb, fmt)
        assert np.array_equal(c.scales.double().cpu().numpy(), s)
        same(out, want)


@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("cols", [1, 2, 3, 4, 5, 6, 7, 8, 31, 32, 33, 34, 36, 38, 40, 97, 1365, 4096])
def test_shapes_and_strides(env, fmt, cols):
    torch, F = env
    rng = np.random.default_rng(cols)
    rows = 19
    wide = rng.standard_normal((rows, cols + 5)) * np.exp(rng.standard_normal((rows, cols + 5)))
    xb = bf16(torch, wide).cuda()[:, 3:3 + cols]
    c, out = save_load(env, xb, fmt)
    s, want = plain_save(xb.double().cpu().numpy(), fmt)
    same(out, want)
    half = torch.full((rows, cols + 2), 9.0, dtype=torch.bfloat16, device="cuda")
    F.ufp4_checkpoint_load(c, half[:, 1:1 + cols])
    assert torch.equal(half[:, 1:1 + cols], out.to(torch.bfloat16))
    assert (half[:, 0] == 9).all() and (half[:, -1] == 9).all()


@pytest.mark.parametrize("fmt", [INT8, E4M3])
def test_edges(env, fmt):
    torch, F = env
    big = 3.3895313892515355e38
    rows = [np.zeros(64), np.r_[np.full(32, 1e-40), np.ones(32)], np.r_[np.full(32, 2.0 ** -126), np.full(32, 2.0 ** -95)],
            np.r_[1.0, np.nan, np.zeros(30), np.full(32, -2.0)], np.r_[np.full(32, 3.0), -np.inf, np.zeros(31)],
            np.r_[np.inf, np.nan, np.zeros(62)], np.r_[big / 2, -1e30, np.zeros(62)], -np.arange(64.0)]
    x = bf16(torch, np.stack(rows)).cuda()
    c, out = save_load(env, x, fmt)
    s, want = plain_save(x.double().cpu().numpy(), fmt)
    assert np.array_equal(c.scales.double().cpu().numpy(), s, equal_nan=True)
    same(out, want)


@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("cols", [24, 96, 1365])
def test_dispatch_from_the_checkpoint(env, fmt, cols):
    torch, F = env
    rng = np.random.default_rng(cols)
    T, k, E = 45, 3, 7
    x = bf16(torch, rng.standard_normal((T, cols))).cuda()
    ids = rng.integers(-1, E, size=(T, k)).astype(np.int32)
    R = F.ufp4_expert_rows(T, k, E, 16)
    off = torch.empty(E + 2, dtype=torch.int64, device="cuda")
    ros, sor = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda")
    F.ufp4_expert_sort(torch.from_numpy(ids).cuda(), E, 16, off, ros, sor)
    c, kept = save_load(env, x, fmt)
    rows = torch.full((R, cols), 4.0, dtype=torch.bfloat16, device="cuda")
    F.ufp4_expert_dispatch_checkpoint(c, ros, sor, rows)
    want = torch.where((sor >= 0)[:, None], kept.to(torch.bfloat16)[(sor.clamp(min=0) // k).long()], 0)
    assert torch.equal(rows, want)


def act64(g, act):
    """f(g) and f'(g) in float64."""
    with np.errstate(all="ignore"):
        if act == SILU:
            y, dy = g, np.ones_like(g)
        else:
            c = 2 * math.sqrt(2 / math.pi)
            t = np.clip(g, -40, 40)
            y, dy = c * (t + 0.044715 * t ** 3), c * (1 + 3 * 0.044715 * t ** 2)
        s = 1 / (1 + np.exp(-y))
        return g * s, s + (g if act == SILU else np.clip(g, -40, 40)) * s * (1 - s) * dy


def gate_input(rng, rows, width):
    a = rng.standard_normal((rows, 2 * width)) * np.where(rng.random(2 * width) < 0.05, 30.0, 1.5)
    if rows > 3:
        a[1] = 0.0
        a[2, :width] = np.linspace(-60, 60, width)
        a[3, :width] = np.where(np.arange(width) % 2, 1e30, -1e30)
    return a


def tolerance(v, size):
    """One rounding to bf16, and fp32 arithmetic (a few roundings and the
    hardware's exp and reciprocal, whose argument's rounding is scaled by up
    to about 90 in the exponential) on terms of the given size."""
    return 2.0 ** -8 * np.abs(v) + 100 * 2.0 ** -24 * size + 1e-37


@pytest.mark.parametrize("act", [SILU, GELU])
@pytest.mark.parametrize("rows,width,pad", [(1, 1, 0), (5, 8, 0), (8, 2048, 0), (9, 33, 1), (4, 2, 0), (4, 3, 0), (4, 4, 1), (4, 6, 0), (5, 39, 0), (33, 1365, 0), (6, 96, 3), (7, 250, 8)])
def test_gated(env, act, rows, width, pad):
    torch, F = env
    rng = np.random.default_rng(rows + width)
    gu = bf16(torch, np.c_[gate_input(rng, rows, width), np.ones((rows, pad))]).cuda()[:, :2 * width]
    x = gu.double().cpu().numpy()
    g, u = x[:, :width], x[:, width:]
    f, _ = act64(g, act)
    h = torch.full((rows, width + pad), 7.0, dtype=torch.bfloat16, device="cuda")[:, :width]
    F.ufp4_gated_act(gu, act, h)
    got = h.double().cpu().numpy()
    assert (np.abs(got - f * u) <= tolerance(f * u, np.abs(g * u))).all()
    for fmt in (INT8, E4M3):
        c = F.alloc_checkpoint(rows, width, fmt, halves=2)
        h2 = torch.empty((rows, width), dtype=torch.bfloat16, device="cuda")
        F.ufp4_gated_act(gu, act, h2, c)
        assert torch.equal(h2, h)
        # each half as checkpoint_save keeps it
        nb = -(-width // 32)
        for half in (0, 1):
            one = F.alloc_checkpoint(rows, width, fmt)
            F.ufp4_checkpoint_save(gu[:, half * width:(half + 1) * width], one)
            assert torch.equal(c.codes[:, half * width:(half + 1) * width], one.codes)
            assert torch.equal(c.scales[:, half * nb:(half + 1) * nb], one.scales)
        kg, ku = plain_save(g, fmt)[1], plain_save(u, fmt)[1]
        dh = bf16(torch, rng.standard_normal((rows, width + pad))).cuda()[:, :width]
        dgu = torch.full((rows, 2 * width + pad), 7.0, dtype=torch.bfloat16, device="cuda")[:, :2 * width]
        again = torch.empty((rows, width), dtype=torch.bfloat16, device="cuda")
        F.ufp4_gated_act_backward(dh, c, act, dgu, again)
        f, df = act64(kg, act)
        d = dh.double().cpu().numpy()
        out = dgu.double().cpu().numpy()
        # f' has terms up to g sigma (1 - sigma) y' beside sigma: size 1 + |g|
        # (the gate's derivative is bounded, its terms' factors are not)
        bound = np.abs(d * ku) * (1 + np.minimum(np.abs(kg), 20.0))
        assert (np.abs(out[:, :width] - d * ku * df) <= tolerance(d * ku * df, bound)).all()
        assert (np.abs(out[:, width:] - d * f) <= tolerance(d * f, np.abs(d * kg))).all()
        assert (np.abs(again.double().cpu().numpy() - f * ku) <= tolerance(f * ku, np.abs(kg * ku))).all()
        dgu2 = torch.empty((rows, 2 * width), dtype=torch.bfloat16, device="cuda")
        F.ufp4_gated_act_backward(dh, c, act, dgu2)
        assert torch.equal(dgu2, dgu)


@pytest.mark.parametrize("act", [SILU, GELU])
def test_gated_gradient_against_differences(env, act):
    """dgu against central differences of the 64-bit activation at the kept
    values."""
    torch, F = env
    rng = np.random.default_rng(2)
    rows, width = 6, 160
    gu = bf16(torch, rng.standard_normal((rows, 2 * width)) * 2).cuda()
    c = F.alloc_checkpoint(rows, width, INT8, halves=2)
    h = torch.empty((rows, width), dtype=torch.bfloat16, device="cuda")
    F.ufp4_gated_act(gu, act, h, c)
    x = gu.double().cpu().numpy()
    g, u = plain_save(x[:, :width], INT8)[1], plain_save(x[:, width:], INT8)[1]
    dh = bf16(torch, rng.standard_normal((rows, width))).cuda()
    dgu = torch.empty((rows, 2 * width), dtype=torch.bfloat16, device="cuda")
    F.ufp4_gated_act_backward(dh, c, act, dgu)
    d, e = dh.double().cpu().numpy(), 1e-4
    dg = d * u * (act64(g + e, act)[0] - act64(g - e, act)[0]) / (2 * e)
    du = d * (act64(g, act)[0] * (u + e) - act64(g, act)[0] * (u - e)) / (2 * e)
    got = dgu.double().cpu().numpy()
    # bf16's rounding; the differences' own error is e^2 f'''/6 < 1e-8
    for a, b in ((got[:, :width], dg), (got[:, width:], du)):
        assert (np.abs(a - b) <= 2.0 ** -8 * np.abs(b) + 1e-4).all()


def test_a_lost_block_reads_back_as_nan_only_itself(env):
    torch, F = env
    rng = np.random.default_rng(3)
    x = rng.standard_normal((2, 128))
    x[0, 40] = np.inf
    gu = bf16(torch, x).cuda()
    c = F.alloc_checkpoint(2, 64, E4M3, halves=2)
    h = torch.empty((2, 64), dtype=torch.bfloat16, device="cuda")
    F.ufp4_gated_act(gu, SILU, h, c)
    dh = torch.ones((2, 64), dtype=torch.bfloat16, device="cuda")
    dgu = torch.empty((2, 128), dtype=torch.bfloat16, device="cuda")
    F.ufp4_gated_act_backward(dh, c, SILU, dgu)
    bad = torch.isnan(dgu).cpu().numpy()
    want = np.zeros((2, 128), bool)
    want[0, 32:64] = want[0, 96:128] = True
    assert np.array_equal(bad, want)


def test_refusals(env):
    torch, F = env
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    c = F.alloc_checkpoint(4, 64, INT8)
    with pytest.raises(ValueError):
        F.ufp4_checkpoint_save(x[:3], c)
    with pytest.raises(TypeError):
        F.ufp4_checkpoint_save(x.float(), c)
    with pytest.raises(F.Ufp4Error):
        F.ufp4_checkpoint_save(x, F.alloc_checkpoint(4, 64, 2))
    with pytest.raises(ValueError):
        F.ufp4_gated_act(x, SILU, torch.zeros((4, 32), dtype=torch.bfloat16, device="cuda"), c)
    with pytest.raises(F.Ufp4Error):
        F.ufp4_gated_act(x, 2, torch.zeros((4, 32), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        F.Checkpoint(c.codes, c.scales[:, :1], INT8)


@pytest.mark.parametrize("act,fmt", [(SILU, INT8), (GELU, E4M3)])
def test_large_calls_equal_their_parts(env, act, fmt):
    """Calls that move more than the last-level cache holds take other loads
    and stores."""
    torch, F = env
    rows, width = 17011, 2003
    assert rows * width * 8 > 256 << 20
    g = torch.Generator(device="cuda").manual_seed(5)
    gu = torch.randn(rows, 2 * width, device="cuda", generator=g).to(torch.bfloat16)
    dh = torch.randn(rows, width, device="cuda", generator=g).to(torch.bfloat16)
    c = F.alloc_checkpoint(rows, width, fmt, halves=2)
    new = lambda r, w: torch.empty((r, w), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    h, again, dgu = new(rows, width), new(rows, width), new(rows, 2 * width)
    F.ufp4_gated_act(gu, act, h, c)
    F.ufp4_gated_act_backward(dh, c, act, dgu, again)
    for r in range(0, rows, 3000):
        n = min(3000, rows - r)
        pc = F.alloc_checkpoint(n, width, fmt, halves=2)
        ph, pa, pd = new(n, width), new(n, width), new(n, 2 * width)
        F.ufp4_gated_act(gu[r:r + n], act, ph, pc)
        F.ufp4_gated_act_backward(dh[r:r + n], pc, act, pd, pa)
        assert torch.equal(ph, h[r:r + n]) and torch.equal(pa, again[r:r + n]) and torch.equal(pd, dgu[r:r + n])
        assert torch.equal(pc.codes, c.codes[r:r + n]) and torch.equal(pc.scales, c.scales[r:r + n])
