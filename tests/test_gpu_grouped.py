"""Grouped products of quantized operands against 64-bit products of the
oracle's dequantized values, segment by segment."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

E1M2, INT4, E2M1, E2M1C = 0, 1, 2, 3


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp4_quantization_amd as F
    import oracle
    oracle.lib()
    return torch, F, oracle


def magnitudes(grid):
    return {E1M2: [0, .5, 1, 1.5, 2, 2.5, 3, 3.5], INT4: [0, 1, 2, 3, 4, 5, 6, 7], E2M1: [0, .5, 1, 1.5, 2, 3, 4, 6],
            E2M1C: [0, .5, 1, 1.5, 2, 0, 0, 0]}[grid]


def values(codes, scales, grid):
    """float64 values of a quantized matrix, without its tensor scale."""
    m = magnitudes(grid)
    table = np.array(m + [-v for v in m]) if grid != INT4 else np.array([0, 1, 2, 3, 4, 5, 6, 7, 0, -7, -6, -5, -4, -3, -2, -1.0])
    n = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], 2 * codes.shape[1])
    e, f = (scales >> 3).astype(int), (scales & 7).astype(float)
    d = np.where(e > 0, np.ldexp(1 + f / 8, e - 7), np.ldexp(f, -9))
    return table[n] * np.repeat(d, 16, axis=1)


def operand(rng, lines, length, grid):
    """Random codes and block scales: every code the quantizer writes, scales
    of every size including zero and the largest."""
    top = 5 if grid == E2M1C else 8
    mag = rng.integers(0, top, size=(lines, length))
    neg = rng.integers(0, 2, size=(lines, length)) * (mag > 0)
    code = np.where(neg, (16 - mag) & 15, mag) if grid == INT4 else mag + 8 * neg
    code = code.astype(np.uint8)
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)
    scales = rng.integers(0x20, 0x50, size=(lines, length // 16)).astype(np.uint8)
    odd = rng.random(scales.shape)
    scales[odd < 0.03] = 0
    scales[odd > 0.97] = 0x7E
    scales[(odd > 0.5) & (odd < 0.53)] = rng.integers(1, 8)
    return codes, scales


def dev(torch, F, codes, scales, ts):
    # (an empty array still needs memory behind it for the pointer checks)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    return F.QTensor(to(codes), to(scales), to(ts.astype(np.float32)))


def close(got, want, size, K, bf16):
    # fp32 sums of K exact products, two tensor scales applied with two
    # roundings, the output's own rounding
    tol = (K + 4) * 2.0 ** -24 * size + (2.0 ** -8 if bf16 else 0.0) * np.abs(want) + 1e-37
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), float(np.max(np.abs(got - want) / tol))


def run_nt(env, counts, N, K, grid, layout, bf16, seed, spare=0, ldc_pad=0):
    torch, F, _ = env
    rng = np.random.default_rng(seed)
    E, R = len(counts), int(sum(counts)) + spare
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    a = operand(rng, R, K, grid)
    b = operand(rng, E * N, K, grid) if layout == 0 else operand(rng, N, E * K, grid)
    ta, tb = rng.uniform(0.5, 2, E), rng.uniform(0.01, 0.1, E)
    ta, tb = ta.astype(np.float32).astype(float), tb.astype(np.float32).astype(float)
    c = torch.full((R, N + ldc_pad), 3.0, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    F.ufp4_gemm_grouped_nt(F.config(grid=grid), dev(torch, F, *a, ta), dev(torch, F, *b, tb), layout,
                           torch.from_numpy(off).cuda(), K, c[:, :N])
    got = c.double().cpu().numpy()
    assert (got[:, N:] == 3.0).all()
    av, bv = values(*a, grid), values(*b, grid)
    for e in range(E):
        x = av[off[e]:off[e + 1]]
        w = bv[e * N:(e + 1) * N] if layout == 0 else bv[:, e * K:(e + 1) * K]
        close(got[off[e]:off[e + 1], :N], x @ w.T * (ta[e] * tb[e]), np.abs(x) @ np.abs(w).T * (ta[e] * tb[e]), K, bf16)
    assert (got[off[-1]:, :N] == 0).all()


COUNTS = {"one row": [1], "one each": [1, 1, 1, 1, 1], "empty ones": [0, 3, 0, 0, 17, 0], "all empty": [0, 0],
          "around the tile": [255, 256, 257, 1, 511], "around 16": [15, 16, 17, 31, 32, 33], "small": [5, 0, 2, 9],
          "many": [int(c) for c in np.random.default_rng(0).integers(0, 7, 150)]}


@pytest.mark.parametrize("counts", COUNTS.values(), ids=COUNTS.keys())
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("N,K", [(48, 64), (1000, 96), (129, 32), (256, 352)])
def test_nt(env, counts, layout, N, K):
    run_nt(env, counts, N, K, E1M2, layout, bool(N & 1), 7 * N + K + layout, spare=3)


@pytest.mark.parametrize("grid", [E1M2, INT4, E2M1, E2M1C])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("counts", [[3, 0, 40], [300, 20, 700]], ids=["few", "more"])
def test_nt_grids_and_types(env, grid, layout, bf16, counts):
    run_nt(env, counts, 272, 160, grid, layout, bf16, grid, ldc_pad=5)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("K", [1024, 2080, 4096])
def test_nt_long_reduction(env, layout, K):
    run_nt(env, [70, 1, 0, 33], 200, K, INT4, layout, False, K)


@pytest.mark.parametrize("N", [1, 2, 15, 17, 63, 65])
def test_nt_narrow(env, N):
    run_nt(env, [3, 300], N, 96, E2M1, 0, True, N)


@pytest.mark.parametrize("counts", [[1500, 0, 255, 257, 3200, 1, 700], [5900, 0], [40, 256, 512, 4700, 300]],
                         ids=["ragged", "one segment", "whole tiles"])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("N,K,grid", [(1030, 160, E1M2), (1024, 128, INT4), (1023, 32, E2M1), (1280, 640, E1M2)])
def test_nt_many_rows(env, counts, layout, N, K, grid):
    run_nt(env, counts, N, K, grid, layout, N % 2 == 0, N + K + layout, spare=5, ldc_pad=3)


def test_nt_no_reduction_and_no_rows(env):
    run_nt(env, [3, 4], 20, 0, E1M2, 0, False, 1)
    run_nt(env, [0, 0], 20, 32, E1M2, 0, False, 1)


def test_nt_takes_the_sorted_offsets(env):
    """ufp4_expert_sort's array has one more entry: the padding rows behind the
    last expert get zeros."""
    torch, F, _ = env
    rng = np.random.default_rng(4)
    E, N, K, R = 3, 40, 64, 96
    a, b = operand(rng, R, K, E1M2), operand(rng, E * N, K, E1M2)
    off = torch.tensor([0, 16, 16, 48, R], dtype=torch.int64, device="cuda")
    one = np.ones(E + 1, np.float32)
    c = torch.full((R, N), 3.0, device="cuda")
    F.ufp4_gemm_grouped_nt(F.config(), dev(torch, F, *a, one), dev(torch, F, *b, one), 0, off, K, c, num_groups=E)
    av, bv = values(*a, E1M2), values(*b, E1M2)
    got = c.double().cpu().numpy()
    for e, (lo, hi) in enumerate([(0, 16), (16, 16), (16, 48)]):
        w = bv[e * N:(e + 1) * N]
        close(got[lo:hi], av[lo:hi] @ w.T, np.abs(av[lo:hi]) @ np.abs(w).T, K, False)
    assert (got[48:] == 0).all()


def run_dw(env, counts, M, N, grid, bf16, seed, spare=0):
    torch, F, _ = env
    rng = np.random.default_rng(seed)
    E = len(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    cols = F.ufp4_grouped_col_offsets(off, 16)
    P = int(cols[-1]) + spare
    a, b = operand(rng, M, P, grid), operand(rng, N, P, grid)
    ta, tb = rng.uniform(0.5, 2, E).astype(np.float32).astype(float), rng.uniform(0.01, 0.1, E).astype(np.float32).astype(float)
    c = torch.full((E, M, N), 3.0, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    F.ufp4_gemm_grouped_dw(F.config(grid=grid), dev(torch, F, *a, ta), dev(torch, F, *b, tb), torch.from_numpy(off).cuda(), c)
    got = c.double().cpu().numpy()
    av, bv = values(*a, grid), values(*b, grid)
    for e in range(E):
        x, w = av[:, cols[e]:cols[e + 1]], bv[:, cols[e]:cols[e + 1]]
        t = ta[e] * tb[e]
        close(got[e], x @ w.T * t, np.abs(x) @ np.abs(w).T * t, x.shape[1], bf16)


@pytest.mark.parametrize("counts", COUNTS.values(), ids=COUNTS.keys())
@pytest.mark.parametrize("M,N", [(48, 64), (257, 130), (16, 1), (300, 513)])
def test_dw(env, counts, M, N):
    run_dw(env, counts[:40], M, N, E1M2, bool(N & 1), M + N, spare=16)


@pytest.mark.parametrize("grid", [E1M2, INT4, E2M1, E2M1C])
@pytest.mark.parametrize("bf16", [False, True])
def test_dw_grids_and_types(env, grid, bf16):
    run_dw(env, [100, 0, 1000, 7], 264, 272, grid, bf16, grid)


@pytest.mark.parametrize("counts", [[16], [16, 16], [48], [1, 40, 70, 100, 140, 10, 250, 16], [176, 16, 16, 48]],
                         ids=["one block", "two of one", "three blocks", "odd blocks", "ends in one block"])
@pytest.mark.parametrize("M,N", [(1, 1), (257, 1), (3, 514), (256, 257)])
@pytest.mark.parametrize("grid", [E1M2, INT4])
def test_dw_ranges_that_end_anywhere(env, counts, M, N, grid):
    """No block behind a segment's last one, and none before its first one,
    reaches its sums, whatever its scale is: a segment's neighbours get NaN
    scales."""
    torch, F, _ = env
    run_dw(env, counts, M, N, grid, False, M + 7 * N + len(counts))
    rng = np.random.default_rng(M + N)
    E = len(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    cols = F.ufp4_grouped_col_offsets(off, 16)
    a, b = operand(rng, M, int(cols[-1]), grid), operand(rng, N, int(cols[-1]), grid)
    one, offsets = np.ones(E, np.float32), torch.from_numpy(off).cuda()
    av, bv = values(*a, grid), values(*b, grid)
    c = torch.empty((E, M, N), device="cuda")
    for odd in (0, 1):
        sa, sb = a[1].copy(), b[1].copy()
        for e in range(odd, E, 2):
            sa[:, cols[e] // 16:cols[e + 1] // 16] = 0x7F
            sb[:, cols[e] // 16:cols[e + 1] // 16] = 0x7F
        F.ufp4_gemm_grouped_dw(F.config(grid=grid), dev(torch, F, a[0], sa, one), dev(torch, F, b[0], sb, one), offsets, c)
        got = c.double().cpu().numpy()
        for e in range(1 - odd, E, 2):
            x, w = av[:, cols[e]:cols[e + 1]], bv[:, cols[e]:cols[e + 1]]
            close(got[e], x @ w.T, np.abs(x) @ np.abs(w).T, x.shape[1], False)
        assert all(np.isnan(got[e]).all() for e in range(odd, E, 2))


def test_products_of_the_quantizers_own_outputs(env):
    """Forward and gradients from ufp4_quantize_grouped's layouts against the
    oracle's dequantized values."""
    torch, F, orc = env
    rng = np.random.default_rng(11)
    E, D, W = 3, 64, 48
    counts = [40, 0, 23]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    woff = (np.arange(E + 1) * W).astype(np.int64)
    R = int(off[-1])
    cols = F.ufp4_grouped_col_offsets(off, 16)
    cfg = F.config(rht=1, rht_seed=3)
    import synth
    x, dy, w = (synth.f32_to_bf16(rng.standard_normal(s).astype(np.float32)) for s in ((R, D), (R, W), (E * W, D)))

    def quant(m, o, padded):
        t = torch.from_numpy(m.view(np.int16)).cuda()
        row, col = F.alloc_layout(t.shape[0], t.shape[1], 0, E), F.alloc_layout(t.shape[1], padded, 0, E)
        ws = F.Workspace(t.shape[0], t.shape[1], E)
        F.ufp4_quantize_grouped(t, torch.from_numpy(o).cuda(), padded, cfg, row, col, ws)
        assert ws.status() == 0
        return row, col

    def vals(q, o):
        v = values(q.codes.cpu().numpy(), q.scales.cpu().numpy(), E1M2)
        return v, q.tensor_scale.double().cpu().numpy()

    xr, xc = quant(x, off, int(cols[-1]))
    dr, dc = quant(dy, off, int(cols[-1]))
    wr, wc = quant(w, woff, E * W)
    o = torch.from_numpy(off).cuda()
    y = torch.empty((R, W), device="cuda")
    F.ufp4_gemm_grouped_nt(cfg, xr, wr, 0, o, D, y)
    # K = 48 is no multiple of 32: refused, nothing written
    dx = torch.full((R, D), 2.0, device="cuda")
    with pytest.raises(F.Ufp4Error):
        F.ufp4_gemm_grouped_nt(cfg, dr, wc, 1, o, W, dx)
    assert (dx == 2).all()
    g = torch.empty((E, W, D), device="cuda")
    F.ufp4_gemm_grouped_dw(cfg, dc, xc, o, g)
    (xv, xt), (wv, wt), (dv, dt), (xcv, xct) = vals(xr, off), vals(wr, woff), vals(dc, off), vals(xc, off)
    f32 = np.asarray([synth.bf16_to_f32(m).astype(np.float64) for m in (x,)][0])
    for e in range(E):
        a, b = xv[off[e]:off[e + 1]], wv[e * W:(e + 1) * W]
        t = xt[e] * wt[e]
        close(y[off[e]:off[e + 1]].double().cpu().numpy(), a @ b.T * t, np.abs(a) @ np.abs(b).T * t, D, False)
        a, b = dv[:, cols[e]:cols[e + 1]], xcv[:, cols[e]:cols[e + 1]]
        t = dt[e] * xct[e]
        close(g[e].double().cpu().numpy(), a @ b.T * t, np.abs(a) @ np.abs(b).T * t, a.shape[1], False)
    # and near the unquantized product: two 4-bit operands, about 0.1 each
    full = f32[:40] @ synth.bf16_to_f32(w[:W]).astype(np.float64).T
    assert np.linalg.norm(y[:40].double().cpu().numpy() - full) < 0.25 * np.linalg.norm(full)


def test_wrapper_refusals(env):
    torch, F, _ = env
    q = F.alloc_layout(32, 64, 0, 2)
    w = F.alloc_layout(2 * 16, 64, 0, 2)
    off = torch.tensor([0, 16, 32], dtype=torch.int64, device="cuda")
    c = torch.zeros((32, 16), device="cuda")
    with pytest.raises(ValueError):
        F.ufp4_gemm_grouped_nt(F.config(), q, w, 0, off, 32, c)
    with pytest.raises(ValueError):
        F.ufp4_gemm_grouped_nt(F.config(), q, w, 1, off, 64, c)
    with pytest.raises(TypeError):
        F.ufp4_gemm_grouped_nt(F.config(), q, w, 0, off.int(), 64, c)
    with pytest.raises(F.Ufp4Error):
        F.ufp4_gemm_grouped_nt(F.config(scaling=F.SCALE_MX32), q, w, 0, off, 64, c)
    with pytest.raises(ValueError):
        F.ufp4_gemm_grouped_dw(F.config(), q, w, off, torch.zeros((2, 16, 16), device="cuda"))
