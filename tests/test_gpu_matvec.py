"""Products of a few rows with 4-bit weights against 64 bits."""
import pytest
import serve_reference as ref

pytestmark = pytest.mark.gpu

E1M2, INT4, E2M1, E2M1C = range(4)
NV16, MX32 = 0, 1


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp4_quantization_amd as F
    return torch, F


def weights(env, N, K, cfg, seed=1, spread=0.02):
    torch, F = env
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn(N, K, device="cuda", generator=g) * spread).bfloat16()
    q = F.alloc_layout(N, K, cfg.scaling)
    if N and K:
        F.ufp4_quantize(w, cfg, q, F.Workspace(N, K))
    return q


def rows(torch, T, K, kind, seed=2, outliers=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, K, device="cuda", generator=g) + torch.randn(K, device="cuda", generator=g) * 0.7
    if outliers and K:
        x[:, :: max(1, K // 3)] *= 50.0
    return x.to(kind)


def expected(env, cfg, x, q, y_kind):
    """y in float64 and the bound of its error.  With ax >= |x'| (the block's sum of
    magnitudes / 4 under the transform), every product is off by at most
      ux, x's own rounding: one fp16 part 2^-11, two 2^-22, bf16 cut from the front
        three times 2^-23, or 0 where x is exact;
      2^-22 of the transform's four roundings;
    and every of K fp32 additions by 2^-23 of the sum of magnitudes.  fp16 parts
    under the token's power of two also lose up to 2^-25, that is 2^-25 / 2^12 of
    the token's largest magnitude."""
    torch, F = env
    mx = cfg.scaling == MX32
    K = x.shape[1]
    w = ref.values(q.codes, q.scales, cfg.grid, mx) * (1.0 if mx else q.tensor_scale.double()[0])
    xd = x.double()
    ax = ref.block_sums(xd) / 4 if cfg.rht else xd.abs()
    if cfg.rht:
        xd = ref.along(xd, ref.hadamard(F.ufp4_rht_signs(cfg.rht_seed)))
    exact = not cfg.rht and x.dtype == torch.bfloat16
    two = y_kind == torch.float32
    ux = 0.0 if exact else 2.0 ** -23 if mx else 2.0 ** -22 if two else 2.0 ** -11
    y = xd @ w.T
    bound = (ux + (2.0 ** -22 if cfg.rht else 0.0) + (K + 8) * 2.0 ** -23) * (ax @ w.abs().T)
    if not mx and K:
        bound += 2.0 ** -37 * x.double().abs().amax(1, keepdim=True) * w.abs().sum(1)
    half = torch.finfo(y_kind).eps / 2
    return y, bound * (1 + half) + half * y.abs() + 1e-44


CASES = [
    (1, 16, 64, E1M2, NV16, 1, "bf16", "bf16"), (1, 1, 32, E1M2, NV16, 1, "bf16", "f32"),
    (1, 257, 4096, E1M2, NV16, 1, "bf16", "bf16"), (1, 4096, 128, INT4, NV16, 1, "f32", "f32"),
    (2, 33, 160, E2M1, NV16, 0, "bf16", "f32"), (3, 100, 992, E2M1C, NV16, 1, "f32", "bf16"),
    (4, 64, 2048, INT4, NV16, 0, "f32", "f32"), (4, 31, 16384, E1M2, NV16, 1, "f32", "f32"),
    (5, 48, 96, E1M2, NV16, 1, "bf16", "f32"), (16, 300, 1056, E2M1, NV16, 0, "bf16", "bf16"),
    (17, 77, 544, INT4, NV16, 1, "bf16", "f32"), (37, 130, 2080, E1M2, NV16, 1, "f32", "f32"),
    (64, 50, 320, E2M1, NV16, 1, "bf16", "f32"), (65, 40, 256, E1M2, NV16, 0, "bf16", "f32"),
    (200, 35, 288, INT4, NV16, 1, "f32", "bf16"), (1, 20000, 64, E1M2, NV16, 1, "bf16", "f32"),
    (1, 40, 256, E1M2, MX32, 1, "bf16", "f32"), (1, 64, 4096, E2M1, MX32, 0, "bf16", "bf16"),
    (3, 65, 96, INT4, MX32, 0, "bf16", "f32"), (7, 129, 1056, E2M1, MX32, 1, "f32", "f32"),
    (33, 47, 2080, INT4, MX32, 1, "f32", "f32"), (70, 30, 160, E2M1C, MX32, 1, "bf16", "bf16"),
    (2, 16, 32768, E1M2, MX32, 0, "f32", "f32"), (4, 20, 11264, E1M2, NV16, 1, "bf16", "bf16"), (4, 19, 65536, E2M1, NV16, 1, "bf16", "f32"),
]


@pytest.mark.parametrize("T,N,K,grid,scaling,rht,xk,yk", CASES)
def test_values(env, T, N, K, grid, scaling, rht, xk, yk):
    torch, F = env
    kinds = {"bf16": torch.bfloat16, "f32": torch.float32}
    cfg = F.config(grid=grid, scaling=scaling, rht=rht, rht_seed=77)
    q = weights(env, N, K, cfg)
    # rows inside wider buffers, at addresses that are no multiple of a vector
    x = rows(torch, T, K + 7, kinds[xk])[:, 3:3 + K]
    full = torch.full((T, N + 5), -7.0, dtype=kinds[yk], device="cuda")
    y = full[:, 1:1 + N]
    F.ufp4_matvec(cfg, x, q, y, F.MatvecWorkspace(T, N, K, cfg))
    want, bound = expected(env, cfg, x, q, kinds[yk])
    err = (y.double() - want).abs()
    print(float((err / bound).max()), flush=True)
    assert bool((err <= bound).all())
    assert bool((full[:, 0] == -7.0).all()) and bool((full[:, 1 + N:] == -7.0).all())


@pytest.mark.parametrize("T", [1, 3, 16, 50])
@pytest.mark.parametrize("scaling", [NV16, MX32])
@pytest.mark.parametrize("grid", [E1M2, INT4, E2M1])
@pytest.mark.parametrize("rht", [0, 1])
def test_whole_numbers(env, T, scaling, grid, rht):
    """Small whole x, block scales that are powers of two, tensor scale 1: every
    product and sum is exact in fp32, so y has no error at all."""
    torch, F = env
    N, K = 53, 480
    g = torch.Generator(device="cuda").manual_seed(T)
    cfg = F.config(grid=grid, scaling=scaling, rht=rht, rht_seed=5)
    q = F.alloc_layout(N, K, scaling)
    codes = torch.randint(0, 256, (N, K // 2), device="cuda", generator=g, dtype=torch.uint8)
    if grid == INT4:  # the nibble 8 is no code
        codes = torch.where((codes & 15) == 8, codes ^ 8, codes)
        codes = torch.where((codes >> 4) == 8, codes ^ 128, codes)
    q.codes.copy_(codes)
    e = torch.randint(-2, 3, q.scales.shape, device="cuda", generator=g)
    q.scales.copy_(127 + e if scaling == MX32 else (7 + e) << 3)
    q.tensor_scale.fill_(1.0)
    x = torch.randint(-8, 9, (T, K), device="cuda", generator=g).to(torch.bfloat16)
    x[:, ::37] = 0
    y = torch.empty(T, N, device="cuda")
    F.ufp4_matvec(cfg, x, q, y, F.MatvecWorkspace(T, N, K, cfg))
    xd = x.double()
    if rht:
        xd = ref.along(xd, ref.hadamard(F.ufp4_rht_signs(5)))
    assert torch.equal(y.double(), xd @ ref.values(q.codes, q.scales, grid, scaling == MX32).T)


def test_empty(env):
    torch, F = env
    cfg = F.config()
    y = torch.full((20, 16), -7.0, device="cuda")
    for T in (1, 20):  # K of 0: zeros
        q = F.QTensor(*(torch.empty(s, dtype=torch.uint8, device="cuda") for s in ((16, 0), (16, 0))), torch.ones(1, device="cuda"))
        F.ufp4_matvec(cfg, torch.empty(T, 0, device="cuda"), q, y[:T], F.MatvecWorkspace(T, 16, 0, cfg))
        assert bool((y[:T] == 0).all())
    q = weights(env, 16, 64, cfg)
    F.ufp4_matvec(cfg, torch.empty(0, 64, device="cuda"), q, y[:0])


@pytest.mark.parametrize("T", [1, 4, 9, 40])
@pytest.mark.parametrize("scaling", [NV16, MX32])
@pytest.mark.parametrize("rht", [0, 1])
def test_a_lost_token_stays_alone(env, T, scaling, rht):
    """NaN or infinity in one token of x: NaN or infinities in its row, the other rows
    bit for bit what they were."""
    torch, F = env
    N, K = 40, 544
    cfg = F.config(scaling=scaling, rht=rht, rht_seed=3)
    q, x = weights(env, N, K, cfg), rows(torch, T, K, torch.bfloat16)
    ws = F.MatvecWorkspace(T, N, K, cfg)
    outs = []
    for bad in (None, float("nan"), float("inf")):
        z = x.clone()
        if bad is not None:
            z[T // 2, 7] = bad
        y = torch.empty(T, N, device="cuda")
        F.ufp4_matvec(cfg, z, q, y, ws)
        outs.append(y)
    for y in outs[1:]:
        assert not bool(torch.isfinite(y[T // 2]).any())
        y[T // 2] = outs[0][T // 2]
        assert torch.equal(y, outs[0])


@pytest.mark.parametrize("size", [1e-38, 1e-20, 1e20, 3e38])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_tokens_of_all_sizes(env, size, kind):
    """One token's magnitude does not matter to its relative error (a token near the
    largest number: without the transform, whose fp32 sums may pass it)."""
    torch, F = env
    N, K = 30, 96
    rht = int(size < 1e38)
    cfg = F.config(rht=rht, rht_seed=3)
    q = weights(env, N, K, cfg, spread=0.01)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (torch.rand(2, K, device="cuda", generator=g) * 2 - 1) * size
    x = x.to(torch.bfloat16) if kind == "bf16" else x
    y = torch.empty(2, N, device="cuda")
    F.ufp4_matvec(cfg, x, q, y)
    want, bound = expected(env, cfg, x, q, torch.float32)
    assert bool(((y.double() - want).abs() <= bound).all())


def test_past_32_bits(env):
    """Weights of more than 4 GiB of codes: rows at the end."""
    torch, F = env
    N, K = (1 << 19) + 37, 16640  # 4.06 GiB
    cfg = F.config(rht=0)
    q = F.alloc_layout(N, K, NV16)
    q.codes.fill_(0)
    q.scales.fill_(0x38)
    q.tensor_scale.fill_(1.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    q.codes[-50:] = torch.randint(0, 256, (50, K // 2), device="cuda", generator=g, dtype=torch.uint8)
    x = torch.randint(-2, 3, (2, K), device="cuda", generator=g).bfloat16()
    y = torch.full((2, N), -7.0, device="cuda")
    F.ufp4_matvec(cfg, x, q, y, F.MatvecWorkspace(2, N, K, cfg))
    assert bool((y[:, :-50] == 0).all())
    assert torch.equal(y[:, -50:].double(), x.double() @ ref.values(q.codes[-50:], q.scales[-50:], E1M2).T)
