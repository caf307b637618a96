"""Products of 17 and more tokens through as many outputs as a model's matrices have
(the kernels that take 32 and 64 tokens a workgroup), and at alignments and scales at
the edge of what is accepted, against 64 bits."""
import pytest
from test_gpu_matvec import E1M2, E2M1, E2M1C, INT4, MX32, NV16, env, expected, rows, weights  # noqa: F401
import serve_reference as ref

pytestmark = pytest.mark.gpu


def check(env, cfg, q, T, N, K, xk, yk):
    torch, F = env
    kinds = {"bf16": torch.bfloat16, "f32": torch.float32}
    x = rows(torch, T, K + 7, kinds[xk])[:, 3:3 + K]
    full = torch.full((T, N + 5), -7.0, dtype=kinds[yk], device="cuda")
    y = full[:, 1:1 + N]
    F.ufp4_matvec(cfg, x, q, y, F.MatvecWorkspace(T, N, K, cfg))
    want, bound = expected(env, cfg, x, q, kinds[yk])
    err = (y.double() - want).abs()
    print(float((err / bound).max()), flush=True)
    assert bool((err <= bound).all())
    assert bool((full[:, 0] == -7.0).all()) and bool((full[:, 1 + N:] == -7.0).all())


# 32 tokens a workgroup: 257 tiles of rows (N 4099) and 17 to 32 tokens, 130 tiles and 33
# to 64; 64 tokens: 257 tiles and more than 32.  One, two and three parts of x'.
SIZES = [(17, 4099, 1056), (32, 4096, 4096), (41, 2080, 2080), (40, 4099, 1088), (64, 4112, 4128), (130, 4099, 1056), (61, 14336, 512)]
FORMATS = [(NV16, 1, "bf16", "bf16"), (NV16, 1, "f32", "f32"), (MX32, 0, "bf16", "f32"), (MX32, 1, "f32", "bf16")]


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("scaling,rht,xk,yk", FORMATS)
def test_values(env, T, N, K, scaling, rht, xk, yk):
    torch, F = env
    cfg = F.config(grid=(E1M2, INT4, E2M1, E2M1C)[(T + N) % 4], scaling=scaling, rht=rht, rht_seed=5)
    check(env, cfg, weights(env, N, K, cfg), T, N, K, xk, yk)


@pytest.mark.parametrize("T,N,K", [(1, 37, 64), (3, 300, 544), (16, 100, 1024), (20, 50, 448), (64, 4099, 1024)])
@pytest.mark.parametrize("scaling,offset", [(NV16, 2), (NV16, 6), (MX32, 1), (MX32, 2), (MX32, 3)])
def test_scales_at_any_alignment(env, T, N, K, scaling, offset):
    torch, F = env
    cfg = F.config(scaling=scaling, rht=1, rht_seed=5)
    q = weights(env, N, K, cfg)
    shape = q.scales.shape
    buf = torch.full((q.scales.numel() + 32,), 0x7F if scaling == NV16 else 0xFF, dtype=torch.uint8, device="cuda")
    at = buf[offset:offset + q.scales.numel()].view(shape)
    at.copy_(q.scales)
    assert at.data_ptr() % 16 == offset
    check(env, cfg, F.QTensor(q.codes, at, q.tensor_scale), T, N, K, "bf16", "f32")


@pytest.mark.parametrize("T", [1, 20])
@pytest.mark.parametrize("grid", [E1M2, INT4, E2M1])
def test_smallest_power_of_two_scales(env, T, grid):
    """MX32 scales 2^-127 and 2^-126 (bytes 0 and 1): the weights from 2^-126 on count, exactly."""
    torch, F = env
    N, K = 33, 256
    g = torch.Generator(device="cuda").manual_seed(T)
    cfg = F.config(grid=grid, scaling=MX32, rht=0)
    q = F.alloc_layout(N, K, MX32)
    q.scales.copy_(torch.randint(0, 2, q.scales.shape, device="cuda", generator=g))
    n = torch.randint(0, 16, (N, K), device="cuda", generator=g, dtype=torch.uint8)
    for pack in (True, False):
        q.codes.copy_(n[:, 0::2] | (n[:, 1::2] << 4))
        w = ref.values(q.codes, q.scales, grid, True)
        n = torch.where((w.abs() < 2.0 ** -126) | (n == 8), 0, n)  # (8 is no code of INT4)
    x = torch.randint(-8, 9, (T, K), device="cuda", generator=g).to(torch.bfloat16) * 2.0 ** 100
    y = torch.empty(T, N, device="cuda")
    F.ufp4_matvec(cfg, x, q, y, F.MatvecWorkspace(T, N, K, cfg))
    assert bool((w != 0).any())
    assert torch.equal(y.double(), x.double() @ w.T)
