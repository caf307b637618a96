"""Products over no values of K: zeros, whatever the tokens, types and formats."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 5, 16, 20, 64])
@pytest.mark.parametrize("scaling", [0, 1])
@pytest.mark.parametrize("rht", [0, 1])
@pytest.mark.parametrize("kinds", ["bf16 bf16", "bf16 f32", "f32 bf16"])
def test_no_values(T, scaling, rht, kinds):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp4_quantization_amd as F
    x, y = ({"bf16": torch.bfloat16, "f32": torch.float32}[k] for k in kinds.split())
    for N in (16, 70):
        cfg = F.config(scaling=scaling, rht=rht)
        q = F.QTensor(*(torch.empty(N, 0, dtype=torch.uint8, device="cuda") for _ in range(2)), torch.ones(1, device="cuda"))
        full = torch.full((T, N + 3), -7.0, dtype=y, device="cuda")
        F.ufp4_matvec(cfg, torch.empty(T, 0, dtype=x, device="cuda"), q, full[:, 1:1 + N], F.MatvecWorkspace(T, N, 0, cfg))
        assert bool((full[:, 1:1 + N] == 0).all())
        assert bool((full[:, 0] == -7.0).all()) and bool((full[:, 1 + N:] == -7.0).all())
