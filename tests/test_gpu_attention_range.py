"""Attention where one token outweighs a long history by many orders of magnitude and
has a value near zero: what the history adds to the result is not lost."""
import pytest
import serve_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gap", [18.0, 20.0, 24.0])
@pytest.mark.parametrize("G,grid", [(1, 0), (1, 1), (20, 2)])
def test_one_token_above_a_long_history(gap, G, grid):
    """As many sequences as fill the device, so that a wave has a quarter of all tokens."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp4_quantization_amd as F
    H, D, P, L = 8, 32, 256, 131072
    B = 96 if G == 1 else 64
    g = torch.Generator(device="cuda").manual_seed(3)
    cfg = F.config(grid=grid, rht=0)
    scale = [torch.full((H,), 0.005, device="cuda") for _ in range(2)]
    c = F.alloc_cache(L // P, P, H, D, *scale)
    k = 0.2 * torch.randn(L, H, D, device="cuda", generator=g)
    v = 1.0 + 0.25 * torch.randn(L, H, D, device="cuda", generator=g)
    k[..., :16] = 0.0
    k[77, :, :16], v[77] = 1.0, 0.0
    slots = torch.arange(L, device="cuda")
    F.ufp4_cache_append(cfg, c, k.view(L, -1).bfloat16(), v.view(L, -1).bfloat16(), slots)
    del k, v
    q = 0.3 * torch.randn(B, H * G, D, device="cuda", generator=g)
    q[..., :16] = gap * D ** 0.5 / 16
    q = q.bfloat16()
    out = torch.empty(B, H * G * D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B, H * G, device="cuda")
    F.ufp4_tree_attention(cfg, c, q.view(B, -1), torch.arange(B + 1, device="cuda"),
                          torch.full((B,), L, dtype=torch.int32, device="cuda"),
                          torch.arange(L // P, dtype=torch.int32, device="cuda").repeat(B, 1), 1, out,
                          F.AttentionWorkspace(c, H * G, B, 1), lse=lse)
    kd = ref.values(*ref.cache_rows(c, slots, "k"), grid) * scale[0].double()[:, None]
    vd = ref.values(*ref.cache_rows(c, slots, "v"), grid) * scale[1].double()[:, None]
    half = torch.finfo(torch.bfloat16).eps / 2
    for b in (0, B // 2, B - 1):
        for h in range(0, H * G, 1 if G == 1 else 37):
            kh, vh, x = kd[:, h // G], vd[:, h // G], q[b, h].double()
            a = kh @ x * D ** -0.5
            assert float(a[77] - a.mean()) > gap - 2
            p = torch.softmax(a, 0)
            want = p @ vh
            # logits: products in fp32 sums of at most 2^-23 each, factors; exp2's argument in fp32
            ea = ((kh.abs() @ x.abs()) * D ** -0.5 * (D + 4) * 2.0 ** -23).max() + 2.0 ** -22 * a.abs().max()
            # weights: twice the logits' error and exp2, fp16's half step.  Sums: a wave
            # has L / 4 products of a value and, over 16 lanes' tokens, L / 16 weights of a
            # lane; rescaled at most L / 128 times each; 64 for the joins.  (fp16 keeps
            # multiples of 2^-24 of a weight times 2^15: 2^-40 of the largest weight is
            # lost of each token's.)
            ep = 2 * ea + 2.0 ** -21 + 2.0 ** -11 + (L / 4 + L / 16 + 2 * L / 128 + 64) * 2.0 ** -23
            bound = ep * (p @ vh.abs()) + 2.0 ** -40 * vh.abs().sum(0)
            err = (out[b].view(H * G, D)[h].double() - want).abs()
            bound = bound * (1 + half) + half * want.abs()
            if b == 0 and h == 0:
                print(gap, "want", float(want.mean()), "err", float(err.max()), "bound", float(bound.min()), flush=True)
            assert bool((err <= bound).all())
            assert abs(float(lse[b, h].double() - torch.logsumexp(a, 0))) <= float(ea) + (L / 16 + L / 128 + 64) * 2.0 ** -23 + 2.0 ** -18
