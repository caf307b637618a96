"""The decoding operators at the largest sizes that they accept: exact results, or bit
for bit those of small calls."""
import pytest
import serve_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp4_quantization_amd as F
    return torch, F


def whole_weights(env, N, K, g):
    """Any E1M2 codes under scales 1: every product of a whole number is a multiple of 1/2."""
    torch, F = env
    q = F.alloc_layout(N, K, 0)
    q.codes.copy_(torch.randint(0, 256, q.codes.shape, device="cuda", generator=g, dtype=torch.uint8))
    q.scales.fill_(0x38)
    q.tensor_scale.fill_(1.0)
    return q


# (sums of at most 4096 terms below 8 * 3.5: exact in fp32)
@pytest.mark.parametrize("T,N,K", [((1 << 21) - 1, 16, 32), (1, (1 << 25) - 1, 32), (5, (1 << 25) - 1, 32), (2, 3, (1 << 25) - 32),
                                   (20, 17, (1 << 25) - 32)])
def test_products(env, T, N, K):
    torch, F = env
    g = torch.Generator(device="cuda").manual_seed(1)
    cfg = F.config(rht=0)
    q = whole_weights(env, N, K, g)
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    at = torch.arange(K, device="cuda") if K <= 4096 else torch.randint(0, K, (4096,), device="cuda", generator=g).unique()
    at[-1] = K - 1
    x[:, at] = torch.randint(-8, 9, (T, at.numel()), device="cuda", generator=g).bfloat16()
    y = torch.empty(T, N, device="cuda")
    F.ufp4_matvec(cfg, x, q, y, F.MatvecWorkspace(T, N, K, cfg))
    for n in range(0, N, 1 << 22):
        w = ref.values(q.codes[n:n + (1 << 22)], q.scales[n:n + (1 << 22)], 0)
        for t in range(0, T, 1 << 19):
            if K <= 4096:
                want = x[t:t + (1 << 19)].double() @ w.T.contiguous()
            else:
                want = x[t:t + (1 << 19)][:, at.unique()].double() @ w[:, at.unique()].T.contiguous()
            assert torch.equal(y[t:t + (1 << 19), n:n + (1 << 22)].double(), want)


def test_most_sequences(env):
    """65535 sequences of 0 to 100 tokens: the rows of calls of a few of them."""
    torch, F = env
    g = torch.Generator(device="cuda").manual_seed(2)
    B, H, D, P = 65535, 2, 32, 32
    cfg = F.config(rht=1, rht_seed=3)
    c = F.alloc_cache(50, P, H, D)
    k, v = (torch.randn(50 * P, H * D, device="cuda", generator=g).bfloat16() for _ in range(2))
    F.ufp4_cache_append(cfg, c, k, v, torch.arange(50 * P, device="cuda"))
    table = torch.randint(0, 50, (B, 4), device="cuda", generator=g, dtype=torch.int32)
    lens = torch.randint(0, 101, (B,), device="cuda", generator=g, dtype=torch.int32)
    q = torch.randn(B, 3 * H * D, device="cuda", generator=g).bfloat16()

    def run(rows):
        n = rows.numel()
        o, e = torch.empty(n, 3 * H * D, dtype=torch.bfloat16, device="cuda"), torch.empty(n, 3 * H, device="cuda")
        F.ufp4_tree_attention(cfg, c, q[rows], torch.arange(n + 1, device="cuda"), lens[rows], table[rows], 1, o,
                              F.AttentionWorkspace(c, 3 * H, n, 1), lse=e)
        return o, e

    o, e = run(torch.arange(B, device="cuda"))
    for rows in (torch.arange(3), torch.arange(40000, 40100), torch.arange(B - 300, B)):
        few = run(rows.cuda())
        assert torch.equal(o[rows.cuda()], few[0]) and torch.equal(e[rows.cuda()], few[1])
    assert bool((o[lens == 0] == 0).all()) and bool(torch.isneginf(e[lens == 0]).all())


def test_most_heads_and_longest_pages(env):
    """1024 key heads under 8192 query heads, pages of 65536 tokens: each head and the
    first tokens of a page as in a cache of one head and short pages."""
    torch, F = env
    g = torch.Generator(device="cuda").manual_seed(4)
    H, G, D, T = 1024, 8, 32, 90
    cfg = F.config(rht=1, rht_seed=3)
    k, v = (torch.randn(T, H * D, device="cuda", generator=g).bfloat16() for _ in range(2))
    q = torch.randn(2, H * G * D, device="cuda", generator=g).bfloat16()
    off, lens = torch.tensor([0, 2], device="cuda"), torch.tensor([T], dtype=torch.int32, device="cuda")

    def run(k, v, q, heads, P):
        c = F.alloc_cache(2, P, heads, D)
        slots = torch.arange(T, device="cuda") + P  # page 1
        if P < T:
            slots = torch.arange(T, device="cuda")
        F.ufp4_cache_append(cfg, c, k, v, slots)
        table = torch.tensor([[1] if P >= T else [0, 1]], dtype=torch.int32, device="cuda")
        o = torch.empty_like(q)
        F.ufp4_tree_attention(cfg, c, q, off, lens, table, 2, o, F.AttentionWorkspace(c, heads * G, 1, 2))
        a, b = torch.empty_like(k), torch.empty_like(v)
        F.ufp4_cache_read(cfg, c, slots, a, b)
        return o, a, b

    whole = run(k, v, q, H, 65536)
    for h in (0, 1, 511, 1023):
        kv, qs = slice(h * D, (h + 1) * D), slice(h * G * D, (h + 1) * G * D)
        one = run(k[:, kv].contiguous(), v[:, kv].contiguous(), q[:, qs].contiguous(), 1, 64)
        assert torch.equal(whole[0][:, qs], one[0]) and torch.equal(whole[1][:, kv], one[1]) and torch.equal(whole[2][:, kv], one[2])
