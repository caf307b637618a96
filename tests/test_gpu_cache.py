"""The 4-bit key-value cache: appended tokens against the oracle's quantizer,
bit for bit, and what is read back."""
import numpy as np
import pytest
import serve_reference as ref

pytestmark = pytest.mark.gpu

E1M2, INT4, E2M1, E2M1C = range(4)


@pytest.fixture(scope="module")
def env(orc):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp4_quantization_amd as F
    return torch, F, orc


def bits(t):
    import torch
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def tensor_scales(torch, heads, grid, seed):
    """(maxima, S_t) of each head: S_t = fl(max / fl(Qmax * 448))."""
    g = np.random.default_rng(seed)
    amax = (1.0 + 5.0 * g.random(heads)).astype(np.float32)
    return amax, torch.from_numpy(amax / np.float32(ref.QMAX[grid] * 448.0)).cuda()


def make(env, pages, P, H, D, grid, scaled=True, fill=0xA7):
    torch, F, _ = env
    ka, ks = tensor_scales(torch, H, grid, 1)
    va, vs = tensor_scales(torch, H, grid, 2)
    if not scaled:  # S_t = 1: what a largest magnitude of Qmax * 448 gives
        ka = va = np.full(H, ref.QMAX[grid] * 448.0, np.float32)
        ks = vs = None
    c = F.alloc_cache(pages, P, H, D, ks, vs)
    for t in c._tensors[:4]:
        t.fill_(fill)
    return c, ka, va


def inputs(torch, T, width, seed, special):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, width, device="cuda", generator=g)
    x *= torch.exp(2.0 * torch.randn(T, width // 16, device="cuda", generator=g)).repeat_interleave(16, 1)
    if special:
        f = x.view(-1)
        i = torch.randperm(f.numel(), device="cuda", generator=g)[: max(1, f.numel() // 50)]
        odd = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38, 1e-40, -0.0], device="cuda")
        f[i] = odd[torch.arange(i.numel(), device="cuda") % 6]
        x[0, :32] = 0.0
    return x.to(torch.bfloat16)


def check_written(env, cfg, c, k, v, slots, ka, va, fill=0xA7):
    """Every slot's codes and scales are the oracle's, every other slot's are untouched."""
    torch, F, orc = env
    H, D, P = c.heads, c.dim, c.page_tokens
    ocfg = orc.config(grid=cfg.grid, rht=cfg.rht, rht_seed=cfg.rht_seed)
    want = [np.full(t.shape, fill, np.uint8) for t in c._tensors[:4]]
    s = slots.cpu().numpy()
    live = np.nonzero((s >= 0) & (s < c.pages * P))[0]
    page, at = s[live] // P, s[live] % P
    for h in range(H):
        for x, amax, codes, scales, value in ((k, ka, want[0], want[1], False), (v, va, want[2], want[3], True)):
            oc, os, _, _ = orc.quantize_given_amax(bits(x[:, h * D:(h + 1) * D]), ocfg, 0, float(amax[h]))
            if value:
                codes[page, h, at // 32, :, at % 32] = oc[live]
                scales[page, h, at // 32, :, at % 32] = os[live]
            else:
                codes[page, h, at] = oc[live]
                scales[page, h, at] = os[live]
    for t, w in zip(c._tensors[:4], want):
        assert np.array_equal(t.cpu().numpy(), w)


CASES = [
    # T, pages, P, H, D, grid, rht, scaled, special
    (1, 2, 32, 1, 32, E1M2, 1, False, False), (1, 3, 64, 8, 128, E1M2, 1, True, False),
    (5, 2, 32, 3, 96, INT4, 1, True, True), (33, 4, 96, 2, 64, E2M1, 0, True, True),
    (200, 7, 64, 2, 160, E1M2, 0, True, True), (130, 3, 256, 5, 256, E2M1C, 1, False, False),
    (1000, 40, 32, 1, 192, INT4, 0, False, True), (64, 5, 32, 2, 224, E2M1, 1, True, False),
]


@pytest.mark.parametrize("order", ["run", "scattered"])
@pytest.mark.parametrize("T,pages,P,H,D,grid,rht,scaled,special", CASES)
def test_append_and_read(env, T, pages, P, H, D, grid, rht, scaled, special, order):
    torch, F, orc = env
    cfg = F.config(grid=grid, rht=rht, rht_seed=9)
    c, ka, va = make(env, pages, P, H, D, grid, scaled)
    n = min(T, pages * P - 1)
    if order == "run":  # neighbouring slots from the middle of a tile on
        slots = (torch.arange(T, device="cuda") + min(5, pages * P - n)).long()
    else:
        slots = torch.randperm(pages * P, device="cuda", generator=torch.Generator(device="cuda").manual_seed(T)).long()
        slots = slots[torch.arange(T, device="cuda") % slots.numel()]
    # dropped tokens: before the cache, behind it, far out
    slots[n:] = pages * P
    for i, s in ((0, -1), (3, pages * P), (4, 1 << 62), (7, -(1 << 62))):
        if T > 8:
            slots[i] = s
    # rows inside a wider buffer, at odd addresses
    k = inputs(torch, T, H * D + 32, 3, special)[:, 1:1 + H * D]
    v = inputs(torch, T, H * D + 16, 4, special)[:, 5:5 + H * D]
    F.ufp4_cache_append(cfg, c, k, v, slots)
    check_written(env, cfg, c, k, v, slots, ka, va)
    # read back: the oracle's values in fp32, rounded once in bf16
    live = (slots >= 0) & (slots < pages * P)
    ocfg = orc.config(grid=grid, rht=rht, rht_seed=9)
    want = []
    for x, amax in ((k, ka), (v, va)):
        w = np.zeros((T, H * D), np.float32)
        for h in range(H):
            oc, os, ts, _ = orc.quantize_given_amax(bits(x[:, h * D:(h + 1) * D]), ocfg, 0, float(amax[h]))
            w[:, h * D:(h + 1) * D] = orc.dequantize(oc, os, ts, T, D, ocfg, bool(rht))
        w[~live.cpu().numpy()] = 0.0
        want.append(torch.from_numpy(w).cuda())
    for kind in (torch.float32, torch.bfloat16):
        full = [torch.full((T, H * D + 3), -7.0, dtype=kind, device="cuda") for _ in range(2)]
        outs = [f[:, 2:2 + H * D] for f in full]
        F.ufp4_cache_read(cfg, c, slots, *outs, bool(rht))
        for o, w, f in zip(outs, want, full):
            assert torch.equal(o, w.to(kind))
            assert bool((f[:, :2] == -7.0).all()) and bool((f[:, 2 + H * D:] == -7.0).all())
        one = torch.empty(T, H * D, dtype=kind, device="cuda")
        F.ufp4_cache_read(cfg, c, slots, None, one, bool(rht))
        assert torch.equal(one, want[1].to(kind))
        F.ufp4_cache_read(cfg, c, slots, one, None, bool(rht))
        assert torch.equal(one, want[0].to(kind))


def test_past_32_bits(env):
    """A cache of more than 4 GiB of codes: slots at its end, read by attention too."""
    torch, F, orc = env
    H, D, P = 8, 256, 256
    pages = (1 << 32) // (P * H * D // 2) + 9
    cfg = F.config(rht=1, rht_seed=4)
    c = F.alloc_cache(pages, P, H, D)
    assert c.k_codes.numel() > 1 << 32
    T = 70
    slots = torch.arange(T, device="cuda") + (pages - 1) * P + 11
    k, v = (inputs(torch, T, H * D, s, False) for s in (3, 4))
    F.ufp4_cache_append(cfg, c, k, v, slots)
    small = F.alloc_cache(2, P, H, D)
    near = torch.arange(T, device="cuda") + 11
    F.ufp4_cache_append(cfg, small, k, v, near)
    outs = []
    for cache, s, page in ((c, slots, pages - 1), (small, near, 0)):
        a, b = (torch.empty(T, H * D, device="cuda") for _ in range(2))
        F.ufp4_cache_read(cfg, cache, s, a, b)
        o = torch.empty(1, H * D, dtype=torch.bfloat16, device="cuda")
        # the first 11 slots of the page: written too
        F.ufp4_cache_append(cfg, cache, k[:11], v[:11], torch.arange(11, device="cuda") + page * P)
        F.ufp4_tree_attention(cfg, cache, k[:1], torch.tensor([0, 1], device="cuda"), torch.tensor([81], dtype=torch.int32, device="cuda"),
                              torch.tensor([[page]], dtype=torch.int32, device="cuda"), 1, o, F.AttentionWorkspace(cache, H, 1, 1))
        outs.append((a, b, o))
    assert all(torch.equal(x, y) for x, y in zip(*outs))


@pytest.mark.parametrize("ts", [0.0, -1.0, float("nan"), float("inf")])
def test_tensor_scales_that_are_none(env, ts):
    torch, F, orc = env
    cfg = F.config(rht=0)
    k = inputs(torch, 40, 64, 1, False)
    slots = torch.arange(40, device="cuda")
    got = []
    for scale in (None, torch.full((2,), ts, device="cuda")):
        c = F.alloc_cache(2, 32, 2, 32, scale, scale)
        F.ufp4_cache_append(cfg, c, k, k, slots)
        a = torch.empty(40, 64, device="cuda")
        F.ufp4_cache_read(cfg, c, slots, a, None, False)
        got.append(a)
    assert torch.equal(*got)


def test_a_slot_read_twice(env):
    torch, F, orc = env
    cfg = F.config(rht=1)
    k = inputs(torch, 5, 32, 1, False)
    c = F.alloc_cache(1, 32, 1, 32)
    F.ufp4_cache_append(cfg, c, k, k, torch.arange(5, device="cuda"))
    a = torch.empty(9, 32, device="cuda")
    F.ufp4_cache_read(cfg, c, torch.tensor([1, 1, 4, 1, 0, 4, 4, 2, 1], device="cuda"), None, a)
    b = torch.empty(5, 32, device="cuda")
    F.ufp4_cache_read(cfg, c, torch.arange(5, device="cuda"), None, b)
    assert torch.equal(a, b[torch.tensor([1, 1, 4, 1, 0, 4, 4, 2, 1], device="cuda")])


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
def test_large_reads(env, kind):
    """Results larger than the caches are stored past them: the same values as in
    calls of a few tokens."""
    torch, F, orc = env
    H, D, P, T = 8, 256, 64, 17000
    kind = getattr(torch, kind)
    cfg = F.config(rht=1, rht_seed=4)
    c = F.alloc_cache(T // P + 1, P, H, D)
    k = inputs(torch, T, H * D, 1, False)
    slots = torch.arange(T, device="cuda")
    F.ufp4_cache_append(cfg, c, k, k.flip(0).contiguous(), slots)
    a, b = (torch.empty(T, H * D, dtype=kind, device="cuda") for _ in range(2))
    F.ufp4_cache_read(cfg, c, slots, a, b)
    for t in (0, 4099, T - 1000):
        x, y = (torch.empty(1000, H * D, dtype=kind, device="cuda") for _ in range(2))
        F.ufp4_cache_read(cfg, c, slots[t:t + 1000], x, y)
        assert torch.equal(a[t:t + 1000], x) and torch.equal(b[t:t + 1000], y)
