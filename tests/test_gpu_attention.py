"""Attention of drafted tokens over the 4-bit cache against 64 bits."""
import math

import pytest
import serve_reference as ref

pytestmark = pytest.mark.gpu

E1M2, INT4, E2M1, E2M1C = range(4)


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp4_quantization_amd as F
    return torch, F


def build(env, lengths, H, D, P, grid, rht, scaled=True, seed=1, spare=2, garbage=True):
    """A cache that holds the sequences, written by ufp4_cache_append, with NaN
    scales and any codes in every slot that no token was written to; cfg, cache,
    page table."""
    torch, F = env
    g = torch.Generator(device="cuda").manual_seed(seed)
    cfg = F.config(grid=grid, rht=rht, rht_seed=13)
    need = [-(-n // P) for n in lengths]
    pages = sum(need) + spare
    scale = [0.004 + 0.004 * torch.rand(H, device="cuda", generator=g) for _ in range(2)] if scaled else [None, None]
    c = F.alloc_cache(pages, P, H, D, *scale)
    if garbage:
        c.k_codes.fill_(0x5B)
        c.v_codes.fill_(0xE3)
        c.k_scales.fill_(0x7F)
        c.v_scales.fill_(0xFF)
    order = torch.randperm(pages, device="cuda", generator=g)
    table = torch.full((len(lengths), max(need + [1])), -1, dtype=torch.int32, device="cuda")
    at, slots = 0, []
    for b, n in enumerate(lengths):
        table[b, :need[b]] = order[at:at + need[b]].int()
        at += need[b]
        t = torch.arange(n, device="cuda")
        slots.append(table[b].long()[t // P] * P + t % P)
    slots = torch.cat(slots)
    n = slots.numel()
    if n:
        big = torch.where(torch.rand(H * D, device="cuda", generator=g) < 0.03, 5.0, 1.0)
        k = ((torch.randn(n, H * D, device="cuda", generator=g) + 0.3) * big).bfloat16()
        v = (torch.randn(n, H * D, device="cuda", generator=g) * big).bfloat16()
        F.ufp4_cache_append(cfg, c, k, v, slots)
    return cfg, c, table


def tree(torch, drafts, seed):
    import random
    r = random.Random(seed)
    out = []
    for n in drafts:
        parents = [r.randint(max(-1, i - 4), i - 1) for i in range(n)]
        for i in range(n):
            m, j = 0, i
            while j >= 0:
                m |= 1 << j
                j = parents[j]
            out.append(m - (1 << 64) if m >> 63 else m)
    return torch.tensor(out, dtype=torch.int64, device="cuda")


def compare(env, cfg, c, table, lengths, drafts, G, mask=None, max_draft=None, scale=None, seed=5, offsets=None, spread=1.5):
    torch, F = env
    g = torch.Generator(device="cuda").manual_seed(seed)
    H, D = c.heads, c.dim
    if offsets is None:
        offsets = [0]
        for n in drafts:
            offsets.append(offsets[-1] + n)
    rows = max(offsets) + 1  # one row behind the last sequence
    off = torch.tensor(offsets, dtype=torch.int64, device="cuda")
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    most = max(drafts + [1]) if max_draft is None else max_draft
    W = H * G * D
    q = (spread * torch.randn(rows, W + 9, device="cuda", generator=g)).bfloat16()[:, 3:3 + W]
    full = torch.full((rows, W + 5), -7.0, dtype=torch.bfloat16, device="cuda")
    out = full[:, 1:1 + W]
    lse = torch.full((rows, H * G), -7.0, device="cuda")
    if mask is not None and mask.numel() < rows:
        mask = torch.cat([mask, torch.full((rows - mask.numel(),), -1, dtype=torch.int64, device="cuda")])
    sc = D ** -0.5 if scale is None else scale
    ws = F.AttentionWorkspace(c, H * G, len(lengths), most)
    F.ufp4_tree_attention(cfg, c, q, off, lens, table, most, out, ws, mask=mask, softmax_scale=sc, lse=lse)
    want, wlse, e_out, e_lse = ref.attention(c, cfg.grid, cfg.rht, F.ufp4_rht_signs(cfg.rht_seed), q, off, lens, table, most,
                                             mask, sc)
    written = ~torch.isnan(want[:, 0, 0])
    o = out.view(rows, H * G, D) if out.is_contiguous() else out.reshape(rows, H * G, D)
    assert bool((o[~written] == -7.0).all()) and bool((lse[~written] == -7.0).all())
    assert bool((full[:, 0] == -7.0).all()) and bool((full[:, 1 + W:] == -7.0).all())
    half = torch.finfo(torch.bfloat16).eps / 2
    err, bound = (o.double() - want).abs()[written], (e_out * (1 + half) + half * want.abs() + 1e-30)[written]
    finite = torch.isfinite(wlse[written])
    assert torch.equal(torch.isfinite(lse[written]), finite) and bool((lse[written][~finite] == -math.inf).all())
    el, bl = (lse.double() - wlse).abs()[written][finite], e_lse[written][finite] + 1e-30
    if err.numel():
        print("out", float((err / bound).max()), "lse", float((el / bl).max()) if el.numel() else None, flush=True)
    assert bool((err <= bound).all()) and bool((el <= bl).all())
    return out, lse


CASES = [
    # lengths, drafts, H, G, D, P, grid, rht, tree
    ([1], [1], 1, 1, 32, 32, E1M2, 1, False),
    ([2], [1], 2, 4, 64, 32, E1M2, 0, False),
    ([31], [1], 1, 16, 128, 32, E1M2, 1, False),
    ([517], [1], 8, 4, 128, 64, E1M2, 1, False),
    ([129, 0, 33, 1, 64], [1, 1, 1, 1, 1], 2, 2, 96, 64, INT4, 1, False),
    ([1000, 5, 300], [4, 5, 2], 2, 3, 160, 96, E2M1, 0, False),
    ([1000, 27, 300, 40], [27, 27, 0, 13], 2, 3, 96, 96, E2M1, 1, True),
    ([4000], [64], 1, 2, 256, 128, INT4, 1, True),
    ([700, 90], [8, 3], 1, 8, 192, 32, E2M1C, 1, False),
    ([2500, 100], [2, 1], 3, 5, 64, 256, INT4, 0, True),
    ([200], [150], 1, 1, 32, 32, E1M2, 1, False),
    ([1500], [16], 2, 1, 224, 64, E1M2, 0, True),
]


@pytest.mark.parametrize("lengths,drafts,H,G,D,P,grid,rht,is_tree", CASES)
def test_values(env, lengths, drafts, H, G, D, P, grid, rht, is_tree):
    cfg, c, table = build(env, lengths, H, D, P, grid, rht)
    compare(env, cfg, c, table, lengths, drafts, G, mask=tree(env[0], drafts, 3) if is_tree else None)
