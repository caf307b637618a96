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


@pytest.mark.parametrize("rht", [0, 1])
def test_rows_that_see_nothing(env, rht):
    """Masks that leave a row (or all of a sequence) empty, histories of no token,
    more drafted tokens than the cache holds, lengths outside the table."""
    torch, F = env
    lengths, drafts = [3, 0, 40, 2, 33], [3, 2, 4, 5, 2]
    cfg, c, table = build(env, lengths, 2, 64, 32, E1M2, rht)
    mask = tree(torch, drafts, 1)
    mask[0] = 0          # no history, sees nothing
    mask[2] = 0b010      # one other token alone
    mask[5] = 0          # sees its history
    mask[9:14] = -1      # bits of tokens that do not exist
    compare(env, cfg, c, table, lengths, drafts, 3, mask=mask)
    compare(env, cfg, c, table, lengths, drafts, 3)
    compare(env, cfg, c, table, [-5, 1 << 30, 40, 0, 33], drafts, 3)


def test_rows_left_out(env):
    """Drafted tokens past max_draft, sequences whose rows lie outside q."""
    torch, F = env
    lengths, drafts = [50, 70, 20], [6, 3, 9]
    cfg, c, table = build(env, lengths, 1, 96, 32, E2M1, 1)
    compare(env, cfg, c, table, lengths, drafts, 2, max_draft=4)
    compare(env, cfg, c, table, lengths, drafts, 2, max_draft=9, offsets=[0, 6, 4, 13])
    compare(env, cfg, c, table, lengths, drafts, 2, max_draft=9, offsets=[-2, 4, 7, 16])


def test_pages_outside_the_cache(env):
    torch, F = env
    lengths, drafts = [300, 64], [2, 1]
    cfg, c, table = build(env, lengths, 2, 128, 32, INT4, 1)
    table[0, 1], table[0, 4], table[1, 0] = -1, c.pages, 1 << 30
    compare(env, cfg, c, table, lengths, drafts, 2)
    table[1, 1] = -(1 << 31)  # nothing left of the second sequence
    compare(env, cfg, c, table, lengths, drafts, 2)


@pytest.mark.parametrize("spread,scale", [(1.5, 0.0), (30.0, 1.0), (1e-30, 0.1), (1e4, 1e-4), (1.5, -0.2)])
def test_logits_of_all_sizes(env, spread, scale):
    cfg, c, table = build(env, [260, 31], 2, 64, 32, E1M2, 1)
    compare(env, cfg, c, table, [260, 31], [3, 1], 2, scale=scale, spread=spread)


@pytest.mark.parametrize("scaled", [True, False])
def test_head_scales(env, scaled):
    """No tensor scales, and entries that are not positive finite numbers: 1."""
    torch, F = env
    cfg, c, table = build(env, [100], 3, 64, 32, E1M2, 0, scaled=scaled)
    if scaled:
        c.k_scale[0], c.k_scale[1], c.v_scale[2] = 0.0, float("nan"), float("inf")
    compare(env, cfg, c, table, [100], [1], 1, scale=0.01)


def test_a_lost_row_stays_alone(env):
    """NaN and infinities in one query row: the others are bit for bit what they were."""
    torch, F = env
    cfg, c, table = build(env, [200, 70], 2, 128, 32, E1M2, 1)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(9, 4 * 128, device="cuda", generator=g).bfloat16()
    off, lens = torch.tensor([0, 6, 9], device="cuda"), torch.tensor([200, 70], dtype=torch.int32, device="cuda")
    ws = F.AttentionWorkspace(c, 4, 2, 6)
    outs = []
    for bad in (None, float("nan"), float("inf")):
        x = q.clone()
        if bad is not None:
            x[4, 130] = bad
        o = torch.empty_like(x)
        F.ufp4_tree_attention(cfg, c, x, off, lens, table, 6, o, ws)
        outs.append(o.view(9, 4, 128))
    for o in outs[1:]:
        assert bool(torch.isnan(o[4, 1].float()).all())
        o[4, 1] = outs[0][4, 1]
        assert torch.equal(o, outs[0])


def test_many_sequences_and_long_runs(env):
    """More sequences than a workgroup has threads, and runs of more steps than a
    wave holds pages of: the same rows as in calls of a few sequences."""
    torch, F = env
    g = torch.Generator(device="cuda").manual_seed(2)
    for B, H, lens in ((700, 1, None), (26, 32, 16384)):
        lengths = [lens or int(n) for n in torch.randint(0, 300, (B,), generator=torch.Generator().manual_seed(1))]
        cfg, c, table = build(env, lengths, H, 32, 64, E1M2, 1, garbage=False)
        q = torch.randn(B, H * 32, device="cuda", generator=g).bfloat16()
        dev = torch.tensor(lengths, dtype=torch.int32, device="cuda")

        def run(rows):
            n = len(rows)
            o = torch.empty(n, H * 32, dtype=torch.bfloat16, device="cuda")
            F.ufp4_tree_attention(cfg, c, q[rows].contiguous(), torch.arange(n + 1, device="cuda"), dev[rows].contiguous(),
                                  table[rows].contiguous(), 1, o, F.AttentionWorkspace(c, H, n, 1))
            return o

        whole = run(list(range(B)))
        for rows in ([0, 1], [B // 2], [B - 2, B - 1]):
            few = run(rows)
            # sums of other lengths: a rounding of bf16 and fp16's of the weights apart
            err = (few.float() - whole[rows].float()).abs()
            assert bool((err <= 2.0 ** -7 * few.float().abs() + 2.0 ** -10 * few.float().abs().amax(1, keepdim=True)).all())
