"""Plain 64-bit forms of the decoding operators, from the layouts and formulas
of include/ufp4.h (helper of the tests; no kernel code)."""
import math

import torch

QMAX = (3.5, 7.0, 6.0, 2.0)
MAGNITUDES = ([0, .5, 1, 1.5, 2, 2.5, 3, 3.5], [0, 1, 2, 3, 4, 5, 6, 7], [0, .5, 1, 1.5, 2, 3, 4, 6], [0, .5, 1, 1.5, 2, 3, 4, 6])


def hadamard(signs):
    """The transform of 16 values as a float64 matrix (row i of the result)."""
    h = [[float(signs[j]) * (-1) ** bin(i & j).count("1") / 4 for j in range(16)] for i in range(16)]
    return torch.tensor(h, dtype=torch.float64)


def along(x, m):
    """m times every 16 neighbouring values of the last axis."""
    return torch.matmul(x.reshape(*x.shape[:-1], -1, 16), m.to(x.device).T).reshape(x.shape)


def block_sums(x):
    """Sum of magnitudes of each block of 16, at each of its values."""
    return x.abs().reshape(*x.shape[:-1], -1, 16).sum(-1).repeat_interleave(16, -1)


def values(codes, scales, grid, mx=False):
    """value(code) * block scale along the last axis, float64."""
    c = codes.view(torch.uint8)
    n = torch.stack([c & 15, c >> 4], -1).flatten(-2).long()
    m = MAGNITUDES[grid]
    table = m + ([0] + [-v for v in m[:0:-1]] if grid == 1 else [-v for v in m])
    v = torch.tensor(table, dtype=torch.float64, device=c.device)[n]
    if mx:
        d = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=c.device), scales.double() - 127)
        return v * d.repeat_interleave(32, -1)
    s = scales.view(torch.uint8).long()
    d = torch.where(s >= 8, (8 + (s & 7)).double() * torch.exp2((s >> 3).double() - 10).round(decimals=12), (s & 7).double() / 512)
    return v * d.repeat_interleave(16, -1)


def cache_rows(cache, slots, which):
    """(codes, scales) [T, heads, ...] of the tokens at `slots` of keys or values."""
    page, at = slots // cache.page_tokens, slots % cache.page_tokens
    if which == "k":
        return cache.k_codes[page, :, at], cache.k_scales[page, :, at]
    return cache.v_codes[page, :, at // 32, :, at % 32], cache.v_scales[page, :, at // 32, :, at % 32]


def head_scales(t, heads, device):
    if t is None:
        return torch.ones(heads, dtype=torch.float64, device=device)
    t = t.double()
    return torch.where((t > 0) & torch.isfinite(t), t, torch.ones_like(t))


def attention(cache, grid, rht, signs, q, q_offsets, lengths, table, max_draft, mask, scale):
    """out, lse in float64, and a bound of the kernel's error of each before the
    rounding to bf16 (arithmetic at the bound's lines); rows that are not to be
    written are NaN."""
    H, D, P = cache.heads, cache.dim, cache.page_tokens
    dev = q.device
    rows, G = q.shape[0], q.shape[1] // D // H
    out = torch.full((rows, H * G, D), math.nan, dtype=torch.float64, device=dev)
    lse = torch.full((rows, H * G), math.nan, dtype=torch.float64, device=dev)
    e_out, e_lse = torch.zeros_like(out), torch.zeros_like(lse)
    T = hadamard(signs)
    kt, vt = head_scales(cache.k_scale, H, dev), head_scales(cache.v_scale, H, dev)
    qd = q.double().view(rows, H * G, D)
    qa = block_sums(qd) / 4 if rht else qd.abs()  # no |transformed value| is larger
    if rht:
        qd = along(qd, T)
    off, lens = q_offsets.tolist(), lengths.tolist()
    for b in range(len(lens)):
        r0, r1, L = off[b], off[b + 1], max(0, min(lens[b], table.shape[1] * P))
        if r0 < 0 or r1 < r0 or r1 > rows:
            continue
        n = r1 - r0
        t = torch.arange(L, device=dev)
        page = table[b].long()[t // P]
        there = (page >= 0) & (page < cache.pages)
        slots = torch.where(there, page, 0) * P + t % P
        for i in range(min(n, max_draft)):
            d = t - (L - n)
            bits = (1 << (i + 1)) - 1 if mask is None else int(mask[r0 + i]) & (2 ** 64 - 1)
            seen = torch.tensor([x < 0 or (x < 64 if mask is not None else True) and bool((bits >> x) & 1) for x in d.tolist()],
                                dtype=torch.bool, device=dev) & there
            at = slots[seen]
            if at.numel() == 0:
                out[r0 + i], lse[r0 + i] = 0.0, -math.inf
                continue
            k = values(*cache_rows(cache, at, "k"), grid) * kt[:, None]
            v = values(*cache_rows(cache, at, "v"), grid) * vt[:, None]
            for h in range(H * G):
                kh, vh, x = k[:, h // G], v[:, h // G], qd[r0 + i, h]
                a = kh @ x * scale
                # logits: transform 4 roundings and 22 bits of two fp16 parts (or
                # exact), D products in fp32 sums of at most 2^-23 each, factors
                ea = (kh.abs() @ qa[r0 + i, h]) * abs(scale) * ((2.0 ** -21 if rht else 0.0) + (D + 4) * 2.0 ** -23)
                ea = ea.max() + 2.0 ** -22 * a.abs().max()  # exp2's argument in fp32
                p = torch.softmax(a, 0)
                out[r0 + i, h] = p @ vh
                lse[r0 + i, h] = torch.logsumexp(a, 0)
                # weights: twice the logits' error and exp2 (numerator and sum), fp16's
                # half step and smallest number (the largest weight is 1, the sum at
                # least 1), fp32 sums of len(p) terms
                ep = 2 * ea + 2.0 ** -21 + 2.0 ** -11 + (at.numel() + 64) * 2.0 ** -23
                e_out[r0 + i, h] = ep * (p @ vh.abs()) + 2.0 ** -25 * vh.abs().sum(0)
                e_lse[r0 + i, h] = ea + (at.numel() + 64) * 2.0 ** -23 + 2.0 ** -22 * (1 + lse[r0 + i, h].abs())
    if rht:
        out = along(out, T.T)
        e_out = block_sums(e_out) / 4 + 2.0 ** -22 * block_sums(out)
    return out, lse, e_out, e_lse
