"""Cases and plain forms of the operators that run a model on the library's 4-bit formats: products of a few rows with
4-bit weights, a key-value cache that is quantized as it is written and read back, and attention of drafted tokens over
that cache.

``run`` computes one pass through an operator, with elementary torch operations in 32 bits (``own`` false) or with
the library's entry points (``own`` true); ``exact`` gives the same outputs from the definitions in 64 bits.

Symbols: T tokens, N outputs and K inputs of a weight matrix; H key/value heads, G query heads that share one, D values
a head, P tokens a page of the cache, B sequences, L tokens of a sequence, S drafted tokens of a sequence.  Cache
layouts (a tile is 32 tokens of a page): key codes [page][H][P][D/2] and scales [page][H][P][D/16]; value codes
[page][H][tile][D/2][32] and scales [page][H][tile][D/16][32].
"""
import math
import random

import torch

own = False

# ---------------------------------------------------------------- cases


def listed():
    return [
        # one decoded token through a square projection (latency)
        {"name": "matvec_token", "op": "matvec", "T": 1, "N": 4096, "K": 4096, "grid": "e1m2", "scaling": "nv16",
         "rht": True, "x": "bf16", "y": "bf16"},
        # one decoded token through the widest matrix of a model: bound by reading the weights
        {"name": "matvec_wide", "op": "matvec", "T": 1, "N": 65536, "K": 8192, "grid": "e1m2", "scaling": "nv16",
         "rht": True, "x": "bf16", "y": "bf16"},
        # a decoded batch through the gate and up projections, baseline format without the transform
        {"name": "matvec_batch", "op": "matvec", "T": 16, "N": 16384, "K": 4096, "grid": "e2m1", "scaling": "nv16",
         "rht": False, "x": "bf16", "y": "bf16"},
        # a few drafted tokens at odd sizes, power-of-two scales, 32-bit outputs (logits)
        {"name": "matvec_odd", "op": "matvec", "T": 37, "N": 1365, "K": 2080, "grid": "int4", "scaling": "mx32",
         "rht": True, "x": "f32", "y": "f32"},
        # a decode step: 64 sequences write one token each, all over the cache, and read it back
        {"name": "append_decode", "op": "append", "T": 64, "run": 1, "H": 8, "D": 128, "P": 64, "grid": "e1m2",
         "rht": True, "out": "bf16", "scaled": True},
        # a prompt's keys and values as they are written, and read back for the rest of the prompt; ragged
        {"name": "append_prompt", "op": "append", "T": 8191, "run": 1021, "H": 8, "D": 128, "P": 64, "grid": "int4",
         "rht": True, "out": "bf16", "scaled": False},
        # one short sequence's cache read back (latency)
        {"name": "read_short", "op": "read", "T": 96, "run": 96, "H": 4, "D": 64, "P": 32, "grid": "e1m2",
         "rht": True, "out": "bf16", "scaled": True},
        # a long history read back, an odd head size, 32-bit values
        {"name": "read_long", "op": "read", "T": 50001, "run": 7000, "H": 4, "D": 160, "P": 128, "grid": "e2m1",
         "rht": False, "out": "f32", "scaled": True},
        # one sequence, one token, a short history (latency)
        {"name": "attend_token", "op": "attend", "B": 1, "S": 1, "L": 517, "H": 8, "G": 4, "D": 128, "P": 64,
         "grid": "e1m2", "rht": True, "ragged": False, "tree": False},
        # a decoded batch over histories of all lengths
        {"name": "attend_batch", "op": "attend", "B": 64, "S": 1, "L": 16384, "H": 8, "G": 4, "D": 128, "P": 64,
         "grid": "e1m2", "rht": True, "ragged": True, "tree": False},
        # trees of drafted tokens, ragged, some sequences without any; an odd head size
        {"name": "attend_tree", "op": "attend", "B": 13, "S": 27, "L": 4999, "H": 5, "G": 3, "D": 96, "P": 96,
         "grid": "e2m1", "rht": False, "ragged": True, "tree": True},
        # two very long histories, chains of drafted tokens, wide heads
        {"name": "attend_long", "op": "attend", "B": 2, "S": 4, "L": 131072, "H": 4, "G": 8, "D": 256, "P": 128,
         "grid": "int4", "rht": True, "ragged": False, "tree": False},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["matvec", "matvec", "append", "read", "attend", "attend"])
    grid = rng.choice(["e1m2", "int4", "e2m1"])
    if op == "matvec":
        T = _spread(rng, 1, 64)
        return {"op": op, "T": T, "N": _spread(rng, 16, 65536 // T), "K": 32 * _spread(rng, 2, 256), "grid": grid,
                "scaling": rng.choice(["nv16", "nv16", "mx32"]), "rht": rng.random() < 0.6,
                "x": rng.choice(["bf16", "bf16", "f32"]), "y": rng.choice(["bf16", "bf16", "f32"])}
    cache = {"H": rng.randint(1, 8), "D": 32 * rng.randint(1, 8), "P": rng.choice([32, 64, 96, 128, 256]), "grid": grid,
             "rht": rng.random() < 0.7}
    if op != "attend":
        T = _spread(rng, 1, 8191 if op == "append" else 32768)
        return {"op": op, "T": T, "run": _spread(rng, -(-T // 128), T), "out": rng.choice(["bf16", "bf16", "f32"]),
                "scaled": rng.random() < 0.5, **cache}
    B, S, G = _spread(rng, 1, 64), _spread(rng, 1, 48), rng.choice([1, 2, 3, 4, 8])
    most = min(1 << 18, (1 << 33) // (S * G * cache["H"] * cache["D"]))  # tokens in all: the largest listed case's work
    return {"op": op, "B": B, "S": S, "L": _spread(rng, 1, most // B), "G": G, "ragged": rng.random() < 0.7,
            "tree": rng.random() < 0.5, **cache}


# ---------------------------------------------------------------- inputs

_GRIDS = {"e1m2": 0, "int4": 1, "e2m1": 2}
_TOP = {"e1m2": 3.5, "int4": 7.0, "e2m1": 6.0}
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_TABLES = {"e1m2": [0, 0.5, 1, 1.5, 2, 2.5, 3, 3.5, 0, -0.5, -1, -1.5, -2, -2.5, -3, -3.5],
           "int4": [0, 1, 2, 3, 4, 5, 6, 7, 0, -7, -6, -5, -4, -3, -2, -1],
           "e2m1": [0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6]}
_DEV = "cuda"
_SEED = 11  # of the transform's signs
_TILE = 32


def _signs(seed):
    """The 16 signs of the transform: bits of word 0 of Philox4x32-10 with the key `seed` and the counter (0, 0, 2, 0)."""
    k0, k1, c = seed & 0xFFFFFFFF, seed >> 32, [0, 0, 2, 0]
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k0, b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k1, a & 0xFFFFFFFF]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return [-1.0 if (c[0] >> j) & 1 else 1.0 for j in range(16)]


def _butterflies(x):
    """The 16-point Walsh-Hadamard transform of every 16 values of the last axis, times 1/4."""
    shape = x.shape
    for h in (1, 2, 4, 8):
        x = x.reshape(-1, 8 // h, 2, h)
        x = torch.stack([x[:, :, 0] + x[:, :, 1], x[:, :, 0] - x[:, :, 1]], 2)
    return (x * 0.25).reshape(shape)


def _signs_along(x):
    return torch.tensor(_signs(_SEED), dtype=x.dtype, device=x.device).repeat(x.shape[-1] // 16)


def _transform(x):
    return _butterflies(x * _signs_along(x))


def _untransform(x):
    return _butterflies(x) * _signs_along(x)


def _nibbles(y, grid):
    """Codes (one a byte) of scaled values, rounded to the nearest grid value, ties to the even index."""
    a = y.abs()
    if grid == "e2m1":
        a = a.clamp(max=6.0)
        k = torch.where(a < 2, torch.round(a * 2), torch.where(a < 4, torch.round(a) + 2, torch.round(a * 0.5) + 4))
    else:
        k = torch.round((a * 2 if grid == "e1m2" else a).clamp(max=7.0))
    k = k.to(torch.int32)
    if grid == "int4":
        return torch.where(y < 0, -k, k) & 15
    return torch.where((y < 0) & (k > 0), k + 8, k)


def _pack(n):
    """Codes of neighbouring values to bytes, the first in the low half."""
    return (n[..., 0::2] | (n[..., 1::2] << 4)).to(torch.uint8)


def _quantized(x, grid, scaling, ts):
    """(codes one a byte, scale bytes) of float values in blocks along the last axis, under the tensor scale `ts` (a
    number, or a tensor that broadcasts over the blocks)."""
    B = 16 if scaling == "nv16" else 32
    blocks = x.reshape(*x.shape[:-1], -1, B)
    top = blocks.abs().amax(-1)
    if scaling == "nv16":
        ts = torch.as_tensor(ts, dtype=torch.float32, device=x.device)
        s = (top / (_TOP[grid] * ts)).clamp(max=448.0).to(torch.float8_e4m3fn)
        d = s.float() * ts
        inv = torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
        s = s.view(torch.uint8)
    else:
        e = torch.where(top > 0, torch.frexp(top)[1] - (2 if grid == "e1m2" else 3), -127).clamp(-127, 127)
        inv = torch.ldexp(torch.ones_like(top), -e)
        s = (e + 127).to(torch.uint8)
    return _nibbles(blocks * inv[..., None], grid).reshape(x.shape), s


def _weights(case, gen):
    """A quantized weight matrix: (codes, scales, tensor scale), made in pieces of rows."""
    N, K, grid, scaling = case["N"], case["K"], case["grid"], case["scaling"]
    codes = torch.empty(N, K // 2, dtype=torch.uint8, device=_DEV)
    scales = torch.empty(N, K // (16 if scaling == "nv16" else 32), dtype=torch.uint8, device=_DEV)
    ts = 0.02 * 6.0 / (_TOP[grid] * 448.0) if scaling == "nv16" else 1.0
    step = max(1, (1 << 26) // K)
    for n in range(0, N, step):
        w = 0.02 * torch.randn(min(step, N - n), K, device=_DEV, generator=gen)
        w = w.to(torch.bfloat16).float()
        c, s = _quantized(_transform(w) if case["rht"] else w, grid, scaling, ts)
        codes[n:n + step], scales[n:n + step] = _pack(c), s
    return codes, scales, torch.tensor([ts], device=_DEV)


def _activation(rows, cols, gen):
    """Rows with a mean for each channel and a few channels far larger than the others."""
    x = torch.randn(rows, cols, device=_DEV, generator=gen)
    x += torch.randn(cols, device=_DEV, generator=gen) * 0.7
    x *= torch.where(torch.rand(cols, device=_DEV, generator=gen) < 0.004, 50.0, 1.0)
    return x


def _keys_values(rows, heads, dim, shape, gen):
    """Keys or values of some tokens: means and a few large channels for each head."""
    x = torch.randn(rows, heads * dim, device=_DEV, generator=gen)
    return (x * shape[0] + shape[1]).to(torch.bfloat16)


def _kv_shape(heads, dim, gen):
    big = torch.where(torch.rand(heads * dim, device=_DEV, generator=gen) < 0.02, 6.0, 1.0)
    return big, 0.3 * big * torch.randn(heads * dim, device=_DEV, generator=gen)


def _into_cache(x, case, ts):
    """Codes (one a byte) and scales of rows [T][H D] of keys or values, as [T][H][D] and [T][H][D/16]."""
    x = x.float().view(-1, case["H"], case["D"])
    return _quantized(_transform(x) if case["rht"] else x, case["grid"], "nv16", ts[:, None])


def _place(cache, slot, kc, ks, vc, vs):
    """Writes tokens' codes (one a byte) and scales at their places of the cache's layouts."""
    P = cache["P"]
    page, at = slot // P, slot % P
    cache["k_codes"][page, :, at] = _pack(kc)
    cache["k_scales"][page, :, at] = ks
    cache["v_codes"][page, :, at // _TILE, :, at % _TILE] = _pack(vc)
    cache["v_scales"][page, :, at // _TILE, :, at % _TILE] = vs


def _empty_cache(case, pages, gen):
    H, D, P = case["H"], case["D"], case["P"]
    c = {"P": P, "pages": pages}
    for name, shape in (("k_codes", (pages, H, P, D // 2)), ("k_scales", (pages, H, P, D // 16)),
                        ("v_codes", (pages, H, P // _TILE, D // 2, _TILE)),
                        ("v_scales", (pages, H, P // _TILE, D // 16, _TILE))):
        c[name] = torch.zeros(shape, dtype=torch.uint8, device=_DEV)
    for name in ("k_ts", "v_ts"):
        # a head's largest magnitude in earlier calls, as a tensor scale; or none: 1
        c[name] = 0.01 * (0.5 + torch.rand(H, device=_DEV, generator=gen)) if case.get("scaled", True) else None
    return c


def _head_scales(cache, name, case):
    return cache[name] if cache[name] is not None else torch.ones(case["H"], device=_DEV)


def _fill(cache, case, gen):
    """Keys and values for every slot of the cache, in pieces of pages."""
    H, D, P = case["H"], case["D"], case["P"]
    ks, vs = _kv_shape(H, D, gen), _kv_shape(H, D, gen)
    step = max(1, (1 << 24) // (P * H * D))
    for p in range(0, cache["pages"], step):
        n = min(step, cache["pages"] - p)
        k, kb = _into_cache(_keys_values(n * P, H, D, ks, gen), case, _head_scales(cache, "k_ts", case))
        v, vb = _into_cache(_keys_values(n * P, H, D, vs, gen), case, _head_scales(cache, "v_ts", case))
        cache["k_codes"][p:p + n] = _pack(k).view(n, P, H, -1).transpose(1, 2)
        cache["k_scales"][p:p + n] = kb.view(n, P, H, -1).transpose(1, 2)
        cache["v_codes"][p:p + n] = _pack(v).view(n, P // _TILE, _TILE, H, -1).permute(0, 3, 1, 4, 2)
        cache["v_scales"][p:p + n] = vb.view(n, P // _TILE, _TILE, H, -1).permute(0, 3, 1, 4, 2)


def _slots(case, pages, gen):
    """Slots of T tokens: runs of `run` neighbouring ones, each in pages of its own, in any order of pages."""
    T, run, P = case["T"], case["run"], case["P"]
    order = torch.randperm(pages, device=_DEV, generator=gen)
    per = -(-(run + P - 1) // P)
    t = torch.arange(T, device=_DEV)
    starts = torch.randint(0, P, (-(-T // run),), device=_DEV, generator=gen)
    at = t % run + starts[t // run]
    return order[t // run * per + at // P] * P + at % P


def _tree_masks(parents_of, n, i):
    """Bits of the drafted tokens that token i sees: itself and its ancestors."""
    m, j = 0, i
    while j >= 0:
        m |= 1 << j
        j = parents_of[j]
    return m - (1 << 64) if m >> 63 else m


def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(seed * 1000003 + 29)
    op, s = case["op"], {"case": case}
    if op == "matvec":
        s["w"] = _weights(case, gen)
        s["x"] = _activation(case["T"], case["K"], gen).to(_TYPES[case["x"]])
        return s
    if op != "attend":
        runs = -(-case["T"] // case["run"])
        pages = runs * -(-(case["run"] + case["P"] - 1) // case["P"]) + 3
        s["cache"] = cache = _empty_cache(case, pages, gen)
        s["slots"] = _slots(case, pages, gen)
        if op == "read":
            _fill(cache, case, gen)
        else:
            shape = _kv_shape(case["H"], case["D"], gen)
            s["k"] = _keys_values(case["T"], case["H"], case["D"], shape, gen)
            s["v"] = _keys_values(case["T"], case["H"], case["D"], shape, gen)
        return s
    B, S, L, P = case["B"], case["S"], case["L"], case["P"]
    # tokens in the cache and drafted ones of each sequence (the drafted ones are its last): the case's own, so that
    # outputs of all seeds have one shape
    rng = random.Random(B * 1000003 + S * 1009 + L)
    lengths = [rng.randint(1, L) if case["ragged"] else L for _ in range(B)]
    drafts = [rng.randint(0 if S > 1 else 1, S) if case["ragged"] else S for _ in range(B)]
    drafts[-1] = S
    lengths = [max(n, d) for n, d in zip(lengths, drafts)]
    need = [-(-n // P) for n in lengths]
    pages = sum(need) + 1
    s["cache"] = cache = _empty_cache(case, pages, gen)
    _fill(cache, case, gen)
    order = torch.randperm(pages, device=_DEV, generator=gen).to(torch.int32)
    table, at = torch.full((B, max(need)), -1, dtype=torch.int32, device=_DEV), 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    s["table"], s["L"], s["S"] = table, lengths, drafts
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=_DEV)
    starts = [0]
    for n in drafts:
        starts.append(starts[-1] + n)
    s["starts"] = starts
    s["offsets"] = torch.tensor(starts, dtype=torch.int64, device=_DEV)
    s["mask"] = None
    if case["tree"]:
        rng, bits = random.Random(seed), []
        for n in drafts:
            parents = [rng.randint(max(-1, i - 6), i - 1) for i in range(n)]
            bits += [_tree_masks(parents, n, i) for i in range(n)]
        s["mask"] = torch.tensor(bits, dtype=torch.int64, device=_DEV)
    s["q"] = (1.5 * torch.randn(starts[-1], case["H"] * case["G"] * case["D"], device=_DEV, generator=gen)).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------- plain forms


def _values(codes, scales, grid, scaling):
    """Values of packed codes times their block scales, along the last axis."""
    table = torch.tensor(_TABLES[grid], dtype=torch.float32, device=codes.device)
    v = table[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    if scaling == "nv16":
        return v * scales.view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)
    return v * torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127).repeat_interleave(32, -1)


def _token_rows(cache, slots):
    """Packed codes and scales [T][H][...] of the tokens at `slots`: keys, then values."""
    page, at = slots // cache["P"], slots % cache["P"]
    return (cache["k_codes"][page, :, at], cache["k_scales"][page, :, at],
            cache["v_codes"][page, :, at // _TILE, :, at % _TILE], cache["v_scales"][page, :, at // _TILE, :, at % _TILE])


def _plain_attend(s):
    case, cache = s["case"], s["cache"]
    H, G, D, P = case["H"], case["G"], case["D"], case["P"]
    rows = s["starts"][-1]
    out = torch.zeros(rows, H * G * D, dtype=torch.bfloat16, device=_DEV)
    lse = torch.full((rows, H * G), -math.inf, device=_DEV)
    kt, vt = _head_scales(cache, "k_ts", case)[:, None, None], _head_scales(cache, "v_ts", case)[:, None, None]
    q = s["q"].float().view(rows, H, G, D)
    if case["rht"]:
        q = _transform(q)
    for b, (L, n) in enumerate(zip(s["L"], s["S"])):
        if n == 0:
            continue
        r0 = s["starts"][b]
        t = torch.arange(L, device=_DEV)
        slots = s["table"][b].long()[t // P] * P + t % P
        kc, ks, vc, vs = _token_rows(cache, slots)
        k = (_values(kc, ks, case["grid"], "nv16").transpose(0, 1) * kt).contiguous()
        v = (_values(vc, vs, case["grid"], "nv16").transpose(0, 1) * vt).contiguous()
        i = torch.arange(n, device=_DEV)
        d = t - (L - n)  # which drafted token a place holds; below 0: the history
        if s["mask"] is None:
            seen = d[None, :] <= i[:, None]
        else:
            seen = (d[None, :] < 0) | ((s["mask"][r0:r0 + n, None] >> d.clamp(min=0)[None, :]) & 1).bool()
        qb = q[r0:r0 + n].permute(1, 0, 2, 3).reshape(H, n * G, D)
        a = torch.matmul(qb, k.transpose(1, 2).contiguous()).view(H, n, G, L) * (1.0 / math.sqrt(D))
        a = torch.where(seen[None, :, None, :], a, -math.inf)
        m = a.amax(-1, keepdim=True)
        p = torch.exp(a - m)
        z = p.sum(-1, keepdim=True)
        o = (torch.matmul(p.view(H, n * G, L), v).view(H, n, G, D) / z).permute(1, 0, 2, 3)
        if case["rht"]:
            o = _untransform(o)
        out[r0:r0 + n] = o.reshape(n, -1).to(torch.bfloat16)
        lse[r0:r0 + n] = (m + torch.log(z))[..., 0].permute(1, 0, 2).reshape(n, -1)
    return {"out": out, "lse": lse}


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "matvec":
        codes, scales, ts = s["w"]
        x = s["x"].float()
        w = _values(codes, scales, case["grid"], case["scaling"])
        y = torch.matmul(_transform(x) if case["rht"] else x, w.T) * ts
        return {"y": y.to(_TYPES[case["y"]])}
    if op == "attend":
        return _plain_attend(s)
    cache = s["cache"]
    kt, vt = _head_scales(cache, "k_ts", case), _head_scales(cache, "v_ts", case)
    if op == "append":
        _place(cache, s["slots"], *_into_cache(s["k"], case, kt), *_into_cache(s["v"], case, vt))
    kc, ks, vc, vs = _token_rows(cache, s["slots"])
    out = {}
    for name, c, b, t in (("k", kc, ks, kt), ("v", vc, vs, vt)):
        x = _values(c, b, case["grid"], "nv16") * t[:, None]
        out[name] = (_untransform(x) if case["rht"] else x).flatten(1).to(_TYPES[case["out"]])
    return out


# ---------------------------------------------------------------- the library's entry points


def _own(s):
    import fp4_quantization_amd as F

    case, op = s["case"], s["case"]["op"]
    if op == "matvec":
        cfg = F.config(grid=_GRIDS[case["grid"]], scaling=F.SCALE_NV16 if case["scaling"] == "nv16" else F.SCALE_MX32,
                       rht=int(case["rht"]), rht_seed=_SEED)
        if "ws" not in s:
            s["ws"] = F.MatvecWorkspace(case["T"], case["N"], case["K"], cfg)
        y = torch.empty(case["T"], case["N"], dtype=_TYPES[case["y"]], device=_DEV)
        F.ufp4_matvec(cfg, s["x"], F.QTensor(*s["w"]), y, s["ws"])
        return {"y": y}
    cfg = F.config(grid=_GRIDS[case["grid"]], rht=int(case["rht"]), rht_seed=_SEED)
    c = s["cache"]
    if "handle" not in s:
        s["handle"] = F.QCache(c["k_codes"], c["k_scales"], c["v_codes"], c["v_scales"], c["k_ts"], c["v_ts"])
    cache = s["handle"]
    if op != "attend":
        if op == "append":
            F.ufp4_cache_append(cfg, cache, s["k"], s["v"], s["slots"])
        shape, kind = (case["T"], case["H"] * case["D"]), _TYPES[case["out"]]
        k, v = torch.empty(shape, dtype=kind, device=_DEV), torch.empty(shape, dtype=kind, device=_DEV)
        F.ufp4_cache_read(cfg, cache, s["slots"], k, v, case["rht"])
        return {"k": k, "v": v}
    rows, heads = s["q"].shape[0], case["H"] * case["G"]
    if "ws" not in s:
        s["ws"] = F.AttentionWorkspace(cache, heads, case["B"], case["S"])
    out = torch.empty(rows, heads * case["D"], dtype=torch.bfloat16, device=_DEV)
    lse = torch.empty(rows, heads, dtype=torch.float32, device=_DEV)
    F.ufp4_tree_attention(cfg, cache, s["q"], s["offsets"], s["lengths"], s["table"], case["S"], out, s["ws"],
                          mask=s["mask"], softmax_scale=1.0 / math.sqrt(case["D"]), lse=lse)
    return {"out": out, "lse": lse}


def run(s):
    return _own(s) if own else _plain(s)


# ---------------------------------------------------------------- work


def work(case):
    op = case["op"]
    if op == "matvec":
        T, N, K = case["T"], case["N"], case["K"]
        x, y = (4 if case[n] == "f32" else 2 for n in ("x", "y"))
        scales = N * K // (16 if case["scaling"] == "nv16" else 32)
        return {"bytes": N * K // 2 + scales + x * T * K + y * T * N, "flops": 2 * T * N * K}
    H, D = case["H"], case["D"]
    token = 2 * H * (D // 2 + D // 16)
    if op != "attend":
        o = 4 if case["out"] == "f32" else 2
        written = 4 * H * D if op == "append" else 0
        return {"bytes": case["T"] * (written + token + 2 * o * H * D + 8), "flops": case["T"] * 2 * H * D}
    mean = 0.5 if case["ragged"] else 1.0
    tokens = mean * case["B"] * case["L"]
    rows = case["B"] * case["S"] * (mean if case["S"] > 1 else 1.0)
    return {"bytes": tokens * token + rows * H * case["G"] * (4 * D + 4),
            "flops": 4 * tokens * rows / case["B"] * H * case["G"] * D}


# ---------------------------------------------------------------- the definitions in 64 bits


def _hadamard64():
    """The transform as a matrix: entry (i, j) is the sign d_j times (-1) to the number of common bits of i and j, / 4."""
    d = _signs(_SEED)
    h = [[d[j] * (-1) ** bin(i & j).count("1") / 4 for j in range(16)] for i in range(16)]
    return torch.tensor(h, dtype=torch.float64, device=_DEV)


def _along(x, matrix):
    return torch.matmul(x.reshape(*x.shape[:-1], -1, 16), matrix.T).reshape(x.shape)


def _pow2(e):
    """2^e in 64 bits, from its encoding."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _decode64(codes, scales, grid, scaling):
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int16)
    if grid == "int4":
        v = torch.where(n >= 8, n - 16, n).double()
    else:
        m = n & 7
        v = m.double() / 2
        if grid == "e2m1":
            v = torch.where(m < 4, v, torch.where(m < 6, m - 2, 2 * m - 8).double())
        v = torch.where(n >= 8, -v, v)
    b = scales.to(torch.int64)
    if scaling == "nv16":
        d = torch.where(b >> 3 > 0, (8 + (b & 7)).double() * _pow2((b >> 3) - 10), (b & 7).double() / 512)
    else:
        d = _pow2(b - 127)
    return (v.view(*d.shape, -1) * d[..., None]).flatten(-2)


def _kept64(x, case, ts):
    """Values that rows [T][H][D] of keys or values have in the cache: the definition's steps, which are those of
    32-bit numbers, each computed in 64 bits and rounded to 32."""
    def r(v):
        return v.float().double()

    x = x.double().view(x.shape[0], case["H"], -1, 16)
    if case["rht"]:
        x = x * torch.tensor(_signs(_SEED), dtype=torch.float64, device=_DEV)
        for h in (1, 2, 4, 8):
            j = torch.arange(16, device=_DEV)
            x = r(x[..., j & ~h] + torch.where((j & h) > 0, -1.0, 1.0).double() * x[..., j | h])
        x = x / 4
    q, ts = _TOP[case["grid"]], ts.double()[:, None]
    s = r(x.abs().amax(-1) / r(q * ts)).clamp(max=448.0)
    step = _pow2(torch.clamp(torch.frexp(s)[1] - 1, min=-6) - 3)
    d = r(torch.round(s / step) * step * ts)
    inv = torch.where(d > 0, r(1 / torch.where(d > 0, d, 1.0)), 0.0)
    y = r(x * inv[..., None])
    if case["grid"] == "e2m1":
        step = _pow2(torch.clamp(torch.frexp(y.abs().clamp(max=6.0))[1] - 2, min=-1))
    else:
        step = 0.5 if case["grid"] == "e1m2" else 1.0
    return ((torch.round(y / step) * step).clamp(-q, q) * d[..., None]).flatten(2)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    T64 = _hadamard64()
    if op == "matvec":
        codes, scales, ts = s["w"]
        x = s["x"].double()
        if case["rht"]:
            x = _along(x, T64)
        y, step = [], max(1, (1 << 26) // case["K"])
        for n in range(0, case["N"], step):
            w = _decode64(codes[n:n + step], scales[n:n + step], case["grid"], case["scaling"])
            y.append(torch.matmul(x, w.T.contiguous()) * ts.double())
        return {"y": torch.cat(y, 1)}
    cache, grid = s["cache"], case["grid"]
    kt, vt = _head_scales(cache, "k_ts", case), _head_scales(cache, "v_ts", case)
    H, D, P = case["H"], case["D"], case["P"]
    if op != "attend":
        out = {}
        for name, t in (("k", kt), ("v", vt)):
            if op == "append":
                x = _kept64(s[name], case, t)
            else:
                slot = s["slots"]
                page, at = slot // P, slot % P
                c, b = cache[name + "_codes"], cache[name + "_scales"]
                if name == "v":  # as the keys' layout
                    c = c.transpose(3, 4).reshape(c.shape[0], H, P, D // 2)
                    b = b.transpose(3, 4).reshape(b.shape[0], H, P, D // 16)
                x = _decode64(c[page, :, at], b[page, :, at], grid, "nv16") * t.double()[:, None]
            out[name] = (_along(x, T64.T) if case["rht"] else x).flatten(1)
        return out
    G, rows = case["G"], s["starts"][-1]
    out = torch.zeros(rows, H, G, D, dtype=torch.float64, device=_DEV)
    lse = torch.full((rows, H, G), -math.inf, dtype=torch.float64, device=_DEV)
    q = s["q"].double().view(rows, H, G, D)
    if case["rht"]:
        q = _along(q, T64)
    for b in range(case["B"]):
        L, n, r0 = s["L"][b], s["S"][b], s["starts"][b]
        if n == 0:
            continue
        pages = s["table"][b, :-(-L // P)].long()
        seen = torch.ones(n, L, dtype=torch.bool, device=_DEV)
        for i in range(n):
            bits = (1 << (i + 1)) - 1 if s["mask"] is None else int(s["mask"][r0 + i])
            seen[i, L - n:] = torch.tensor([bool((bits >> j) & 1) for j in range(n)], device=_DEV)
        for h in range(H):
            k = _decode64(cache["k_codes"][pages, h].flatten(0, 1)[:L], cache["k_scales"][pages, h].flatten(0, 1)[:L],
                          grid, "nv16") * kt[h].double()
            v = _decode64(cache["v_codes"][pages, h].transpose(2, 3).flatten(0, 2)[:L],
                          cache["v_scales"][pages, h].transpose(2, 3).flatten(0, 2)[:L], grid, "nv16") * vt[h].double()
            a = torch.matmul(q[r0:r0 + n, h].reshape(n * G, D), k.T.contiguous()).view(n, G, L) / math.sqrt(D)
            a = a.masked_fill(~seen[:, None], -math.inf)
            lse[r0:r0 + n, h] = torch.logsumexp(a, -1)
            out[r0:r0 + n, h] = torch.matmul(torch.softmax(a, -1).view(n * G, L), v).view(n, G, D)
    if case["rht"]:
        out = _along(out, T64.T)
    return {"out": out.flatten(1), "lse": lse.flatten(1)}
