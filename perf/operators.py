"""Cases and plain forms of the expert-layer operators: routing rows to experts and back, 8-bit activation
checkpoints with the gated activation that uses them, and the experts' products of 4-bit operands.

``run`` computes one pass through an operator, with elementary torch operations in 32 bits (``own`` false) or with
the library's entry points (``own`` true); ``exact`` gives the same outputs from the definitions in 64 bits.

Symbols: T tokens, k slots (experts chosen) a token, E experts, D model width, F width of an expert's hidden layer, R rows
in expert order.  The widths and the routing (8192 tokens, 8 of 64 experts, width 4096) are those of the grouped
quantization workload; 2048 is the width of the activation and weight workloads.
"""
import math

import torch

own = False

# ---------------------------------------------------------------- cases


def listed():
    return [
        # one decoded token: its row to the 8 experts it chose (latency)
        {"name": "dispatch_token", "op": "dispatch", "T": 1, "k": 8, "E": 64, "D": 4096, "align": 1, "drop": 0.0},
        # a training step's tokens to their experts, segments padded to the quantizer's block
        {"name": "dispatch_train", "op": "dispatch", "T": 8192, "k": 8, "E": 64, "D": 4096, "align": 16, "drop": 0.0},
        # the backward pass dispatches the layer input again, from its 8-bit checkpoint; odd width, dropped slots
        {"name": "redispatch_odd", "op": "redispatch", "T": 3001, "k": 4, "E": 40, "D": 1365, "align": 16, "drop": 0.05,
         "format": "e4m3"},
        # the experts' outputs back to their tokens with the routing weights; ragged sizes, dropped slots
        {"name": "combine_ragged", "op": "combine", "T": 5119, "k": 6, "E": 48, "D": 2050, "align": 1, "drop": 0.1,
         "type": "bf16"},
        # gradient of the combination in a training step
        {"name": "combine_grad_train", "op": "combine_grad", "T": 8192, "k": 8, "E": 64, "D": 4096, "align": 16,
         "drop": 0.0, "type": "bf16"},
        # one decoded token's 8 rows through the gated activation: nothing is kept
        {"name": "gated_token", "op": "gated", "R": 8, "F": 2048, "act": "silu"},
        # a training step's gated activation, forward with its checkpoint and backward from it
        {"name": "gated_train", "op": "gated_step", "R": 65536, "F": 2048, "act": "silu", "format": "int8"},
        # the same at an odd width and row count
        {"name": "gated_odd", "op": "gated_step", "R": 4099, "F": 1365, "act": "gelu_tanh", "format": "e4m3"},
        # 16 tokens decoded together: 128 rows over 64 experts, bound by reading the experts' weights
        {"name": "experts_decode", "op": "product", "R": 128, "E": 64, "N": 4096, "K": 4096, "grid": "e1m2",
         "type": "bf16"},
        # forward product of a training step (gate and up projections side by side)
        {"name": "experts_forward", "op": "product", "R": 65536, "E": 64, "N": 4096, "K": 4096, "grid": "e1m2",
         "type": "bf16"},
        # input gradient: weights in their column-wise layout; ragged sizes
        {"name": "experts_dx_ragged", "op": "product_dx", "R": 9001, "E": 24, "N": 1000, "K": 2080, "grid": "int4",
         "type": "bf16"},
        # weight gradients of every expert, reduced over its rows
        {"name": "experts_dw", "op": "product_dw", "R": 65536, "E": 64, "M": 4096, "N": 2048, "grid": "e1m2",
         "type": "f32"},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["dispatch", "redispatch", "combine", "combine_grad", "gated", "gated_step", "product", "product_dx",
                     "product_dw"])
    if op in ("dispatch", "redispatch", "combine", "combine_grad"):
        E = _spread(rng, 1, 64)
        case = {"op": op, "T": _spread(rng, 1, 8192), "k": rng.randint(1, min(8, E)), "E": E, "D": _spread(rng, 64, 4096),
                "align": rng.choice([1, 16, 32]), "drop": rng.choice([0.0, 0.05, 0.5])}
        if op == "redispatch":
            case["format"] = rng.choice(["int8", "e4m3"])
        elif op != "dispatch":
            case["type"] = rng.choice(["bf16", "f32"])
        return case
    if op in ("gated", "gated_step"):
        case = {"op": op, "R": _spread(rng, 1, 65536), "F": _spread(rng, 16, 2048), "act": rng.choice(["silu", "gelu_tanh"])}
        if op == "gated_step":
            case["format"] = rng.choice(["int8", "e4m3"])
        return case
    case = {"op": op, "R": _spread(rng, 1, 65536), "E": _spread(rng, 1, 64), "N": _spread(rng, 16, 2048 if op == "product_dw" else 4096)}
    if op == "product_dw":
        case["M"] = _spread(rng, 16, 4096)
    else:
        case["K"] = 32 * _spread(rng, 1, 128)
    case["grid"] = rng.choice(["e1m2", "int4", "e2m1"])
    case["type"] = rng.choice(["bf16", "f32"])
    return case


# ---------------------------------------------------------------- inputs

_ACTS = {"silu": 0, "gelu_tanh": 1}
_FORMATS = {"int8": 0, "e4m3": 1}
_GRIDS = {"e1m2": 0, "int4": 1, "e2m1": 2}
_MAGNITUDES = {"e1m2": [0, 0.5, 1, 1.5, 2, 2.5, 3, 3.5], "int4": [0, 1, 2, 3, 4, 5, 6, 7], "e2m1": [0, 0.5, 1, 1.5, 2, 3, 4, 6]}
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_DEV = "cuda"


def _capacity(slots, experts, align):
    """Rows in expert order when every segment is padded to a multiple of `align`."""
    return -(-(slots + min(experts, slots) * (align - 1)) // align) * align


def _activation(rows, cols, gen):
    """Rows with a mean for each channel and a few channels far larger than the others."""
    x = torch.randn(rows, cols, device=_DEV, generator=gen)
    x += torch.randn(cols, device=_DEV, generator=gen) * 0.7
    x *= torch.where(torch.rand(cols, device=_DEV, generator=gen) < 0.004, 50.0, 1.0)
    return x


def _routing(case, gen):
    """Expert ids and weights of every token's slots (some experts are chosen more than others)."""
    T, k, E = case["T"], case["k"], case["E"]
    scores = torch.randn(T, E, device=_DEV, generator=gen) + 0.3 * torch.randn(E, device=_DEV, generator=gen)
    top, ids = torch.topk(scores, k, dim=1)
    ids = torch.where(torch.rand(T, k, device=_DEV, generator=gen) < case["drop"], -1, ids)
    return ids.to(torch.int32).contiguous(), torch.softmax(top, dim=1).contiguous()


def _rows_of(ids, E, align, R):
    """(offsets, row_of_slot, slot_of_row) of expert ids: rows in expert order, slots of one expert in their own order,
    segments padded to a multiple of `align`, rows past the last segment left empty."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    starts = torch.cumsum(counts, 0) - counts
    padded = (counts[:E] + align - 1) // align * align
    offsets = torch.zeros(E + 2, dtype=torch.int64, device=ids.device)
    offsets[1:E + 1] = torch.cumsum(padded, 0)
    offsets[E + 1] = R
    order = torch.argsort(key, stable=True)
    of = key[order]
    row = offsets[of] + torch.arange(n, device=ids.device) - starts[of]
    row = torch.where(of < E, row, -1)
    row_of_slot = torch.empty(n, dtype=torch.int64, device=ids.device)
    row_of_slot[order] = row
    # dropped slots are written to one row past the end
    slot_of_row = torch.full((R + 1,), -1, dtype=torch.int64, device=ids.device)
    slot_of_row[torch.where(row >= 0, row, R)] = order
    return offsets, row_of_slot.to(torch.int32).view(ids.shape), slot_of_row[:R].to(torch.int32)


def _block_max(x, block):
    """Largest magnitude of each block of `block` values along the rows (the last one may be short)."""
    pad = -x.shape[-1] % block
    return torch.nn.functional.pad(x.abs(), (0, pad)).view(*x.shape[:-1], -1, block).amax(-1)


def _checkpoint(x, fmt):
    """(codes, scales) of the 8-bit checkpoint of a matrix of bf16 values."""
    top = 127.0 if fmt == "int8" else 448.0
    # divided by a tensor: torch multiplies by the reciprocal of a plain number, which rounds twice
    bits = (_block_max(x.float(), 32) / torch.tensor(top, device=x.device)).view(torch.int32)
    s = (((bits + 0xFFFF) >> 16) << 16).view(torch.float32).clamp(min=2.0 ** -100)
    y = x.float() / s.repeat_interleave(32, -1)[..., :x.shape[-1]]
    codes = torch.round(y).to(torch.int8).view(torch.uint8) if fmt == "int8" else y.to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, s.to(torch.bfloat16)


def _checkpoint_values(codes, scales, fmt):
    v = codes.view(torch.int8).float() if fmt == "int8" else codes.view(torch.float8_e4m3fn).float()
    return v * scales.float().repeat_interleave(32, -1)[..., :v.shape[-1]]


def _quantized(x, grid, ts):
    """(codes, scales) of a float matrix in blocks of 16 along its rows, under the tensor scale `ts`."""
    table = torch.tensor(_MAGNITUDES[grid], device=x.device)
    scale = (_block_max(x, 16) / (float(table[-1]) * ts)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = scale.float().repeat_interleave(16, -1) * ts
    y = torch.where(d > 0, x / d, torch.zeros_like(x))
    index = torch.bucketize(y.abs(), (table[1:] + table[:-1]) / 2)
    if grid == "int4":
        code = torch.where(y < 0, -index, index) & 15
    else:
        code = torch.where((y < 0) & (index > 0), index + 8, index)
    code = code.to(torch.uint8)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), scale.view(torch.uint8)


def _operand(lines, segments, length, grid, gen, spread):
    """A quantized matrix of `lines` lines, `segments` pieces of `length` values side by side in each, with one tensor
    scale a piece; made piece by piece.  Returns codes, scales and the pieces' tensor scales."""
    codes = torch.empty(lines, segments * length // 2, dtype=torch.uint8, device=_DEV)
    scales = torch.empty(lines, segments * length // 16, dtype=torch.uint8, device=_DEV)
    ts = torch.empty(segments, device=_DEV)
    for e in range(segments):
        x = torch.randn(lines, length, device=_DEV, generator=gen) * spread
        t = float(x.abs().max()) / (_MAGNITUDES[grid][-1] * 448.0) if x.numel() else 1.0
        c, s = _quantized(x, grid, t)
        codes[:, e * length // 2:(e + 1) * length // 2] = c
        scales[:, e * length // 16:(e + 1) * length // 16] = s
        ts[e] = t
    return codes, scales, ts


def _segments(case, gen):
    """Offsets of ragged segments whose lengths sum to the case's rows (some may be empty)."""
    R, E = case["R"], case["E"]
    logits = 0.3 * torch.randn(E, device=_DEV, generator=gen)
    of = torch.multinomial(torch.softmax(logits, 0).expand(R, E), 1, generator=gen).view(-1)
    counts = torch.zeros(E, dtype=torch.int64, device=_DEV).scatter_add_(0, of, torch.ones_like(of))
    return torch.cat([torch.zeros(1, dtype=torch.int64, device=_DEV), torch.cumsum(counts, 0)])


def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(seed * 1000003 + 17)
    op, s = case["op"], {"case": case}
    if op in ("dispatch", "redispatch", "combine", "combine_grad"):
        T, k, E, D = case["T"], case["k"], case["E"], case["D"]
        R = _capacity(T * k, E, case["align"])
        ids, weights = _routing(case, gen)
        s["R"] = R
        if op == "dispatch":
            s["ids"], s["x"] = ids, _activation(T, D, gen).to(torch.bfloat16)
            return s
        s["offsets"], s["row_of_slot"], s["slot_of_row"] = _rows_of(ids, E, case["align"], R)
        if op == "redispatch":
            s["codes"], s["scales"] = _checkpoint(_activation(T, D, gen).to(torch.bfloat16), case["format"])
            return s
        s["weights"], s["z"] = weights, torch.randn(R, D, device=_DEV, generator=gen).to(_TYPES[case["type"]])
        if op == "combine_grad":
            s["dy"] = (1e-3 * torch.randn(T, D, device=_DEV, generator=gen)).to(torch.bfloat16)
        return s
    if op in ("gated", "gated_step"):
        R, F = case["R"], case["F"]
        s["gu"] = _activation(R, 2 * F, gen).to(torch.bfloat16)
        if op == "gated_step":
            s["dh"] = (1e-3 * torch.randn(R, F, device=_DEV, generator=gen)).to(torch.bfloat16)
        return s
    R, E, N, grid = case["R"], case["E"], case["N"], case["grid"]
    s["offsets"] = off = _segments(case, gen)
    if op == "product_dw":
        # each segment's columns are padded to the block of 16
        counts = off[1:] - off[:-1]
        starts = torch.cat([torch.zeros_like(off[:1]), torch.cumsum((counts + 15) // 16 * 16, 0)])
        P = int(starts[-1])
        s["P"] = P
        for name, lines, spread in (("a", case["M"], 1e-3), ("b", N, 1.0)):
            codes, scales, _ = _operand(lines, 1, P, grid, gen, spread)
            s[name] = (codes, scales, spread * 0.01 * (0.5 + torch.rand(E, device=_DEV, generator=gen)))
        return s
    K = case["K"]
    codes, scales, _ = _operand(R, 1, K, grid, gen, 1.0)
    s["a"] = (codes, scales, 0.01 * (0.5 + torch.rand(E, device=_DEV, generator=gen)))
    if op == "product":
        codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device=_DEV)
        scales = torch.empty(E, N, K // 16, dtype=torch.uint8, device=_DEV)
        ts = torch.empty(E, device=_DEV)
        for e in range(E):
            codes[e], scales[e], t = _operand(N, 1, K, grid, gen, 0.02)
            ts[e] = t[0]
        s["b"] = (codes.view(E * N, K // 2), scales.view(E * N, K // 16), ts)
    else:
        s["b"] = _operand(N, E, K, grid, gen, 0.02)
    return s


# ---------------------------------------------------------------- plain forms


def _values(codes, scales, grid):
    """The values of a quantized matrix, without its tensor scale."""
    m = _MAGNITUDES[grid]
    signed = m + [-v for v in m] if grid != "int4" else m + [0] + [-v for v in m[:0:-1]]
    table = torch.tensor(signed, dtype=torch.float32, device=codes.device)
    index = torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1).int()
    return table[index] * scales.view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)


def _gate(g, act):
    """sigmoid part s(g) of f(g) = g s(g), and s + g s'(g)."""
    if act == "silu":
        y, dy = g, 1.0
    else:
        g = g.clamp(-16.0, 16.0)  # beyond it s is 0 or 1 to the last bit
        c = 2.0 * math.sqrt(2.0 / math.pi)
        y, dy = c * (g + 0.044715 * g * g * g), c * (1.0 + 3 * 0.044715 * g * g)
    s = 1.0 / (1.0 + torch.exp(-y))
    return s, s + g * dy * s * (1.0 - s)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op in ("dispatch", "redispatch"):
        if op == "dispatch":
            x = s["x"].float()
            offsets, row_of_slot, slot_of_row = _rows_of(s["ids"], case["E"], case["align"], s["R"])
        else:
            x = _checkpoint_values(s["codes"], s["scales"], case["format"])
            slot_of_row = s["slot_of_row"]
        token = slot_of_row.clamp(min=0).long() // case["k"]
        rows = torch.where((slot_of_row >= 0)[:, None], x[token], 0.0).to(torch.bfloat16)
        return {"rows": rows} if op == "redispatch" else {"rows": rows, "offsets": offsets, "row_of_slot": row_of_slot,
                                                          "slot_of_row": slot_of_row}
    if op == "combine":
        row = s["row_of_slot"]
        z = s["z"].float()[row.clamp(min=0).long()]
        y = torch.where((row >= 0)[..., None], z * s["weights"][..., None], 0.0).sum(1)
        return {"y": y.to(s["z"].dtype)}
    if op == "combine_grad":
        row, slot, dy = s["row_of_slot"], s["slot_of_row"], s["dy"].float()
        w = s["weights"].reshape(-1)[slot.clamp(min=0).long()]
        dz = torch.where((slot >= 0)[:, None], w[:, None] * dy[slot.clamp(min=0).long() // case["k"]], 0.0)
        z = s["z"].float()[row.clamp(min=0).long()]
        dw = torch.where(row >= 0, (z * dy[:, None, :]).sum(-1), 0.0)
        return {"dz": dz.to(s["z"].dtype), "dweights": dw}
    if op == "gated":
        F = case["F"]
        g, u = s["gu"][:, :F].float(), s["gu"][:, F:].float()
        return {"h": (g * _gate(g, case["act"])[0] * u).to(torch.bfloat16)}
    if op == "gated_step":
        F, fmt = case["F"], case["format"]
        g, u = s["gu"][:, :F].float(), s["gu"][:, F:].float()
        h = (g * _gate(g, case["act"])[0] * u).to(torch.bfloat16)
        g = _checkpoint_values(*_checkpoint(s["gu"][:, :F], fmt), fmt)
        u = _checkpoint_values(*_checkpoint(s["gu"][:, F:], fmt), fmt)
        sig, slope = _gate(g, case["act"])
        dh = s["dh"].float()
        dgu = torch.cat([dh * u * slope, dh * g * sig], 1).to(torch.bfloat16)
        return {"h": h, "h_again": (g * sig * u).to(torch.bfloat16), "dgu": dgu}
    off, E, grid = s["offsets"], case["E"], case["grid"]
    (ac, asc, ats), (bc, bsc, bts) = s["a"], s["b"]
    a, b = _values(ac, asc, grid), _values(bc, bsc, grid)
    counts = off[1:] - off[:-1]
    t = (ats * bts)[:, None, None]
    if op == "product_dw":
        # every segment's columns side by side, zeros behind the shorter ones
        padded = (counts + 15) // 16 * 16
        start = torch.cumsum(padded, 0) - padded
        at = torch.arange(int(padded.max()), device=a.device)
        inside = at[None, :] < padded[:, None]
        at = torch.where(inside, start[:, None] + at[None, :], 0)
        a = torch.where(inside[None], a[:, at.reshape(-1)].view(-1, *at.shape), 0.0).transpose(0, 1).contiguous()
        b = torch.where(inside[None], b[:, at.reshape(-1)].view(-1, *at.shape), 0.0).transpose(0, 1).contiguous()
        return {"c": (torch.bmm(a, b.transpose(1, 2)) * t).to(_TYPES[case["type"]])}
    # every segment's rows under each other, zeros below the shorter ones
    at = torch.arange(int(counts.max()), device=a.device)
    inside = at[None, :] < counts[:, None]
    a = torch.where(inside[..., None], a[torch.where(inside, off[:-1, None] + at[None, :], 0)], 0.0)
    b = b.view(E, case["N"], case["K"]) if op == "product" else b.view(case["N"], E, case["K"]).transpose(0, 1)
    return {"c": (torch.bmm(a, b.transpose(1, 2)) * t)[inside].to(_TYPES[case["type"]])}


# ---------------------------------------------------------------- the library's entry points


def _new(shape, dtype):
    return torch.empty(shape, dtype=dtype, device=_DEV)


def _own(s):
    import fp4_quantization_amd as F

    case, op = s["case"], s["case"]["op"]
    if op in ("dispatch", "redispatch"):
        rows = _new((s["R"], case["D"]), torch.bfloat16)
        if op == "redispatch":
            kept = F.Checkpoint(s["codes"], s["scales"], _FORMATS[case["format"]])
            F.ufp4_expert_dispatch_checkpoint(kept, s["row_of_slot"], s["slot_of_row"], rows)
            return {"rows": rows}
        offsets = _new((case["E"] + 2,), torch.int64)
        row_of_slot, slot_of_row = _new(s["ids"].shape, torch.int32), _new((s["R"],), torch.int32)
        F.ufp4_expert_sort(s["ids"], case["E"], case["align"], offsets, row_of_slot, slot_of_row)
        F.ufp4_expert_dispatch(s["x"], row_of_slot, slot_of_row, rows)
        return {"rows": rows, "offsets": offsets, "row_of_slot": row_of_slot, "slot_of_row": slot_of_row}
    if op == "combine":
        y = _new((case["T"], case["D"]), s["z"].dtype)
        F.ufp4_expert_combine(s["z"], s["row_of_slot"], s["weights"], y)
        return {"y": y}
    if op == "combine_grad":
        dz, dw = _new(s["z"].shape, s["z"].dtype), _new(s["weights"].shape, torch.float32)
        F.ufp4_expert_combine_backward(s["dy"], s["z"], s["row_of_slot"], s["slot_of_row"], s["weights"], dz, dw)
        return {"dz": dz, "dweights": dw}
    if op in ("gated", "gated_step"):
        R, W, act = case["R"], case["F"], _ACTS[case["act"]]
        h = _new((R, W), torch.bfloat16)
        if op == "gated":
            F.ufp4_gated_act(s["gu"], act, h)
            return {"h": h}
        kept = F.alloc_checkpoint(R, W, _FORMATS[case["format"]], halves=2)
        F.ufp4_gated_act(s["gu"], act, h, kept)
        dgu, again = _new((R, 2 * W), torch.bfloat16), _new((R, W), torch.bfloat16)
        F.ufp4_gated_act_backward(s["dh"], kept, act, dgu, again)
        return {"h": h, "h_again": again, "dgu": dgu}
    cfg = F.config(grid=_GRIDS[case["grid"]])
    a, b = F.QTensor(*s["a"]), F.QTensor(*s["b"])
    if op == "product_dw":
        c = _new((case["E"], case["M"], case["N"]), _TYPES[case["type"]])
        F.ufp4_gemm_grouped_dw(cfg, a, b, s["offsets"], c)
        return {"c": c}
    c = _new((case["R"], case["N"]), _TYPES[case["type"]])
    F.ufp4_gemm_grouped_nt(cfg, a, b, 0 if op == "product" else 1, s["offsets"], case["K"], c)
    return {"c": c}


def run(s):
    return _own(s) if own else _plain(s)


# ---------------------------------------------------------------- work


def work(case):
    op = case["op"]
    if op in ("dispatch", "redispatch", "combine", "combine_grad"):
        n, D = case["T"] * case["k"], case["D"]
        R = _capacity(n, case["E"], case["align"])
        kept = n * (1.0 - case["drop"])
        z = 4 if case.get("type") == "f32" else 2
        if op == "dispatch":
            return {"bytes": 2 * case["T"] * D + 2 * R * D + 8 * n + 4 * R + 8 * (case["E"] + 2), "flops": 0}
        if op == "redispatch":
            return {"bytes": case["T"] * (D + 2 * -(-D // 32)) + 2 * R * D + 4 * n + 4 * R, "flops": case["T"] * D}
        if op == "combine":
            return {"bytes": kept * D * z + case["T"] * D * z + 8 * n, "flops": 2 * kept * D}
        return {"bytes": 2 * case["T"] * D + kept * D * z + R * D * z + 12 * n + 4 * R, "flops": 3 * kept * D}
    if op in ("gated", "gated_step"):
        n = case["R"] * case["F"]
        if op == "gated":
            return {"bytes": 6 * n, "flops": 8 * n}
        kept = 2 * case["R"] * (case["F"] + 2 * -(-case["F"] // 32))
        return {"bytes": 6 * n + kept + 2 * n + kept + 6 * n, "flops": 40 * n}
    c = 4 if case["type"] == "f32" else 2
    if op == "product_dw":
        return {"bytes": 0.5625 * case["R"] * (case["M"] + case["N"]) + c * case["E"] * case["M"] * case["N"],
                "flops": 2 * case["R"] * case["M"] * case["N"]}
    # experts that no row is likely to choose are not read
    used = case["E"] * (1.0 - (1.0 - 1.0 / case["E"]) ** case["R"])
    return {"bytes": 0.5625 * case["K"] * (case["R"] + used * case["N"]) + c * case["R"] * case["N"],
            "flops": 2 * case["R"] * case["N"] * case["K"]}


# ---------------------------------------------------------------- the definitions in 64 bits


def _pow2(e):
    """2^e in 64 bits, from its encoding (torch's own power of two is off by a rounding on some devices)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _decode64(codes, scales, grid):
    low, high = (codes & 15).to(torch.int64), (codes >> 4).to(torch.int64)
    n = torch.stack([low, high], 2).flatten(1)
    if grid == "int4":
        v = torch.where(n >= 8, n - 16, n).double()
    else:
        m = n & 7
        v = m.double() / 2 if grid == "e1m2" else torch.where(m < 4, m.double() / 2, torch.where(m < 6, m - 2, 2 * m - 8).double())
        v = torch.where(n >= 8, -v, v)
    b = scales.to(torch.int64)
    e, f = b >> 3, (b & 7).double()
    d = torch.where(e > 0, (1 + f / 8) * _pow2(e - 7), f * 2.0 ** -9)
    return (v.view(*d.shape, 16) * d[:, :, None]).flatten(1)


def _kept64(x, fmt):
    """A row's values after the 8-bit checkpoint: blocks of 32, scale rounded up to 8 significant bits."""
    top, n = 127.0 if fmt == "int8" else 448.0, x.shape[1]
    x = torch.cat([x, x.new_zeros(x.shape[0], -n % 32)], 1).view(x.shape[0], -1, 32)
    m, e = torch.frexp(x.abs().amax(2, keepdim=True) / top)
    s = torch.maximum(torch.ceil(m * 256) * _pow2(e - 8), torch.tensor(2.0 ** -100, dtype=torch.float64, device=x.device))
    q = x / s
    if fmt == "int8":
        q = torch.round(q)
    else:
        # step of an E4M3 number: 2^-3 of its leading power of two, 2^-9 below 2^-6
        p = _pow2(torch.clamp(torch.frexp(q)[1] - 1, min=-6) - 3)
        q = torch.round(q / p) * p
    return (q * s).flatten(1)[:, :n]


def _act64(g, act):
    if act == "silu":
        y, dy = g, torch.ones_like(g)
    else:
        c = math.sqrt(8.0 / math.pi)
        y, dy = c * (g + 0.044715 * g ** 3), c * (1 + 0.134145 * g ** 2)
    s = torch.sigmoid(y)
    return g * s, s + g * s * torch.sigmoid(-y) * dy


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("dispatch", "redispatch", "combine", "combine_grad"):
        k = case["k"]
        if op == "dispatch":
            flat = s["ids"].flatten().long()
            n = flat.numel()
            rows = torch.zeros(s["R"], case["D"], dtype=torch.float64, device=_DEV)
            at, x = 0, s["x"].double()
            for e in range(case["E"]):
                mine = torch.nonzero(flat == e).flatten()
                rows[at:at + mine.numel()] = x[mine // k]
                at += -(-mine.numel() // case["align"]) * case["align"]
            return {"rows": rows, "offsets": None, "row_of_slot": None, "slot_of_row": None}
        row = s["row_of_slot"].flatten().long()
        used = torch.nonzero(row >= 0).flatten()
        if op == "redispatch":
            if case["format"] == "int8":
                c = s["codes"].view(torch.int8).double()
            else:
                b = s["codes"].to(torch.int64)
                e, f = (b >> 3) & 15, (b & 7).double()
                c = torch.where(e > 0, (1 + f / 8) * _pow2(e - 7), f / 512) * torch.where(b >= 128, -1.0, 1.0)
            block = torch.arange(case["D"], device=_DEV) // 32
            x = c * s["scales"].double()[:, block]
            rows = torch.zeros(s["R"], case["D"], dtype=torch.float64, device=_DEV)
            rows[row[used]] = x[used // k]
            return {"rows": rows}
        w = s["weights"].double().flatten()
        if op == "combine":
            y = torch.zeros(case["T"], case["D"], dtype=torch.float64, device=_DEV)
            y.index_add_(0, used // k, w[used, None] * s["z"].double()[row[used]])
            return {"y": y}
        dy = s["dy"].double()
        dz = torch.zeros(s["R"], case["D"], dtype=torch.float64, device=_DEV)
        dz[row[used]] = w[used, None] * dy[used // k]
        dw = torch.zeros(row.numel(), dtype=torch.float64, device=_DEV)
        dw[used] = (dy[used // k] * s["z"].double()[row[used]]).sum(1)
        return {"dz": dz, "dweights": dw.view(s["weights"].shape)}
    if op in ("gated", "gated_step"):
        W = case["F"]
        gu = s["gu"].double()
        h = _act64(gu[:, :W], case["act"])[0] * gu[:, W:]
        if op == "gated":
            return {"h": h}
        g, u = _kept64(gu[:, :W], case["format"]), _kept64(gu[:, W:], case["format"])
        f, slope = _act64(g, case["act"])
        dh = s["dh"].double()
        return {"h": h, "h_again": f * u, "dgu": torch.cat([dh * u * slope, dh * f], 1)}
    off, E, grid, out = s["offsets"].tolist(), case["E"], case["grid"], []
    (ac, asc, ats), (bc, bsc, bts) = s["a"], s["b"]
    t = ats.double() * bts.double()
    if op == "product_dw":
        at = 0
        for e in range(E):
            end = at + -(-(off[e + 1] - off[e]) // 16) * 16
            a = _decode64(ac[:, at // 2:end // 2], asc[:, at // 16:end // 16], grid)
            b = _decode64(bc[:, at // 2:end // 2], bsc[:, at // 16:end // 16], grid)
            out.append(a @ b.T * t[e])
            at = end
        return {"c": torch.stack(out)}
    N, K = case["N"], case["K"]
    for e in range(E):
        a = _decode64(ac[off[e]:off[e + 1]], asc[off[e]:off[e + 1]], grid)
        if op == "product":
            b = _decode64(bc[e * N:(e + 1) * N], bsc[e * N:(e + 1) * N], grid)
        else:
            b = _decode64(bc[:, e * K // 2:(e + 1) * K // 2], bsc[:, e * K // 16:(e + 1) * K // 16], grid)
        out.append(a @ b.T * t[e])
    return {"c": torch.cat(out)}
