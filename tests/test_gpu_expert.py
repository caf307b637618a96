"""Sort, dispatch and combine of expert rows against a plain implementation in
64 bits, at the sizes, masks and layouts where they can go wrong."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8  # one rounding to bf16: at most half an ulp, 2^-9 relative; stored error bound doubled below


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp4_quantization_amd as F
    return torch, F


def plain_sort(ids, E, align, total):
    flat = np.asarray(ids).reshape(-1)
    offsets = np.zeros(E + 2, np.int64)
    row_of_slot = np.full(flat.size, -1, np.int32)
    slot_of_row = np.full(total, -1, np.int32)
    at = 0
    for e in range(E):
        offsets[e] = at
        mine = np.nonzero(flat == e)[0]
        row_of_slot[mine] = at + np.arange(mine.size)
        slot_of_row[at:at + mine.size] = mine
        at += -(-mine.size // align) * align
    offsets[E], offsets[E + 1] = at, total
    return offsets, row_of_slot.reshape(np.asarray(ids).shape), slot_of_row


def gpu_sort(env, ids, E, align, total=None, stream=None):
    torch, F = env
    d = ids if isinstance(ids, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(ids, np.int32)).cuda()
    T, k = d.shape
    total = F.ufp4_expert_rows(T, k, E, align) if total is None else total
    off = torch.full((E + 2,), -7, dtype=torch.int64, device="cuda")
    ros = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    sor = torch.full((total,), -7, dtype=torch.int32, device="cuda")
    F.ufp4_expert_sort(d, E, align, off, ros, sor, stream)
    return off, ros, sor


# (tokens, slots, experts, align, share of dropped slots)
SORTS = [(0, 2, 4, 1, 0), (1, 1, 1, 1, 0), (1, 8, 64, 16, 0), (3, 5, 7, 1, 0.4), (64, 1, 64, 32, 0), (511, 8, 64, 16, 0),
         (512, 8, 64, 16, 0), (4097, 1, 3, 1, 0.1), (700, 7, 1023, 16, 0.05), (2000, 5, 1023, 4096, 0), (1500, 8, 40, 16, 1.0),
         (9000, 8, 64, 16, 0), (30011, 3, 33, 1, 0.2), (100, 1024, 9, 16, 0)]


@pytest.mark.parametrize("T,k,E,align,drop", SORTS)
def test_sort(env, T, k, E, align, drop):
    torch, F = env
    rng = np.random.default_rng(T + 31 * k + E)
    # popular experts, and ids outside [0, E) on both sides for dropped slots
    ids = np.minimum((rng.random((T, k)) ** 2 * E).astype(np.int32), E - 1)
    bad = rng.random((T, k)) < drop
    ids[bad] = rng.choice(np.array([-1, E, -2**31, 2**31 - 1], np.int64), bad.sum()).astype(np.int32)
    off, ros, sor = gpu_sort(env, ids, E, align)
    want = plain_sort(np.where((ids >= 0) & (ids < E), ids, -1), E, align, sor.numel())
    for got, w, name in zip((off, ros, sor), want, ("offsets", "row_of_slot", "slot_of_row")):
        assert np.array_equal(got.cpu().numpy(), w), name


def test_sort_strided_ids_and_spare_rows(env):
    torch, F = env
    rng = np.random.default_rng(5)
    wide = torch.from_numpy(rng.integers(0, 12, size=(900, 11)).astype(np.int32)).cuda()
    ids = wide[:, 2:8]
    off, ros, sor = gpu_sort(env, ids, 12, 16, total=F.ufp4_expert_rows(900, 6, 12, 16) + 333)
    want = plain_sort(ids.cpu().numpy(), 12, 16, sor.numel())
    for got, w in zip((off, ros, sor), want):
        assert np.array_equal(got.cpu().numpy(), w)


def test_sorted_offsets_feed_the_grouped_quantizer(env):
    torch, F = env
    g = torch.Generator(device="cuda").manual_seed(1)
    T, k, E, D = 70, 3, 9, 64
    ids = torch.randint(-1, E, (T, k), device="cuda", generator=g, dtype=torch.int32)
    off, ros, sor = gpu_sort(env, ids, E, 16)
    R = sor.numel()
    x = torch.randn(T, D, device="cuda", generator=g).to(torch.bfloat16)
    rows = torch.empty(R, D, dtype=torch.bfloat16, device="cuda")
    F.ufp4_expert_dispatch(x, ros, sor, rows)
    row, col = F.alloc_layout(R, D, 0, E + 1), F.alloc_layout(D, R, 0, E + 1)
    ws = F.Workspace(R, D, E + 1)
    F.ufp4_quantize_grouped(rows, off, R, F.config(), row, col, ws)
    assert ws.status() == 0
    lo, hi = int(off[2]), int(off[3])
    one = F.alloc_layout(hi - lo, D, 0)
    F.ufp4_quantize(rows[lo:hi].contiguous(), F.config(), one, F.Workspace(max(hi - lo, 16), D))
    assert torch.equal(row.codes[lo:hi], one.codes) and torch.equal(row.scales[lo:hi], one.scales)


def routing(env, T, k, E, align, drop, seed):
    torch, F = env
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, E, size=(T, k)).astype(np.int32)
    ids[rng.random((T, k)) < drop] = -1
    if T > 2:
        ids[T // 2] = -1  # a token without experts
    off, ros, sor = gpu_sort(env, ids, E, align)
    return rng, ros, sor


def matrix(torch, rng, rows, cols, dtype, pad=0, shift=0):
    """rows x cols values with `pad` spare columns, starting `shift` elements
    into its allocation."""
    t = torch.from_numpy(rng.standard_normal(rows * (cols + pad) + shift).astype(np.float32)).to(dtype).cuda()
    return t[shift:].view(rows, cols + pad)[:, :cols]


COLS = [1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 12, 14, 64, 515, 1024, 1025, 1365, 4096]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1), (8, 8)])
def test_dispatch(env, cols, pad, shift):
    torch, F = env
    T, k, E = 37, 3, 5
    rng, ros, sor = routing(env, T, k, E, 16, 0.2, cols)
    x = matrix(torch, rng, T, cols, torch.bfloat16, pad, shift)
    R = sor.numel()
    store = torch.full((R * (cols + pad) + shift,), 3.0, dtype=torch.bfloat16, device="cuda")
    out = store[shift:].view(R, cols + pad)[:, :cols]
    F.ufp4_expert_dispatch(x, ros, sor, out)
    want = torch.where((sor >= 0)[:, None], x[(sor.clamp(min=0) // k).long()], 0)
    assert torch.equal(out, want)
    # columns between the rows stay as they were
    if pad:
        assert (store[shift:].view(R, cols + pad)[:, cols:] == 3.0).all() and (store[:shift] == 3.0).all()


def test_dispatch_of_no_tokens_zeroes_the_rows(env):
    torch, F = env
    ros = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    sor = torch.full((40,), -1, dtype=torch.int32, device="cuda")
    out = torch.ones((40, 24), dtype=torch.bfloat16, device="cuda")
    F.ufp4_expert_dispatch(torch.empty((0, 24), dtype=torch.bfloat16, device="cuda"), ros, sor, out)
    assert (out == 0).all()


def test_dispatch_passes_every_bit_pattern(env):
    torch, F = env
    x = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(256, 256).cuda()
    ids = (torch.arange(256, dtype=torch.int32) % 7)[:, None].cuda().contiguous()
    off, ros, sor = gpu_sort(env, ids, 7, 1)
    out = torch.empty_like(x)
    F.ufp4_expert_dispatch(x, ros, sor, out)
    assert torch.equal(out, x[sor.long()])


@pytest.mark.parametrize("zt,ot", [("bfloat16", "bfloat16"), ("bfloat16", "float32"), ("float32", "bfloat16"), ("float32", "float32")])
@pytest.mark.parametrize("T,k,cols,pad,shift", [(1, 8, 4096, 0, 0), (29, 3, 9, 3, 1), (130, 2, 1365, 1, 3), (64, 13, 520, 0, 0),
                                                (5, 1, 1, 0, 0)])
def test_combine(env, zt, ot, T, k, cols, pad, shift):
    torch, F = env
    rng, ros, sor = routing(env, T, k, 6, 16, 0.25, T + cols)
    R = sor.numel()
    z = matrix(torch, rng, R, cols, getattr(torch, zt), pad, shift)
    # what nobody may read: padding rows, and weights of dropped slots
    z[sor < 0] = float("nan")
    w = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    w[ros < 0] = float("inf")
    out = torch.empty((T, cols), dtype=getattr(torch, ot), device="cuda")
    for weights in (w, None):
        F.ufp4_expert_combine(z, ros, weights, out)
        zz, rr = z.double().cpu(), ros.cpu().long()
        live = (rr >= 0)[..., None]
        terms = torch.where(live, zz[rr.clamp(min=0)] * (w.double().cpu()[..., None] if weights is not None else 1.0), 0.0)
        want, size = terms.sum(1), terms.abs().sum(1)
        # fp32 sum of k terms, one fused rounding each, then the output's own
        tol = k * 2.0 ** -24 * size + (2.0 ** -8 if ot == "bfloat16" else 0.0) * want.abs() + 1e-38
        assert ((out.double().cpu() - want).abs() <= tol).all()
        assert (out[(ros < 0).all(1)] == 0).all()


@pytest.mark.parametrize("dt,zt", [("bfloat16", "bfloat16"), ("float32", "bfloat16"), ("bfloat16", "float32"), ("float32", "float32")])
@pytest.mark.parametrize("T,k,cols,pad,shift", [(1, 8, 4096, 0, 0), (29, 3, 9, 3, 1), (61, 2, 1365, 1, 3), (33, 13, 520, 0, 0),
                                                (9, 9, 1032, 0, 0), (5, 1, 1, 0, 0)])
def test_combine_backward(env, dt, zt, T, k, cols, pad, shift):
    torch, F = env
    rng, ros, sor = routing(env, T, k, 6, 16, 0.25, 7 * T + cols)
    R = sor.numel()
    z = matrix(torch, rng, R, cols, getattr(torch, zt), pad, shift)
    z[sor < 0] = float("nan")
    dout = matrix(torch, rng, T, cols, getattr(torch, dt), pad, shift)
    w = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    w[ros < 0] = float("nan")
    dz = torch.full((R, cols + pad), 5.0, dtype=z.dtype, device="cuda")[:, :cols]
    dw = torch.full((T, k), 5.0, device="cuda")
    F.ufp4_expert_combine_backward(dout, z, ros, sor, w, dz, dw)
    s = sor.cpu().long()
    d64, w64 = dout.double().cpu(), w.double().cpu()
    want = torch.where((s >= 0)[:, None], w64.reshape(-1)[s.clamp(min=0)][:, None] * d64[s.clamp(min=0) // k], 0.0)
    tol = want.abs() * (2.0 ** -8 if zt == "bfloat16" else 2.0 ** -23) + 1e-38
    assert ((dz.double().cpu() - want).abs() <= tol).all()
    r = ros.cpu().long()
    terms = torch.where((r >= 0)[..., None], d64[:, None, :] * z.double().cpu()[r.clamp(min=0)], 0.0)
    assert ((dw.double().cpu() - terms.sum(-1)).abs() <= cols * 2.0 ** -24 * terms.abs().sum(-1) + 1e-38).all()
    # each output alone, and the same bits again
    dz2, dw2 = torch.empty_like(dz), torch.empty_like(dw)
    F.ufp4_expert_combine_backward(dout, None, ros, sor, w, dz2, None)
    F.ufp4_expert_combine_backward(dout, z, ros, sor, None, None, dw2)
    assert torch.equal(dz, dz2) and torch.equal(dw, dw2)
    F.ufp4_expert_combine_backward(dout, None, ros, sor, None, dz2, None)
    plain = torch.where((s >= 0)[:, None], d64[s.clamp(min=0) // k], 0.0)
    assert ((dz2.double().cpu() - plain).abs() <= plain.abs() * 2.0 ** -8).all()


def test_combine_gradient_against_differences(env):
    """The loss sum(combine(z, w) * dout) is linear in z and in w: its
    differences along any direction are the gradients' products with it."""
    torch, F = env
    T, k, cols = 12, 4, 96
    rng, ros, sor = routing(env, T, k, 5, 16, 0.2, 3)
    R = sor.numel()
    z, dout = matrix(torch, rng, R, cols, torch.float32), matrix(torch, rng, T, cols, torch.float32)
    w = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    dz, dw = torch.empty_like(z), torch.empty_like(w)
    F.ufp4_expert_combine_backward(dout, z, ros, sor, w, dz, dw)

    def loss(zz, ww):
        y = torch.empty((T, cols), device="cuda")
        F.ufp4_expert_combine(zz, ros, ww, y)
        return float((y.double() * dout.double()).sum())

    vz, vw = torch.randn_like(z), torch.randn_like(w)
    h = 0.5
    for got, num in (((dz.double() * vz.double()).sum(), (loss(z + h * vz, w) - loss(z - h * vz, w)) / (2 * h)),
                     ((dw.double() * vw.double()).sum(), (loss(z, w + h * vw) - loss(z, w - h * vw)) / (2 * h))):
        # fp32 rounding of about 5000 terms of size one
        assert abs(float(got) - num) < 1e-3


def test_dispatch_gradient_is_the_unweighted_combine(env):
    torch, F = env
    T, k, cols = 23, 3, 130
    rng, ros, sor = routing(env, T, k, 5, 16, 0.2, 4)
    x, drows = matrix(torch, rng, T, cols, torch.bfloat16), matrix(torch, rng, sor.numel(), cols, torch.float32)
    rows, dx = torch.empty((sor.numel(), cols), dtype=torch.bfloat16, device="cuda"), torch.empty((T, cols), device="cuda")
    F.ufp4_expert_dispatch(x, ros, sor, rows)
    F.ufp4_expert_combine(drows, ros, None, dx)
    a, b = (rows.double() * drows.double()).sum(), (x.double() * dx.double()).sum()
    assert abs(float(a - b)) < 1e-3


def test_on_another_stream(env):
    torch, F = env
    T, k, E, cols = 300, 4, 16, 512
    rng = np.random.default_rng(9)
    ids = torch.from_numpy(rng.integers(0, E, size=(T, k)).astype(np.int32)).cuda()
    x = matrix(torch, rng, T, cols, torch.bfloat16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    off, ros, sor = gpu_sort(env, ids, E, 16, stream=s)
    # (the fills before the sort ran on the current stream)
    torch.cuda.synchronize()
    off, ros, sor = gpu_sort(env, ids, E, 16)
    torch.cuda.synchronize()
    rows, y = torch.empty((sor.numel(), cols), dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
    torch.cuda.synchronize()
    F.ufp4_expert_dispatch(x, ros, sor, rows, stream=s)
    w = torch.full((T, k), 0.25, device="cuda")
    torch.cuda.synchronize()
    F.ufp4_expert_combine(rows, ros, w, y, stream=s)
    s.synchronize()
    assert torch.equal(y, x)


def test_rows_outside_the_matrix_count_as_dropped(env):
    torch, F = env
    ros = torch.tensor([[0, 9], [-5, 1]], dtype=torch.int32, device="cuda")
    z = torch.ones((2, 16), device="cuda")
    y = torch.empty((2, 16), device="cuda")
    F.ufp4_expert_combine(z, ros, None, y)
    assert (y == 1).all()


def test_wrapper_refusals(env):
    torch, F = env
    i32 = dict(dtype=torch.int32, device="cuda")
    ids = torch.zeros((4, 2), **i32)
    off, ros, sor = gpu_sort(env, ids, 3, 16)
    x = torch.zeros((4, 8), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((sor.numel(), 8), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        F.ufp4_expert_sort(ids.long(), 3, 16, off, ros, sor)
    with pytest.raises(ValueError):
        F.ufp4_expert_sort(ids, 4, 16, off, ros, sor)
    with pytest.raises(F.Ufp4Error):
        F.ufp4_expert_sort(ids, 3, 16, off, ros, sor[:8].contiguous())
    with pytest.raises(ValueError):
        F.ufp4_expert_dispatch(x[:3], ros, sor, out)
    with pytest.raises(ValueError):
        F.ufp4_expert_dispatch(x, ros, sor, out[:, :7])
    with pytest.raises(TypeError):
        F.ufp4_expert_dispatch(x.float(), ros, sor, out)
    with pytest.raises(ValueError):
        F.ufp4_expert_dispatch(x.t(), ros, sor, out)
    with pytest.raises(TypeError):
        F.ufp4_expert_combine(out, ros, torch.zeros((4, 2), dtype=torch.float64, device="cuda"), x)
    with pytest.raises(ValueError):
        F.ufp4_expert_combine_backward(x, None, ros, sor, None, None, torch.zeros((4, 2), device="cuda"))


def test_large_calls(env):
    """Calls that move more than the last-level cache holds take other loads
    and stores: the same results as their parts, which do not."""
    torch, F = env
    rng = np.random.default_rng(12)
    T, k, E, cols = 5000, 8, 24, 4104
    ids = torch.from_numpy(rng.integers(-1, E, size=(T, k)).astype(np.int32)).cuda()
    off, ros, sor = gpu_sort(env, ids, E, 16)
    R = sor.numel()
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, cols, device="cuda", generator=g).to(torch.bfloat16)
    w = torch.rand(T, k, device="cuda", generator=g)
    want = torch.where((sor >= 0)[:, None], x[(sor.clamp(min=0) // k).long()], 0)
    rows = torch.full((R, cols), 3.0, dtype=torch.bfloat16, device="cuda")
    assert (T + R) * cols * 2 > 256 << 20
    F.ufp4_expert_dispatch(x, ros, sor, rows)
    assert torch.equal(rows, want)
    c = F.alloc_checkpoint(T, cols, F.CKPT_E4M3)
    F.ufp4_checkpoint_save(x, c)
    kept = torch.empty_like(x)
    F.ufp4_checkpoint_load(c, kept)
    F.ufp4_expert_dispatch_checkpoint(c, ros, sor, rows)
    assert torch.equal(rows, torch.where((sor >= 0)[:, None], kept[(sor.clamp(min=0) // k).long()], 0))
    F.ufp4_expert_dispatch(x, ros, sor, rows)
    for dtype in (torch.bfloat16, torch.float32):
        z = rows.to(dtype) * 0.5
        y, part = torch.empty((T, cols), dtype=dtype, device="cuda"), torch.empty((500, cols), dtype=dtype, device="cuda")
        F.ufp4_expert_combine(z, ros, w, y)
        for t in range(0, T, 500):
            F.ufp4_expert_combine(z, ros[t:t + 500], w[t:t + 500], part)
            assert torch.equal(part, y[t:t + 500])
        dz, dw = torch.empty_like(z), torch.empty_like(w)
        F.ufp4_expert_combine_backward(x, z, ros, sor, w, dz, dw)
        # columns of dz on their own; dw against 64 bits
        small = torch.empty((R, 600), dtype=dtype, device="cuda")
        for col in (0, 1000, cols - 600):
            F.ufp4_expert_combine_backward(x[:, col:col + 600], None, ros, sor, w, small, None)
            assert torch.equal(small, dz[:, col:col + 600])
        for t in range(0, T, 1000):
            r = ros[t:t + 1000].long()
            terms = x[t:t + 1000, None, :].double() * z[r.clamp(min=0)].double()
            terms = torch.where((r >= 0)[..., None], terms, 0.0)
            assert ((dw[t:t + 1000].double() - terms.sum(-1)).abs() <= cols * 2.0 ** -24 * terms.abs().sum(-1)).all()
