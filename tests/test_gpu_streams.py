"""The expert-layer operators on a stream that is not the current one: each
result right on that stream, where its inputs appear only after other work, and
nothing done on the current stream."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp4_quantization_amd as F
    return torch, F


class Side:
    """A stream with slow work ahead of what it is given next.  Tensors handed
    to `check` as `late` are zeros until that work is done, so a call that does
    not run on the stream computes from zeros."""

    def __init__(self, torch):
        self.torch, self.stream = torch, torch.cuda.Stream()
        self.busy = torch.randn(8192, 8192, device="cuda").bfloat16()

    def check(self, late, outputs, call):
        torch = self.torch
        values = [t.clone() for t in late]
        for t in late:
            t.zero_()
        for t in outputs:
            t.view(torch.uint8).fill_(0x21)
        torch.cuda.synchronize()
        with torch.cuda.stream(self.stream):
            for _ in range(12):
                torch.mm(self.busy, self.busy)
            for t, v in zip(late, values):
                t.copy_(v)
        call(self.stream)
        self.stream.synchronize()
        return [t.clone() for t in outputs]


@pytest.fixture(scope="module")
def side(env):
    return Side(env[0])


def plain_sort(ids, E, align, total):
    flat = ids.reshape(-1)
    offsets, ros, sor, at = np.zeros(E + 2, np.int64), np.full(flat.size, -1, np.int32), np.full(total, -1, np.int32), 0
    for e in range(E):
        offsets[e] = at
        mine = np.nonzero(flat == e)[0]
        ros[mine] = at + np.arange(mine.size)
        sor[at:at + mine.size] = mine
        at += -(-mine.size // align) * align
    offsets[E], offsets[E + 1] = at, total
    return offsets, ros.reshape(ids.shape), sor


# one launch, and three
@pytest.mark.parametrize("T,k,E", [(300, 4, 16), (3000, 4, 16)])
def test_sort_dispatch_combine(env, side, T, k, E):
    torch, F = env
    rng = np.random.default_rng(T)
    ids = rng.integers(-1, E, size=(T, k)).astype(np.int32)
    d = torch.from_numpy(ids).cuda()
    R, cols = F.ufp4_expert_rows(T, k, E, 16), 72
    off = torch.empty(E + 2, dtype=torch.int64, device="cuda")
    ros, sor = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda")
    got = side.check([d], [off, ros, sor], lambda s: F.ufp4_expert_sort(d, E, 16, off, ros, sor, s))
    for a, b in zip(got, plain_sort(ids, E, 16, R)):
        assert np.array_equal(a.cpu().numpy(), b)
    x = torch.from_numpy(rng.standard_normal((T, cols)).astype(np.float32)).cuda().bfloat16()
    rows = torch.empty((R, cols), dtype=torch.bfloat16, device="cuda")
    got, = side.check([x], [rows], lambda s: F.ufp4_expert_dispatch(x, ros, sor, rows, s))
    assert torch.equal(got, torch.where((sor >= 0)[:, None], x[(sor.clamp(min=0) // k).long()], 0))
    # sums of at most four bf16 values times 1/4: exact to fp32
    w, y = torch.full((T, k), 0.25, device="cuda"), torch.empty((T, cols), device="cuda")
    got, = side.check([rows, w], [y], lambda s: F.ufp4_expert_combine(rows, ros, w, y, s))
    kept = (ros >= 0).sum(1)
    assert torch.allclose(got.double(), x.double() * kept[:, None] / 4, rtol=4 * 2.0 ** -24, atol=0)
    dz, dw = torch.empty_like(rows), torch.empty((T, k), device="cuda")
    got, gw = side.check([x, w], [dz, dw], lambda s: F.ufp4_expert_combine_backward(x, rows, ros, sor, w, dz, dw, s))
    assert torch.equal(got, rows / 4)
    size = x.double().square().sum(1, keepdim=True)
    assert ((gw.double() - torch.where(ros >= 0, size, 0.0)).abs() <= cols * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("fmt", [0, 1])
def test_checkpoint_and_gated_activation(env, side, fmt):
    torch, F = env
    g = torch.Generator(device="cuda").manual_seed(fmt)
    rows, width = 100, 96
    gu = torch.randn(rows, 2 * width, device="cuda", generator=g).bfloat16()
    dh = torch.randn(rows, width, device="cuda", generator=g).bfloat16()
    c = F.alloc_checkpoint(rows, 2 * width, fmt)
    F.ufp4_checkpoint_save(gu, c)
    want = (c.codes.clone(), c.scales.clone())
    got = side.check([gu], [c.codes, c.scales], lambda s: F.ufp4_checkpoint_save(gu, c, s))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = torch.empty((rows, 2 * width), device="cuda")
    got, = side.check([c.codes, c.scales], [out], lambda s: F.ufp4_checkpoint_load(c, out, s))
    v = c.codes.view(torch.int8 if fmt == 0 else torch.float8_e4m3fn).float() * c.scales.float().repeat_interleave(32, 1)
    assert torch.equal(got, v)
    # (the current stream's results are tested against 64 bits elsewhere)
    h, again, dgu = torch.empty_like(dh), torch.empty_like(dh), torch.empty_like(gu)
    kept = F.alloc_checkpoint(rows, width, fmt, halves=2)

    def forward(s):
        F.ufp4_gated_act(gu, F.ACT_SILU, h, kept, s)

    def backward(s):
        F.ufp4_gated_act_backward(dh, kept, F.ACT_SILU, dgu, again, s)

    forward(None)
    backward(None)
    want = [t.clone() for t in (h, kept.codes, kept.scales, dgu, again)]
    got = side.check([gu], [h, kept.codes, kept.scales], forward) + side.check([dh], [dgu, again], backward)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    T, k, E = 50, 2, 3
    ids = torch.randint(0, E, (T, k), device="cuda", generator=g, dtype=torch.int32)
    R = F.ufp4_expert_rows(T, k, E, 16)
    off = torch.empty(E + 2, dtype=torch.int64, device="cuda")
    ros, sor = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda")
    F.ufp4_expert_sort(ids, E, 16, off, ros, sor)
    half = F.Checkpoint(c.codes[:T], c.scales[:T], fmt)
    rows_out = torch.empty((R, 2 * width), dtype=torch.bfloat16, device="cuda")
    got, = side.check([c.codes], [rows_out], lambda s: F.ufp4_expert_dispatch_checkpoint(half, ros, sor, rows_out, s))
    assert torch.equal(got, torch.where((sor >= 0)[:, None], v[(sor.clamp(min=0) // k).long()].bfloat16(), 0))


# the kernel for few rows, and the tiles
@pytest.mark.parametrize("rows", [40, 9000])
def test_grouped_products(env, side, rows):
    torch, F = env
    g = torch.Generator(device="cuda").manual_seed(rows)
    E, N, K = 2, 1024, 128
    off = torch.tensor([0, rows // 2 // 16 * 16, rows // 16 * 16], dtype=torch.int64, device="cuda")
    P = rows // 16 * 16

    def operand(lines, length):
        return F.QTensor(torch.randint(0, 256, (lines, length // 2), device="cuda", generator=g, dtype=torch.uint8),
                         torch.randint(0x28, 0x48, (lines, length // 16), device="cuda", generator=g, dtype=torch.uint8),
                         torch.rand(E, device="cuda", generator=g) + 0.5)

    cfg = F.config(grid=F.GRID_E2M1)
    a, b, c = operand(P, K), operand(E * N, K), torch.empty((P, N), device="cuda")
    F.ufp4_gemm_grouped_nt(cfg, a, b, 0, off, K, c)
    want = c.clone()
    assert want.abs().mean() > 0
    got, = side.check([a.codes, b.codes, off], [c], lambda s: F.ufp4_gemm_grouped_nt(cfg, a, b, 0, off, K, c, stream=s))
    assert torch.equal(got, want)
    x, d, dw = operand(96, P), operand(64, P), torch.empty((E, 96, 64), device="cuda")
    F.ufp4_gemm_grouped_dw(cfg, x, d, off, dw)
    want = dw.clone()
    assert want.abs().mean() > 0
    got, = side.check([x.codes, d.codes, off], [dw], lambda s: F.ufp4_gemm_grouped_dw(cfg, x, d, off, dw, stream=s))
    assert torch.equal(got, want)
