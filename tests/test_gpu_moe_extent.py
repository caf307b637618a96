"""The expert-layer operators where offsets pass 32 bits, and replayed from a
captured graph."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp4_quantization_amd as F
    yield torch, F
    torch.cuda.empty_cache()


def test_rows_past_2_to_the_31_elements(env):
    torch, F = env
    T, k, E, cols = 70000, 8, 16, 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, E, (T, k), device="cuda", generator=g, dtype=torch.int32)
    R = F.ufp4_expert_rows(T, k, E, 16)
    assert R * cols > 1 << 31
    off = torch.empty(E + 2, dtype=torch.int64, device="cuda")
    ros, sor = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda")
    F.ufp4_expert_sort(ids, E, 16, off, ros, sor)
    x = torch.randn(T, cols, device="cuda", generator=g).to(torch.bfloat16)
    rows = torch.empty((R, cols), dtype=torch.bfloat16, device="cuda")
    F.ufp4_expert_dispatch(x, ros, sor, rows)
    for lo in (0, R // 2, R - 5000):
        s = sor[lo:lo + 5000]
        assert torch.equal(rows[lo:lo + 5000], torch.where((s >= 0)[:, None], x[(s.clamp(min=0) // k).long()], 0))
    w = torch.full((T, k), 1.0 / k, device="cuda")
    y = torch.empty_like(x)
    F.ufp4_expert_combine(rows, ros, w, y)
    assert torch.equal(y, x)  # eight equal rows, weights a power of two
    dz, dw = torch.empty_like(rows), torch.empty_like(w)
    F.ufp4_expert_combine_backward(x, rows, ros, sor, w, dz, dw)
    s = sor[R - 5000:]
    assert torch.equal(dz[R - 5000:], torch.where((s >= 0)[:, None], x[(s.clamp(min=0) // k).long()] / k, 0))
    want = x[-1000:].double().square().sum(1)
    assert ((dw[-1000:].double() - want[:, None]).abs() <= cols * 2.0 ** -24 * want[:, None]).all()


def test_gated_past_2_to_the_31_elements(env):
    torch, F = env
    rows, width = 300000, 4000
    assert 2 * rows * width > 1 << 31
    gu = torch.empty((rows, 2 * width), dtype=torch.bfloat16, device="cuda").normal_()
    dh = torch.empty((rows, width), dtype=torch.bfloat16, device="cuda").normal_()
    c = F.alloc_checkpoint(rows, width, F.CKPT_INT8, halves=2)
    h, dgu = torch.empty_like(dh), torch.empty_like(gu)
    F.ufp4_gated_act(gu, F.ACT_SILU, h, c)
    F.ufp4_gated_act_backward(dh, c, F.ACT_SILU, dgu)
    for lo in (0, rows - 200):
        part = slice(lo, lo + 200)
        pc = F.alloc_checkpoint(200, width, F.CKPT_INT8, halves=2)
        ph, pd = torch.empty_like(h[part]), torch.empty_like(dgu[part])
        F.ufp4_gated_act(gu[part], F.ACT_SILU, ph, pc)
        F.ufp4_gated_act_backward(dh[part], pc, F.ACT_SILU, pd)
        assert torch.equal(ph, h[part]) and torch.equal(pd, dgu[part]) and torch.equal(pc.codes, c.codes[part])


def random_operand(torch, F, lines, length, E, g):
    codes = torch.randint(0, 256, (lines, length // 2), device="cuda", generator=g, dtype=torch.uint8)
    scales = torch.randint(0x28, 0x48, (lines, length // 16), device="cuda", generator=g, dtype=torch.uint8)
    return F.QTensor(codes, scales, torch.rand(E, device="cuda", generator=g) + 0.5)


@pytest.mark.parametrize("rows", [300, 40000])
def test_products_with_weights_past_4_gigabytes(env, rows):
    torch, F = env
    E, N, K = 600, 4096, 4096
    g = torch.Generator(device="cuda").manual_seed(2)
    cfg = F.config()
    b = random_operand(torch, F, E * N, K, E, g)
    assert b.codes.numel() > 1 << 32
    a = random_operand(torch, F, rows, K, E, g)
    # all rows in the last two experts
    off = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    off[E - 1], off[E] = rows // 3, rows
    c, part = torch.empty((rows, N), device="cuda"), torch.empty((rows, N), device="cuda")
    F.ufp4_gemm_grouped_nt(cfg, a, b, 0, off, K, c)
    last = F.QTensor(b.codes[(E - 2) * N:], b.scales[(E - 2) * N:], b.tensor_scale[E - 2:].contiguous())
    two = F.QTensor(a.codes, a.scales, a.tensor_scale[E - 2:].contiguous())
    F.ufp4_gemm_grouped_nt(cfg, two, last, 0, off[E - 2:].contiguous(), K, part)
    # (the two calls may take different kernels: same products, another order)
    assert ((c - part).abs() <= 1e-4 * part.abs().mean() + 1e-5 * part.abs()).all()
    assert c.abs().mean() > 0


def test_weight_gradients_past_2_to_the_31_elements(env):
    torch, F = env
    E, M, N, P = 70, 8192, 4096, 70 * 16
    assert E * M * N > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(3)
    a, b = random_operand(torch, F, M, P, E, g), random_operand(torch, F, N, P, E, g)
    off = torch.arange(E + 1, dtype=torch.int64, device="cuda") * 16
    c = torch.empty((E, M, N), device="cuda")
    F.ufp4_gemm_grouped_dw(F.config(), a, b, off, c)
    one = torch.empty((1, M, N), device="cuda")
    pick = lambda q: F.QTensor(q.codes[:, -8:].contiguous(), q.scales[:, -1:].contiguous(), q.tensor_scale[-1:].contiguous())  # noqa: E731
    F.ufp4_gemm_grouped_dw(F.config(), pick(a), pick(b), off[:2].contiguous(), one)
    assert torch.equal(c[-1], one[0]) and one.abs().mean() > 0


def test_captured_in_a_graph(env):
    """The layer's calls captured once and replayed over changed inputs."""
    torch, F = env
    T, k, E, D = 200, 4, 12, 256
    g = torch.Generator(device="cuda").manual_seed(4)
    R = F.ufp4_expert_rows(T, k, E, 16)
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    x = torch.empty((T, D), dtype=torch.bfloat16, device="cuda")
    w = torch.empty((T, k), device="cuda")
    off = torch.empty(E + 2, dtype=torch.int64, device="cuda")
    ros, sor = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda")
    rows = torch.empty((R, D), dtype=torch.bfloat16, device="cuda")
    weights = random_operand(torch, F, E * 2 * D, D, E, g)
    q = F.alloc_layout(R, D, 0, E + 1)
    ws = F.Workspace(R, D, E + 1)
    gu = torch.empty((R, 2 * D), dtype=torch.bfloat16, device="cuda")
    kept = F.alloc_checkpoint(R, D, F.CKPT_INT8, halves=2)
    h, dgu = torch.empty_like(rows), torch.empty_like(gu)
    y = torch.empty_like(x)
    cfg = F.config()

    def step():
        F.ufp4_expert_sort(ids, E, 16, off, ros, sor)
        F.ufp4_expert_dispatch(x, ros, sor, rows)
        F.ufp4_quantize_grouped(rows, off, R, cfg, q, None, ws)
        F.ufp4_gemm_grouped_nt(cfg, q, weights, 0, off, D, gu, E)
        F.ufp4_gated_act(gu, F.ACT_SILU, h, kept)
        F.ufp4_gated_act_backward(h, kept, F.ACT_SILU, dgu)
        F.ufp4_expert_combine(h, ros, w, y)

    def fill(seed):
        n = torch.Generator(device="cuda").manual_seed(seed)
        ids.copy_(torch.randint(-1, E, (T, k), device="cuda", generator=n, dtype=torch.int32))
        x.copy_(torch.randn(T, D, device="cuda", generator=n))
        w.copy_(torch.rand(T, k, device="cuda", generator=n))

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2, 3, 1):
        fill(seed)
        graph.replay()
        got = [t.clone() for t in (off, ros, sor, rows, gu, dgu, y)]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (off, ros, sor, rows, gu, dgu, y)):
            assert torch.equal(a, b)
