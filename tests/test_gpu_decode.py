"""The decoding operators together, as a layer's step runs them: projection,
cache, attention, projection; on another stream, and captured in a graph."""
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


class Layer:
    """An attention layer whose weights and cache are in 4 bits: W model width, H
    key heads, G query heads for each, D values a head."""

    def __init__(self, env, B, L, W=256, H=2, G=3, D=64, P=32, seed=1):
        torch, F = env
        self.env, self.B, self.H, self.G, self.D, self.P = env, B, H, G, D, P
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.cfg = F.config(rht=1, rht_seed=21)

        def weight(n, k):
            q = F.alloc_layout(n, k, 0)
            F.ufp4_quantize((torch.randn(n, k, device="cuda", generator=g) * k ** -0.5).bfloat16(), self.cfg, q, F.Workspace(n, k))
            return q

        self.qkv, self.out = weight((G + 2) * H * D, W), weight(W, G * H * D)
        per = -(-(L + 8) // P)
        self.cache = F.alloc_cache(B * per, P, H, D)
        self.table = torch.randperm(B * per, device="cuda", generator=g).int().view(B, per)
        self.ws = (F.MatvecWorkspace(B, 1 << 12, W, self.cfg), F.MatvecWorkspace(B, W, G * H * D, self.cfg),
                   F.AttentionWorkspace(self.cache, H * G, B, 1))
        self.offsets = torch.arange(B + 1, device="cuda")
        n = B * L
        t = torch.arange(L, device="cuda")
        slots = (self.table.long()[:, t // P] * P + t % P).flatten()
        F.ufp4_cache_append(self.cfg, self.cache, *(torch.randn(n, H * D, device="cuda", generator=g).bfloat16() for _ in range(2)), slots)

    def step(self, x, lengths, slots, stream=None):
        """x [B, W]; lengths with the new token; its slots.  All results."""
        torch, F = self.env
        H, G, D = self.H, self.G, self.D
        qkv = torch.empty(self.B, (G + 2) * H * D, dtype=torch.bfloat16, device="cuda")
        F.ufp4_matvec(self.cfg, x, self.qkv, qkv, self.ws[0], stream=stream)
        q, k, v = qkv[:, :G * H * D], qkv[:, G * H * D:(G + 1) * H * D], qkv[:, (G + 1) * H * D:]
        F.ufp4_cache_append(self.cfg, self.cache, k, v, slots, stream=stream)
        a = torch.empty(self.B, G * H * D, dtype=torch.bfloat16, device="cuda")
        F.ufp4_tree_attention(self.cfg, self.cache, q, self.offsets, lengths, self.table, 1, a, self.ws[2], stream=stream)
        y = torch.empty(self.B, x.shape[1], device="cuda")
        F.ufp4_matvec(self.cfg, a, self.out, y, self.ws[1], stream=stream)
        return qkv, a, y

    def slots_of(self, at):
        return self.table.long().gather(1, (at // self.P)[:, None])[:, 0] * self.P + at % self.P


@pytest.mark.parametrize("B,L", [(1, 45), (7, 130)])
def test_steps(env, B, L):
    """Three tokens: every link against 64 bits on its own inputs."""
    torch, F = env
    m = Layer(env, B, L)
    T = ref.hadamard(F.ufp4_rht_signs(21))
    g = torch.Generator(device="cuda").manual_seed(5)
    for i in range(3):
        x = torch.randn(B, 256, device="cuda", generator=g).bfloat16()
        at = torch.full((B,), L + i, device="cuda")
        lengths = (at + 1).int()
        qkv, a, y = m.step(x, lengths, m.slots_of(at))
        half = 2.0 ** -8  # bf16
        for z, w, out, u, r in ((x, m.qkv, qkv, 2.0 ** -11, half), (a, m.out, y, 2.0 ** -22, 2.0 ** -24)):
            v = ref.values(w.codes, w.scales, 0) * w.tensor_scale.double()[0]
            want = ref.along(z.double(), T) @ v.T
            # roundings of the transformed row and of the transform, K sums, the result's
            bound = (u + 2.0 ** -22 + 400 * 2.0 ** -23) * ((ref.block_sums(z.double()) / 4) @ v.abs().T)
            assert bool(((out.double() - want).abs() <= bound * 1.01 + r * want.abs()).all())
        back = torch.empty(B, m.H * m.D, dtype=torch.bfloat16, device="cuda")
        F.ufp4_cache_read(m.cfg, m.cache, m.slots_of(at), back, None)
        k = qkv[:, m.G * m.H * m.D:(m.G + 1) * m.H * m.D].double()
        # E1M2 codes: half a step of the block's largest transformed value / 3.5 and
        # the scale's own rounding (2^-4), 16 of them in a value; bf16's
        top = ref.along(k, T).reshape(B, -1, 16).abs().amax(-1).repeat_interleave(16, -1)
        assert bool(((back.double() - k).abs() <= 4 * top * (0.25 / 3.5 * 17 / 16 + 1 / 16) + half * k.abs()).all())
        q = qkv[:, :m.G * m.H * m.D].contiguous()
        want, _, e, _ = ref.attention(m.cache, 0, 1, F.ufp4_rht_signs(21), q, m.offsets, lengths, m.table, 1, None, m.D ** -0.5)
        assert bool(((a.double().view_as(want) - want).abs() <= e * 1.01 + half * want.abs()).all())


def test_another_stream(env):
    """Inputs ready only behind slow work of the stream that the calls are given."""
    torch, F = env
    a, b = Layer(env, 5, 70, seed=3), Layer(env, 5, 70, seed=3)
    x = torch.randn(5, 256, device="cuda").bfloat16()
    at = torch.full((5,), 70, device="cuda")
    want = a.step(x, (at + 1).int(), a.slots_of(at))
    busy = torch.randn(8192, 8192, device="cuda").bfloat16()
    late, lengths, slots = torch.zeros_like(x), (at + 1).int(), b.slots_of(at)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(6):
            torch.mm(busy, busy)
        late.copy_(x)
    got = b.step(late, lengths, slots, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_captured(env):
    """A step captured once and replayed over new inputs, lengths and slots, with
    eager work in between; every replay against the eager step."""
    torch, F = env
    a, b = Layer(env, 6, 90, seed=4), Layer(env, 6, 90, seed=4)
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.zeros(6, 256, dtype=torch.bfloat16, device="cuda")
    lengths, slots = torch.zeros(6, dtype=torch.int32, device="cuda"), torch.full((6,), -1, device="cuda")
    b.step(x, lengths, slots)  # (slots outside: nothing is written)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = b.step(x, lengths, slots)
    for i in range(5):
        z = torch.randn(6, 256, device="cuda", generator=g).bfloat16()
        at = torch.tensor([90 + i, 90, 3, 91 + i, 50, 0], device="cuda")
        x.copy_(z)
        lengths.copy_((at + 1).int())
        slots.copy_(b.slots_of(at))
        graph.replay()
        want = a.step(z, (at + 1).int(), a.slots_of(at))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        for p, q in zip(a.cache._tensors[:2], b.cache._tensors[:2]):
            s = a.slots_of(at)
            assert torch.equal(p[s // 32, :, s % 32], q[s // 32, :, s % 32])


def test_two_streams_at_once(env):
    """Calls with workspaces of their own on two streams at the same time."""
    torch, F = env
    layers = [Layer(env, 5, 300, seed=s) for s in (6, 7)]
    x = torch.randn(5, 256, device="cuda").bfloat16()
    at = torch.full((5,), 300, device="cuda")
    args = [(m, (at + 1).int(), m.slots_of(at)) for m in layers]
    want = [m.step(x, n, s) for m, n, s in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    for _ in range(20):
        got = []
        for (m, n, s), st in zip(args, streams):
            with torch.cuda.stream(st):
                got.append(m.step(x, n, s))
        torch.cuda.synchronize()
        for p, q in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(p, q))
