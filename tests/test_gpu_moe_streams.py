"""The expert layer on a stream of its own, behind work that keeps that stream
busy, while the current stream takes and overwrites all memory it is given."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from fp4_quantization_amd.moe import ExpertLayer
    return torch, ExpertLayer


def make(torch, seed, T=257, k=3, E=5, W=128, H=96):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    ids = torch.randint(-1, E, (T, k), device="cuda", generator=g, dtype=torch.int32)
    # (the gate's weights as a transposed view: load copies it)
    return ((new(E, W, 2 * H) * W ** -0.5).bfloat16().transpose(1, 2), (new(E, W, H) * H ** -0.5).bfloat16(), new(T, W).bfloat16(),
            ids, torch.rand(T, k, device="cuda", generator=g), new(T, W).bfloat16())


def overwrite(torch):
    """Takes memory of many sizes from the current stream's pool and fills it."""
    for n in (512, 4096, 1 << 14, 1 << 16, 1 << 18, 1 << 20, 1 << 22):
        for _ in range(24):
            torch.full((n,), 0x55, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("one_stream", [True, False])
def test_another_stream(env, one_stream):
    torch, Layer = env
    w_in, w_out, x, ids, w, dy = make(torch, 3)
    layer = Layer(w_in, w_out, rht_seed=5)
    y, saved = layer.forward(x, ids, w)
    want = (y, *layer.backward(saved, dy, sr_seed=7))
    saved = None
    other = Layer(*make(torch, 4)[:2], rht_seed=5)
    torch.cuda.synchronize()
    busy = torch.randn(8192, 8192, device="cuda").bfloat16()
    cur = torch.cuda.current_stream()
    streams = [torch.cuda.Stream() for _ in range(3)]
    s = streams[0]

    def occupy(stream):
        stream.wait_stream(cur)
        with torch.cuda.stream(stream):
            for _ in range(8):
                torch.mm(busy, busy)

    occupy(s)
    # inputs made on the current stream right before, and dropped right after
    args = [t.clone() for t in (w_in, w_out)]
    other.load(*args, stream=s)
    args = None
    overwrite(torch)
    if not one_stream:
        cur.wait_stream(s)
        s = streams[1]
        occupy(s)
    args = [t.clone() for t in (x, ids, w)]
    y, saved = other.forward(*args, stream=s)
    args = None
    overwrite(torch)
    if not one_stream:
        cur.wait_stream(s)
        s = streams[2]
        occupy(s)
    arg = dy.clone()
    got = (y, *other.backward(saved, arg, sr_seed=7, stream=s))
    saved = arg = None
    overwrite(torch)
    other.load(*make(torch, 6)[:2])  # (the weights in use are dropped)
    overwrite(torch)
    cur.wait_stream(s)
    for name, a, b in zip(("y", "dx", "dw_in", "dw_out", "dweights"), got, want):
        assert torch.equal(a, b), name


def test_captured_in_a_graph(env):
    """A forward and a backward pass captured once (on the capture's own
    stream, the weights loaded on another) and replayed over changed inputs."""
    torch, Layer = env
    w_in, w_out, x, ids, w, dy = make(torch, 3)
    layer = Layer(w_in, w_out, rht_seed=5)

    def step():
        y, saved = layer.forward(x, ids, w)
        return (y, *layer.backward(saved, dy, sr_seed=7))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (8, 9, 10, 8):
        for t, v in zip((x, ids, w, dy), make(torch, seed)[2:]):
            t.copy_(v)
        graph.replay()
        copies = [t.clone() for t in got]
        want = step()
        torch.cuda.synchronize()
        for name, a, b in zip(("y", "dx", "dw_in", "dw_out", "dweights"), copies, want):
            assert torch.equal(a, b), name
