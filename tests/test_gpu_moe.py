"""The expert layer end to end against the same layer in 64 bits without
quantization."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp4_quantization_amd as F
    from fp4_quantization_amd.moe import ExpertLayer
    return torch, F, ExpertLayer


def reference(torch, x, ids, w, w_in, w_out):
    """y and the gradients' graph of the layer in float64 on the CPU."""
    y = torch.zeros_like(x)
    E, F = w_in.shape[0], w_out.shape[2]
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gu = x[t] @ w_in[e].T
        h = torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]
        y = y.index_add(0, t, (h @ w_out[e].T) * w[t, j][:, None])
    return y


@pytest.mark.parametrize("T,k,E,W,H,drop", [(96, 2, 4, 128, 64, 0.1), (1, 3, 8, 96, 160, 0.0), (300, 4, 40, 64, 96, 0.3)])
@pytest.mark.parametrize("recipe", [0, 1, 2])
def test_layer(env, T, k, E, W, H, drop, recipe):
    torch, F, ExpertLayer = env
    g = torch.Generator().manual_seed(T + E + recipe)
    x = torch.randn(T, W, generator=g).to(torch.bfloat16)
    w_in = (torch.randn(E, 2 * H, W, generator=g) * W ** -0.5).to(torch.bfloat16)
    w_out = (torch.randn(E, W, H, generator=g) * H ** -0.5).to(torch.bfloat16)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    ids[torch.rand(T, k, generator=g) < drop] = -1
    w = torch.softmax(torch.randn(T, k, generator=g), 1)
    dy = torch.randn(T, W, generator=g).to(torch.bfloat16)
    layer = ExpertLayer(w_in.cuda(), w_out.cuda(), recipe=recipe, rht_seed=5)
    y, saved = layer.forward(x.cuda(), ids.cuda(), w.cuda())
    grads = layer.backward(saved, dy.cuda(), sr_seed=7)
    ref = [t.double().requires_grad_() for t in (x, w, w_in, w_out)]
    want = reference(torch, ref[0], ids, ref[1], ref[2], ref[3])
    want.backward(dy.double())
    dropped = ids < 0
    assert (grads[3].cpu()[dropped] == 0).all()
    # every product rounds two operands to 4 bits (about 0.1 relative each)
    # and the chain has two products forward, four backward
    for name, got, exact, limit in (("y", y, want, 0.3), ("dx", grads[0], ref[0].grad, 0.5), ("dw_in", grads[1], ref[2].grad, 0.5),
                                    ("dw_out", grads[2], ref[3].grad, 0.5), ("dweights", grads[3], ref[1].grad, 0.4)):
        err = (got.double().cpu() - exact).norm() / exact.norm()
        print(name, float(err), flush=True)
        assert torch.isfinite(got).all() and err < limit, name
    # without a backward pass the same output, and the same bits again
    assert torch.equal(layer.forward(x.cuda(), ids.cuda(), w.cuda(), train=False)[0], y)
    again = layer.backward(saved, dy.cuda(), sr_seed=7)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_refusals(env):
    torch, F, ExpertLayer = env
    with pytest.raises(ValueError):
        ExpertLayer(torch.zeros(2, 64, 40).cuda().bfloat16(), torch.zeros(2, 40, 32).cuda().bfloat16())
    with pytest.raises(ValueError):
        ExpertLayer(torch.zeros(2, 64, 32).cuda().bfloat16(), torch.zeros(2, 32, 64).cuda().bfloat16())
