"""The keys of the expert layer's stochastic rounding (no GPU): a gradient that
is computed from a rounded one is rounded with other random numbers."""
import numpy as np
import pytest
import torch


@pytest.fixture
def quantized(monkeypatch):
    """The layer with stubs for all device calls; the configurations of its
    quantizations, each with the tensor that it was of."""
    from fp4_quantization_amd import moe
    calls = []

    class Stream:
        cuda_stream = 0

    class Workspace:
        def __init__(self, *args, **kwargs):
            self.buf = torch.empty(1)

    for name in [n for n in vars(moe) if n.startswith("ufp4_") and n not in ("ufp4_recipe_config", "ufp4_expert_rows")]:
        monkeypatch.setattr(moe, name, lambda *args, **kwargs: None)
    monkeypatch.setattr(moe, "ufp4_quantize_grouped", lambda x, off, rows, cfg, row, col, ws, stream=None: calls.append((x, cfg)))
    monkeypatch.setattr(moe, "Workspace", Workspace)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    E, H, W, T, k = 2, 32, 64, 4, 2
    layer = moe.ExpertLayer(torch.zeros(E, 2 * H, W).bfloat16(), torch.zeros(E, W, H).bfloat16())
    y, saved = layer.forward(torch.zeros(T, W).bfloat16(), torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k))
    assert all(cfg.rounding == 0 for _, cfg in calls)  # weights and activations to nearest

    def backward(seed):
        calls.clear()
        layer.backward(saved, torch.zeros(T, W).bfloat16(), sr_seed=seed)
        keys = {}
        for x, cfg in calls:
            if cfg.rounding == 1:
                keys.setdefault(id(x), set()).add(cfg.sr_seed)
        return list(keys.values())

    return backward


def test_every_gradient_has_its_own_key(quantized):
    seen = set()
    for seed in (0, 1, 2, 1 << 40):
        keys = quantized(seed)
        # the experts' output gradient and the gated activation's, each by one
        # key in both of its layouts (which draw from streams of their own)
        assert len(keys) == 2 and all(len(k) == 1 for k in keys)
        keys = {next(iter(k)) for k in keys}
        assert len(keys) == 2 and not keys & seen
        seen |= keys


def test_a_shared_key_is_biased(orc):
    """Why: a value that depends on a rounded one, rounded by the same random
    number, does not have the mean of its argument."""
    import synth
    rng = np.random.default_rng(0)
    xb = synth.f32_to_bf16(rng.standard_normal((16, 32)).astype(np.float32))
    x = synth.bf16_to_f32(xb).astype(float)
    d = rng.uniform(0.5, 1.5, x.shape)

    def rounded(v, seed):
        cfg = orc.config(rounding=1, rht=0, sr_seed=seed)
        return orc.dequantize(*orc.quantize(v, cfg, 0), *v.shape, cfg, 0).astype(float)

    total, n = {0: 0, 1 << 63: 0}, 1000
    for s in range(n):
        y = synth.f32_to_bf16((d * rounded(xb, s)).astype(np.float32))
        for flip in total:
            total[flip] = total[flip] + rounded(y, s ^ flip)
    rms = {f: np.sqrt(np.mean((t / n - d * x) ** 2)) for f, t in total.items()}
    assert rms[0] > 1.5 * rms[1 << 63]
