"""Caches and workspaces whose buffers get other memory after they were made: a call
takes the addresses as they are, and refuses what no longer fits."""
import pytest
import torch


@pytest.fixture(scope="module")
def F():
    import fp4_quantization_amd as F
    return F


NAMES = ["k_codes", "k_scales", "v_codes", "v_scales", "k_scale", "v_scale"]
FIELDS = NAMES[:4] + ["k_tensor_scale", "v_tensor_scale"]


def make(F, device="cpu"):
    return F.alloc_cache(3, 64, 2, 96, *(torch.full((2,), 0.01, device=device) for _ in range(2)), device=device)


@pytest.mark.parametrize("i", range(6))
def test_replaced_memory(F, i):
    c = make(F)
    for _ in range(2):
        t = getattr(c, NAMES[i])
        t.data = t.clone()
        got = c.c()
        assert [getattr(got, f) for f in FIELDS] == [getattr(c, n).data_ptr() for n in NAMES]


@pytest.mark.parametrize("i", range(6))
def test_memory_that_no_longer_fits(F, i):
    for change in (lambda t: t.resize_(0), lambda t: t.resize_(t.shape[0] + 1, *t.shape[1:]), lambda t: setattr(t, "data", t[1:].clone()),
                   lambda t: setattr(t, "data", t.double())):
        c = make(F)
        c.c()
        change(getattr(c, NAMES[i]))
        for _ in range(2):
            with pytest.raises(ValueError):
                c.c()


def test_other_geometry(F):
    """All buffers of another cache: valid, but not this one's pages."""
    c, other = make(F), F.alloc_cache(4, 64, 2, 96, device="cpu")
    for n in NAMES[:4]:
        getattr(c, n).data = getattr(other, n)
    with pytest.raises(ValueError, match="geometry"):
        c.c()


def test_workspaces(F):
    for ws in (F.AttentionWorkspace(make(F), 4, 3, 2), F.MatvecWorkspace(20, 64, 128, F.config(), device="cpu")):
        n = ws.nbytes
        assert n > 0 and ws.ptr == ws.buf.data_ptr()
        ws.buf.resize_(64 * n)
        assert ws.ptr == ws.buf.data_ptr() and ws.nbytes == 64 * n
        ws.buf.resize_(n - 1)
        assert ws.nbytes == n - 1


@pytest.mark.gpu
def test_calls_follow_the_memory(F):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cfg, T, g = F.config(), 50, torch.Generator(device="cuda").manual_seed(1)
    c = make(F, "cuda")
    k, v = (torch.randn(T, 192, device="cuda", generator=g).bfloat16() for _ in range(2))
    slots = torch.arange(T, device="cuda")
    q = torch.randn(1, 384, device="cuda", generator=g).bfloat16()
    off, lens = torch.tensor([0, 1], device="cuda"), torch.tensor([T], dtype=torch.int32, device="cuda")
    table, ws = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), F.AttentionWorkspace(c, 4, 1, 1)

    def results():
        a, b, o = (torch.empty(n, w, dtype=torch.bfloat16, device="cuda") for n, w in ((T, 192), (T, 192), (1, 384)))
        F.ufp4_cache_read(cfg, c, slots, a, b)
        F.ufp4_tree_attention(cfg, c, q, off, lens, table, 1, o, ws)
        return a, b, o

    F.ufp4_cache_append(cfg, c, k, v, slots)
    want, kept = results(), []
    for n in NAMES:
        t = getattr(c, n)
        old = t.data
        t.data = t.clone()
        old.zero_()
        kept.append(old)  # (its memory stays this test's)
    ws.buf.data = torch.empty_like(ws.buf)
    assert all(torch.equal(x, y) for x, y in zip(results(), want))
    F.ufp4_cache_append(cfg, c, v, k, slots)
    a, b, _ = results()
    assert torch.equal(a, want[1]) and torch.equal(b, want[0])
    assert not any(bool(t.any()) for t in kept)
    ws.buf.data = ws.buf[:-16].clone()
    with pytest.raises(F.Ufp4Error):
        results()
