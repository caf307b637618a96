"""Host-side checks of the decoding entry points: bad arguments are refused
before anything is enqueued (fake pointers, CPU tensors, no GPU)."""
import ctypes

import pytest
import torch

P = 1 << 40  # aligned, never touched


@pytest.fixture(scope="module")
def F():
    import fp4_quantization_amd as F
    return F


def cfg_of(F, **kw):
    return ctypes.byref(F.config(**kw))


def test_matvec_arguments(F):
    def call(cfg=None, x=P, xt=0, T=1, K=64, ldx=64, codes=P, scales=P, ts=P, N=32, y=P, yt=0, ldy=32, ws=None, nb=0, **kw):
        cfg = cfg_of(F, **kw) if cfg is None else cfg
        return F.lib.ufp4_matvec(cfg, x, xt, T, K, ldx, F.ufp4_qtensor(codes, scales, ts), N, y, yt, ldy, ws, nb, None)

    assert F.lib.ufp4_matvec(None, P, 0, 1, 64, 64, F.ufp4_qtensor(P, P, P), 32, P, 0, 32, None, 0, None) == 1
    assert call(grid=4) == 1 and call(grid=-1) == 1 and call(scaling=2) == 1
    assert call(xt=2) == 1 and call(yt=-1) == 1 and call(ldx=63) == 1 and call(ldy=31) == 1
    assert call(T=-1) == 1 and call(N=-1) == 1 and call(K=-32, ldx=64) == 1
    assert call(K=48) == 2 and call(K=1 << 25, ldx=1 << 25) == 2 and call(N=1 << 25, ldy=1 << 25) == 2 and call(T=1 << 21) == 2
    assert call(x=None) == 1 and call(codes=None) == 1 and call(scales=None) == 1 and call(ts=None) == 1 and call(y=None) == 1
    assert call(x=P + 1) == 3 and call(x=P + 2, xt=1) == 3 and call(y=P + 1) == 3 and call(y=P + 2, yt=1) == 3
    assert call(codes=P + 8) == 3 and call(scales=P + 1) == 3 and call(ts=P + 2) == 3
    assert call(T=0, x=None, y=None) == 0 and call(N=0, y=None) == 0
    # the workspace: none for a few tokens, needed for more
    size = F.lib.ufp4_matvec_workspace
    assert size(cfg_of(F), 1, 32, 4096) == 0 and size(cfg_of(F), 16, 32, 4096) >= 16 * 4096 * 2 * 2
    assert size(cfg_of(F), 16, 32, 48) == 0 and size(cfg_of(F), 0, 32, 64) == 0 and size(None, 16, 32, 64) == 0
    n = size(cfg_of(F), 16, 32, 64)
    assert call(T=16) == 4 and call(T=16, ws=P, nb=n - 1) == 4 and call(T=16, ws=P + 8, nb=n) == 4
    assert size(cfg_of(F, scaling=1), 16, 32, 64) > n  # three parts


def cache(F, kc=P, ks=P, vc=P, vs=P, kt=None, vt=None, pages=4, P_=64, heads=2, dim=128):
    return F._lib.ufp4_cache(kc, ks, vc, vs, kt, vt, pages, P_, heads, dim)


BAD_CACHES = [(dict(pages=-1), 1), (dict(heads=0), 1), (dict(heads=1025), 1), (dict(dim=0), 1), (dict(P_=0), 1),
              (dict(dim=48), 2), (dict(dim=288), 2), (dict(P_=48), 2), (dict(P_=65568), 2), (dict(pages=1 << 34), 2),
              (dict(kc=None), 1), (dict(vs=None), 1), (dict(kc=P + 8), 3), (dict(ks=P + 4), 3), (dict(vc=P + 1), 3),
              (dict(kt=P + 2), 3), (dict(vt=P + 1), 3)]


def test_append_arguments(F):
    def call(c=None, k=P, ldk=256, v=P, ldv=256, T=3, slots=P, **kw):
        c = cache(F) if c is None else c
        return F.lib.ufp4_cache_append(cfg_of(F, **kw), ctypes.byref(c), k, ldk, v, ldv, T, slots, None)

    for kw, rc in BAD_CACHES:
        assert call(cache(F, **kw)) == rc, kw
    assert F.lib.ufp4_cache_append(cfg_of(F), None, P, 256, P, 256, 3, P, None) == 1
    assert F.lib.ufp4_cache_append(None, ctypes.byref(cache(F)), P, 256, P, 256, 3, P, None) == 1
    assert call(grid=4) == 1 and call(scaling=1) == 1 and call(rounding=1) == 1
    assert call(ldk=255) == 1 and call(ldv=255) == 1 and call(T=-1) == 1 and call(T=1 << 28) == 2
    assert call(k=None) == 1 and call(v=None) == 1 and call(slots=None) == 1
    assert call(k=P + 1) == 3 and call(v=P + 1) == 3 and call(slots=P + 4) == 3
    assert call(T=0, k=None, v=None, slots=None) == 0


def test_read_arguments(F):
    def call(c=None, slots=P, T=3, inv=1, k=P, ldk=256, v=P, ldv=256, kind=0, **kw):
        c = cache(F) if c is None else c
        return F.lib.ufp4_cache_read(cfg_of(F, **kw), ctypes.byref(c), slots, T, inv, k, ldk, v, ldv, kind, None)

    for kw, rc in BAD_CACHES:
        assert call(cache(F, **kw)) == rc, kw
    assert call(grid=4) == 1 and call(scaling=1) == 1 and call(kind=2) == 1 and call(T=-1) == 1 and call(T=1 << 28) == 2
    assert call(ldk=255) == 1 and call(ldv=255) == 1 and call(slots=None) == 1
    assert call(k=P + 1) == 3 and call(v=P + 2, kind=1) == 3 and call(slots=P + 4) == 3
    assert call(T=0) == 0 and call(k=None, v=None) == 0


def test_attention_arguments(F):
    def call(c=None, q=P, ldq=1024, heads=8, off=P, n=3, rows=5, most=2, lens=P, table=P, ld=7, mask=None, scale=0.1, out=P,
             ldo=1024, lse=None, ws=P, nb=1 << 40, **kw):
        c = cache(F) if c is None else c
        return F.lib.ufp4_tree_attention(cfg_of(F, **kw), ctypes.byref(c), q, ldq, heads, off, n, rows, most, lens, table, ld, mask,
                                         scale, out, ldo, lse, ws, nb, None)

    for kw, rc in BAD_CACHES:
        assert call(cache(F, **kw)) == rc, kw
    assert call(grid=4) == 1 and call(scaling=1) == 1
    assert call(heads=0) == 1 and call(heads=7) == 1 and call(heads=8194) == 1 and call(n=-1) == 1 and call(rows=-1) == 1
    assert call(most=0) == 1 and call(ld=-1) == 1 and call(most=65, mask=P) == 1
    assert call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(ldq=1023) == 1 and call(ldo=1023) == 1
    assert call(n=65536) == 2 and call(rows=1 << 28) == 2 and call(ld=1 << 25) == 2 and call(most=1 << 28) == 2
    assert call(q=None) == 1 and call(out=None) == 1 and call(off=None) == 1 and call(lens=None) == 1 and call(table=None) == 1
    assert call(q=P + 1) == 3 and call(out=P + 1) == 3 and call(off=P + 4) == 3 and call(lens=P + 2) == 3
    assert call(table=P + 2) == 3 and call(mask=P + 4) == 3 and call(lse=P + 2) == 3
    assert call(n=0) == 0 and call(rows=0) == 0
    size = F.lib.ufp4_tree_attention_workspace
    need = size(ctypes.byref(cache(F)), 8, 3, 2)
    assert need > 0 and call(nb=need - 1) == 4 and call(ws=None) == 4 and call(ws=P + 8) == 4
    for bad in ((0, 3, 2), (7, 3, 2), (8, -1, 2), (8, 65536, 2), (8, 3, 0), (8, 3, 1 << 28)):
        assert size(ctypes.byref(cache(F)), *bad) == 0
    assert size(None, 8, 3, 2) == 0 and size(ctypes.byref(cache(F, dim=48)), 8, 3, 2) == 0


def test_matvec_tensors(F):
    def call(x=None, w=None, y=None, cfg=None):
        F.ufp4_matvec(cfg or F.config(), torch.zeros(2, 64).bfloat16() if x is None else x,
                      F.alloc_layout(32, 64, 0, device="cpu") if w is None else w, torch.zeros(2, 32) if y is None else y)

    with pytest.raises(ValueError, match="on the GPU"):
        call()
    with pytest.raises(ValueError, match="one row a token"):
        call(y=torch.zeros(3, 32))
    with pytest.raises(ValueError, match="w must hold 32 contiguous lines of 64"):
        call(w=F.alloc_layout(33, 64, 0, device="cpu"))
    with pytest.raises(ValueError, match="w must hold"):
        call(cfg=F.config(scaling=F.SCALE_MX32))
    with pytest.raises(TypeError):
        call(x=torch.zeros(2, 64).half())
    with pytest.raises(ValueError, match="unit column stride"):
        call(x=torch.zeros(64, 2).bfloat16().T)
    w = F.alloc_layout(32, 64, 0, device="cpu")
    w.codes = w.codes.to(torch.int16)
    with pytest.raises(ValueError, match="w must hold"):
        call(w=w)


def test_cache_tensors(F):
    c = F.alloc_cache(4, 64, 2, 128, device="cpu")
    assert (c.pages, c.page_tokens, c.heads, c.dim) == (4, 64, 2, 128)
    for bad in ((4, 48, 2, 128), (4, 64, 2, 144)):
        with pytest.raises(ValueError):
            F.alloc_cache(*bad, device="cpu")
    with pytest.raises(ValueError, match="float32"):
        F.alloc_cache(4, 64, 2, 128, k_scale=torch.ones(3), device="cpu")
    with pytest.raises(ValueError, match="contiguous bytes"):
        F.QCache(c.k_codes, c.k_scales, c.v_codes.transpose(3, 4), c.v_scales)
    k, slots = torch.zeros(3, 256).bfloat16(), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="on the GPU"):
        F.ufp4_cache_append(F.config(), c, k, k, slots)
    with pytest.raises(ValueError, match="one slot a token"):
        F.ufp4_cache_append(F.config(), c, k, k, slots[:2])
    with pytest.raises(ValueError, match="heads \\* dim"):
        F.ufp4_cache_append(F.config(), c, k[:, :128], k[:, :128], slots)
    with pytest.raises(TypeError, match="int64"):
        F.ufp4_cache_append(F.config(), c, k, k, slots.int())
    with pytest.raises(TypeError, match="bf16"):
        F.ufp4_cache_append(F.config(), c, k.float(), k, slots)
    with pytest.raises(TypeError, match="one type"):
        F.ufp4_cache_read(F.config(), c, slots, k, k.float())
    with pytest.raises(ValueError, match="one row a slot"):
        F.ufp4_cache_read(F.config(), c, slots, k[:2], None)


def test_attention_tensors(F):
    c = F.alloc_cache(4, 64, 2, 128, device="cpu")
    with pytest.raises(ValueError, match="attention shape"):
        F.AttentionWorkspace(c, 7, 3, 2)
    base = dict(q=torch.zeros(5, 1024).bfloat16(), q_offsets=torch.tensor([0, 2, 3, 5]), lengths=torch.zeros(3, dtype=torch.int32),
                page_table=torch.zeros(3, 7, dtype=torch.int32), max_draft=2, out=torch.zeros(5, 1024).bfloat16(),
                ws=F.AttentionWorkspace(c, 8, 3, 2))

    def call(**kw):
        F.ufp4_tree_attention(F.config(), c, **{**base, **kw})

    for match, kw in (("on the GPU", {}), ("multiple of the cache", dict(q=base["q"][:, :896], out=base["out"][:, :896])),
                      ("multiple of the cache", dict(out=base["out"][:4])), ("one entry more", dict(q_offsets=torch.tensor([0, 5]))),
                      ("one line a sequence", dict(page_table=torch.zeros(2, 7, dtype=torch.int32))),
                      ("one entry a row", dict(mask=torch.zeros(4, dtype=torch.int64)))):
        with pytest.raises(ValueError, match=match):
            call(**kw)
    for match, kw in (("int64", dict(q_offsets=torch.zeros(4, dtype=torch.int32))), ("int32", dict(lengths=torch.zeros(3, dtype=torch.int64))),
                      ("int64", dict(mask=torch.zeros(5, dtype=torch.int32))), ("lse", dict(lse=torch.zeros(5, 7))),
                      ("bf16", dict(q=torch.zeros(5, 1024)))):
        with pytest.raises(TypeError, match=match):
            call(**kw)


def test_workspaces_of_larger_calls_do_for_smaller_ones(F):
    """A workspace for up to so many tokens is large enough for fewer of them."""
    for dim in (32, 64, 96, 128, 192, 256):
        for heads in (2, 8, 16, 64):
            c = cache(F, dim=dim)
            sizes = [F.lib.ufp4_tree_attention_workspace(ctypes.byref(c), heads, 3, n) for n in range(1, 65)]
            assert sizes[0] > 0 and sizes == sorted(sizes)
    for K in (32, 4096, 65536):
        for scaling in (0, 1):
            sizes = [F.lib.ufp4_matvec_workspace(cfg_of(F, scaling=scaling), n, 64, K) for n in range(1, 130)]
            assert sizes == sorted(sizes)
