"""Host-side checks of the expert-layer entry points: bad arguments are
refused before anything is enqueued (fake pointers, no GPU)."""
import ctypes

import pytest

P = 1 << 40  # aligned, never touched


@pytest.fixture(scope="module")
def F():
    import fp4_quantization_amd as F
    return F


def test_expert_rows(F):
    f = F.lib.ufp4_expert_rows
    assert f(8192, 8, 64, 16) == 8192 * 8 + 64 * 15 and f(1, 8, 64, 16) == 128
    assert f(8192, 8, 64, 1) == 65536 and f(0, 8, 64, 16) == 0
    assert f(5, 3, 4, 16) == 80  # 15 + 4 * 15 = 75, rounded up
    for bad in ((-1, 8, 64, 1), (1, 0, 64, 1), (1, 8, 0, 1), (1, 8, 1024, 1), (1, 8, 64, 0), (1, 8, 64, 4097)):
        assert f(*bad) == 0
    with pytest.raises(ValueError):
        F.ufp4_expert_rows(5, 3, 0)


def test_sort_arguments(F):
    def call(ids=P, tokens=10, slots=2, ld=2, E=4, align=16, rows=1000, off=P, ros=P, sor=P):
        return F.lib.ufp4_expert_sort(ids, tokens, slots, ld, E, align, rows, off, ros, sor, None)

    assert call(rows=79) == 2  # 20 + 4 * 15 = 80
    assert call(tokens=-1) == 1 and call(slots=0) == 1 and call(slots=1025, ld=1025) == 1
    assert call(ld=1) == 1 and call(E=0) == 1 and call(E=1024) == 1 and call(align=0) == 1 and call(align=4097) == 1
    assert call(ids=None) == 1 and call(off=None) == 1 and call(ros=None) == 1 and call(sor=None) == 1
    assert call(ids=P + 2) == 3 and call(off=P + 4) == 3 and call(ros=P + 1) == 3 and call(sor=P + 2) == 3
    assert call(tokens=1 << 28, slots=1, rows=(1 << 28) + 64) == 2


def test_dispatch_arguments(F):
    def call(x=P, tokens=10, cols=64, ld=64, slots=2, ros=P, sor=P, rows=20, out=P, ldo=64):
        return F.lib.ufp4_expert_dispatch(x, tokens, cols, ld, slots, ros, sor, rows, out, ldo, None)

    assert call(ld=63) == 1 and call(ldo=63) == 1 and call(x=None) == 1 and call(out=None) == 1 and call(ros=None) == 1
    assert call(sor=None) == 1 and call(rows=-1) == 1 and call(cols=-1) == 1 and call(slots=0) == 1
    assert call(x=P + 1) == 3 and call(out=P + 1) == 3 and call(ros=P + 2) == 3
    assert call(cols=1 << 25, ld=1 << 25, ldo=1 << 25) == 2 and call(rows=1 << 28) == 2
    assert call(cols=0) == 0 and call(rows=0, sor=None, out=None) == 0

    def kept(codes=P, scales=P, fmt=0, tokens=10, cols=64, slots=2, ros=P, sor=P, rows=20, out=P, ldo=64):
        return F.lib.ufp4_expert_dispatch_checkpoint(codes, scales, fmt, tokens, cols, slots, ros, sor, rows, out, ldo, None)

    assert kept(codes=None) == 1 and kept(scales=None) == 1 and kept(fmt=2) == 1 and kept(fmt=-1) == 1
    assert kept(scales=P + 1) == 3 and kept(ldo=63) == 1 and kept(cols=0) == 0


def test_combine_arguments(F):
    def call(z=P, zt=0, rows=20, cols=64, ldz=64, ros=P, w=None, tokens=10, slots=2, out=P, ot=0, ldo=64):
        return F.lib.ufp4_expert_combine(z, zt, rows, cols, ldz, ros, w, tokens, slots, out, ot, ldo, None)

    assert call(zt=2) == 1 and call(ot=-1) == 1 and call(ldz=63) == 1 and call(ldo=63) == 1 and call(z=None) == 1
    assert call(out=None) == 1 and call(ros=None) == 1 and call(slots=1025) == 1
    assert call(z=P + 2, zt=1) == 3 and call(out=P + 1) == 3 and call(w=P + 2) == 3
    assert call(tokens=0) == 0 and call(cols=0) == 0

    def back(d=P, dt=0, tokens=10, cols=64, ldd=64, slots=2, z=P, zt=0, rows=20, ldz=64, ros=P, sor=P, w=None, dz=P,
             lddz=64, dw=P):
        return F.lib.ufp4_expert_combine_backward(d, dt, tokens, cols, ldd, slots, z, zt, rows, ldz, ros, sor, w, dz,
                                                  lddz, dw, None)

    assert back(d=None) == 1 and back(dt=2) == 1 and back(zt=2) == 1 and back(ldd=1) == 1 and back(ldz=1) == 1
    assert back(lddz=1) == 1 and back(z=None) == 1 and back(ros=None) == 1 and back(sor=None) == 1
    assert back(dz=P + 1) == 3 and back(dw=P + 2) == 3 and back(d=P + 2, dt=1) == 3
    assert back(dz=None, dw=None) == 0


def test_checkpoint_arguments(F):
    def save(x=P, rows=4, cols=64, ld=64, fmt=0, codes=P, scales=P):
        return F.lib.ufp4_checkpoint_save(x, rows, cols, ld, fmt, codes, scales, None)

    assert save(x=None) == 1 and save(rows=-1) == 1 and save(ld=63) == 1 and save(fmt=2) == 1 and save(codes=None) == 1
    assert save(scales=None) == 1 and save(scales=P + 1) == 3 and save(x=P + 1) == 3
    assert save(cols=1 << 25, ld=1 << 25) == 2 and save(rows=0) == 0 and save(cols=0) == 0

    def load(codes=P, scales=P, rows=4, cols=64, fmt=0, out=P, ot=0, ldo=64):
        return F.lib.ufp4_checkpoint_load(codes, scales, rows, cols, fmt, out, ot, ldo, None)

    assert load(codes=None) == 1 and load(ot=2) == 1 and load(fmt=-1) == 1 and load(ldo=1) == 1 and load(out=None) == 1
    assert load(out=P + 2, ot=1) == 3 and load(rows=0) == 0


def test_gated_arguments(F):
    def fwd(gu=P, rows=4, width=64, ld=128, act=0, h=P, ldh=64, fmt=0, codes=None, scales=None):
        return F.lib.ufp4_gated_act(gu, rows, width, ld, act, h, ldh, fmt, codes, scales, None)

    assert fwd(ld=127) == 1 and fwd(ldh=63) == 1 and fwd(act=2) == 1 and fwd(fmt=2) == 1 and fwd(gu=None) == 1
    assert fwd(h=None) == 1 and fwd(codes=P) == 1 and fwd(scales=P) == 1 and fwd(codes=P, scales=P + 1) == 3
    assert fwd(width=1 << 24, ld=1 << 25, ldh=1 << 24) == 2 and fwd(rows=0) == 0

    def bwd(dh=P, lddh=64, codes=P, scales=P, fmt=0, rows=4, width=64, act=0, dgu=P, lddg=128, h=None, ldho=0):
        return F.lib.ufp4_gated_act_backward(dh, lddh, codes, scales, fmt, rows, width, act, dgu, lddg, h, ldho, None)

    assert bwd(dh=None) == 1 and bwd(lddh=63) == 1 and bwd(lddg=127) == 1 and bwd(h=P, ldho=63) == 1
    assert bwd(codes=None) == 1 and bwd(scales=None) == 1 and bwd(act=-1) == 1 and bwd(dgu=P + 1) == 3 and bwd(rows=0) == 0


def qt(F, codes=P, scales=P, ts=P):
    return F.ufp4_qtensor(ctypes.c_void_p(codes), ctypes.c_void_p(scales), ctypes.c_void_p(ts))


def test_grouped_product_arguments(F):
    cfg, mx, bad = F.config(), F.config(scaling=F.SCALE_MX32), F.config(grid=4)

    def nt(cfg=cfg, rows=32, N=16, K=64, a=None, b=None, layout=0, off=P, E=2, c=P, ct=1, ldc=16):
        return F.lib.ufp4_gemm_grouped_nt(ctypes.byref(cfg), rows, N, K, a or qt(F), b or qt(F), layout, off, E, c, ct,
                                          ldc, None)

    assert nt(cfg=mx) == 1 and nt(cfg=bad) == 1 and nt(rows=-1) == 1 and nt(ldc=15) == 1 and nt(E=0) == 1 and nt(E=1025) == 1
    assert nt(ct=2) == 1 and nt(layout=2) == 1 and nt(c=None) == 1 and nt(off=None) == 1
    assert nt(K=48) == 2 and nt(rows=1 << 25) == 2 and nt(N=65535 * 256 + 1, ldc=1 << 25) == 2
    assert nt(a=qt(F, codes=None)) == 1 and nt(b=qt(F, ts=None)) == 1 and nt(a=qt(F, scales=None)) == 1
    assert nt(a=qt(F, codes=P + 8)) == 3 and nt(b=qt(F, scales=P + 1)) == 3 and nt(c=P + 2) == 3 and nt(off=P + 4) == 3
    assert nt(rows=0) == 0 and nt(N=0) == 0

    def dw(cfg=cfg, M=16, N=16, P_=64, a=None, b=None, off=P, E=2, c=P, ct=1):
        return F.lib.ufp4_gemm_grouped_dw(ctypes.byref(cfg), M, N, P_, a or qt(F), b or qt(F), off, E, c, ct, None)

    assert dw(cfg=mx) == 1 and dw(P_=40) == 2 and dw(M=-1) == 1 and dw(E=0) == 1 and dw(ct=-1) == 1 and dw(c=None) == 1
    assert dw(off=None) == 1 and dw(a=qt(F, codes=P + 4)) == 3 and dw(b=qt(F, codes=None)) == 1 and dw(M=0) == 0 and dw(N=0) == 0
    assert dw(M=65535 * 256 + 1) == 2
