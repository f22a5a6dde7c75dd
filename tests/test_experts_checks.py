"""What the grouped and 4-bit operators refuse, without a GPU: the C ABI's argument checks
(before any HIP call) and the binding's (CPU tensors reach every check; a call that passes
all of them ends in the "must be on the GPU" error)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import swiglu_gemm_amd as sg
from swiglu_gemm_amd import build as sgbuild

ON_GPU = "on the GPU"
P, ODD, NUL = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1001), ctypes.c_void_p(0)
BF, F16, F8, F32 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.float32


@pytest.fixture(scope="module")
def L():
    if sgbuild.is_stale():
        sgbuild.build()
    return sg.lib()


def expect(fn, order, base, cases):
    """fn called with base's values in `order`, each case changing some of them."""
    for want, change in cases:
        args = dict(base, **change)
        assert fn(*[args[k] for k in order]) == want, change


def test_grouped_gemm_abi(L):
    order = "tb E off M N K alpha scale A lda B ldb sB beta C ldc dt st".split()
    base = dict(tb=b"N", E=2, off=P, M=4, N=8, K=16, alpha=1.0, scale=NUL, A=P, lda=16, B=P, ldb=8,
                sB=128, beta=0.0, C=P, ldc=8, dt=2, st=NUL)
    expect(L.sg_grouped_gemm, order, base, [
        (-1, dict(tb=b"X")), (-2, dict(E=0)), (-2, dict(E=65537)), (-3, dict(off=NUL)),
        (-4, dict(M=-1)), (-5, dict(N=-1)), (-6, dict(K=-1)), (-9, dict(A=NUL)), (-10, dict(lda=15)),
        (-11, dict(B=NUL)), (-12, dict(ldb=7)), (-12, dict(tb=b"T", ldb=15)), (-13, dict(sB=-1)),
        (-15, dict(C=NUL)), (-16, dict(ldc=7)), (-17, dict(dt=0)), (-17, dict(dt=4)),
        (0, dict(M=0, A=NUL, B=NUL, C=NUL)), (0, dict(N=0, B=NUL, C=NUL))])


def test_grouped_wgrad_abi(L):
    order = "E off M N K alpha A lda D ldd beta C ldc sC dt cdt st".split()
    base = dict(E=2, off=P, M=4, N=8, K=16, alpha=1.0, A=P, lda=16, D=P, ldd=8, beta=0.0, C=P, ldc=8,
                sC=128, dt=2, cdt=0, st=NUL)
    expect(L.sg_grouped_gemm_wgrad, order, base, [
        (-1, dict(E=0)), (-2, dict(off=NUL)), (-3, dict(M=-1)), (-4, dict(N=-1)), (-5, dict(K=-1)),
        (-7, dict(A=NUL)), (-8, dict(lda=15)), (-9, dict(D=NUL)), (-10, dict(ldd=7)),
        (-12, dict(C=NUL)), (-13, dict(ldc=7)), (-14, dict(sC=127)), (-15, dict(dt=3)),
        (-16, dict(cdt=1)), (0, dict(K=0, C=NUL)), (0, dict(N=0, C=NUL))])


def test_grouped_swiglu_abi(L):
    order = "E off A W Y M N K dt alpha scale st".split()
    base = dict(E=2, off=P, A=P, W=P, Y=P, M=4, N=8, K=16, dt=2, alpha=1.0, scale=NUL, st=NUL)
    expect(L.sg_grouped_swiglu_gemm, order, base, [
        (-1, dict(E=0)), (-2, dict(off=NUL)), (-3, dict(A=NUL)), (-4, dict(W=NUL)), (-5, dict(Y=NUL)),
        (-6, dict(M=-1)), (-7, dict(N=-1)), (-8, dict(K=-1)), (-9, dict(dt=0)),
        (-10, dict(alpha=2.0)), (-10, dict(dt=3, alpha=0.0)), (-10, dict(dt=3, alpha=float("nan"))),
        (-11, dict(scale=P)), (0, dict(M=0)), (0, dict(N=0))])
    order = "E off A W dY dH M N K dt st".split()
    base = dict(E=2, off=P, A=P, W=P, dY=P, dH=P, M=4, N=8, K=16, dt=2, st=NUL)
    expect(L.sg_grouped_swiglu_gemm_bwd, order, base, [
        (-1, dict(E=0)), (-2, dict(off=NUL)), (-3, dict(A=NUL)), (-4, dict(W=NUL)),
        (-5, dict(dY=NUL)), (-6, dict(dH=NUL)), (-7, dict(M=-1)), (-8, dict(N=-1)), (-9, dict(K=-1)),
        (-10, dict(dt=3)), (0, dict(M=0))])


def test_mxfp4_abi(L):
    order = "X ldx sX batch M K dt codes scales values st".split()
    base = dict(X=P, ldx=64, sX=0, batch=1, M=4, K=64, dt=2, codes=P, scales=P, values=NUL, st=NUL)
    expect(L.sg_mxfp4_quantize, order, base, [
        (-1, dict(X=NUL)), (-2, dict(ldx=63)), (-3, dict(sX=-1)), (-4, dict(batch=-1)),
        (-4, dict(batch=65536)), (-5, dict(M=-1)), (-6, dict(K=-1)), (-7, dict(dt=3)),
        (-8, dict(codes=NUL, scales=NUL)), (-8, dict(codes=ODD)), (-9, dict(scales=ODD)),
        (0, dict(M=0)), (0, dict(K=0)), (0, dict(batch=0))])
    order = "codes scales batch M K X ldx sX dt st".split()
    base = dict(codes=P, scales=P, batch=2, M=4, K=64, X=P, ldx=64, sX=256, dt=2, st=NUL)
    expect(L.sg_mxfp4_dequantize, order, base, [
        (-1, dict(codes=NUL)), (-1, dict(codes=ODD)), (-2, dict(scales=NUL)), (-3, dict(batch=-1)),
        (-4, dict(M=-1)), (-5, dict(K=-1)), (-6, dict(X=NUL)), (-7, dict(ldx=63)),
        (-8, dict(sX=255)), (-9, dict(dt=3)), (0, dict(M=0))])
    order = "src ld stride batch M nb dst st".split()
    base = dict(src=P, ld=4, stride=16, batch=1, M=4, nb=4, dst=P, st=NUL)
    expect(L.sg_mxfp4_tile_scales, order, base, [
        (-1, dict(src=NUL)), (-2, dict(ld=3)), (-3, dict(stride=-1)), (-4, dict(batch=-1)),
        (-5, dict(M=-1)), (-6, dict(nb=-1)), (-7, dict(dst=NUL)), (-7, dict(dst=ODD)),
        (0, dict(M=0))])
    order = "E off M N K alpha A As B Bs C ldc dt st".split()
    base = dict(E=1, off=NUL, M=4, N=8, K=64, alpha=1.0, A=P, As=P, B=P, Bs=P, C=P, ldc=8, dt=2,
                st=NUL)
    expect(L.sg_mxfp4_gemm, order, base, [
        (-1, dict(E=0)), (-2, dict(E=2)), (-3, dict(M=-1)), (-4, dict(N=-1)), (-5, dict(K=-1)),
        (-7, dict(A=NUL)), (-7, dict(A=ODD)), (-8, dict(As=NUL)), (-8, dict(As=ODD)),
        (-9, dict(B=NUL)), (-9, dict(B=ODD)), (-10, dict(Bs=NUL)), (-11, dict(C=NUL)),
        (-12, dict(ldc=7)), (-13, dict(dt=3)), (0, dict(M=0))])
    order = "E off M N K A As W Ws Y dt st".split()
    base = dict(E=1, off=NUL, M=4, N=8, K=64, A=P, As=P, W=P, Ws=P, Y=P, dt=2, st=NUL)
    expect(L.sg_mxfp4_swiglu_gemm, order, base, [
        (-1, dict(E=0)), (-2, dict(E=2)), (-3, dict(M=-1)), (-4, dict(N=-1)), (-5, dict(K=-1)),
        (-6, dict(A=ODD)), (-7, dict(As=NUL)), (-8, dict(W=NUL)), (-9, dict(Ws=ODD)),
        (-10, dict(Y=NUL)), (-11, dict(dt=0)), (0, dict(N=0))])


# ------------------------------------------------------------------ the binding
def t(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def off(n, dtype=torch.int32):
    return torch.zeros(n, dtype=dtype)


def raises(exc, match, fn, *a, **k):
    with pytest.raises(exc, match=match):
        fn(*a, **k)


def test_grouped_gemm_binding():
    g = sg.grouped_gemm
    A, B, C, o = t(8, 16), t(3, 16, 4), t(8, 4), off(4)
    raises(ValueError, ON_GPU, g, A, B, C, o)
    raises(ValueError, ON_GPU, g, A, t(3, 4, 16), C, o, transB="T", scale=t(3, dtype=F32))
    raises(ValueError, ON_GPU, g, t(8, 16, dtype=F8), t(3, 16, 4, dtype=F8), C, o)
    raises(ValueError, ON_GPU, g, t(8, 24)[:, :16], t(3, 20, 8)[:, :16, :4], t(8, 6)[:, :4], o)
    raises(ValueError, ON_GPU, g, A, t(1, 16, 4).expand(3, 16, 4), C, o)
    raises(TypeError, "bf16, fp16 or e4m3", g, t(8, 16, dtype=F32), t(3, 16, 4, dtype=F32), C, o)
    raises(TypeError, "A's dtype", g, A, t(3, 16, 4, dtype=F16), C, o)
    raises(TypeError, "C has dtype", g, A, B, t(8, 4, dtype=F16), o)
    raises(ValueError, "transB", g, A, B, C, o, transB="X")
    raises(ValueError, "2-D", g, t(16), B, C, o)
    raises(ValueError, "3-D", g, A, t(16, 4), C, o)
    raises(ValueError, "as rows", g, A, t(3, 15, 4), C, o)
    raises(ValueError, "expected rows of 4", g, A, B, t(8, 5), o)
    raises(ValueError, "rows, A", g, A, B, t(7, 4), o)
    raises(ValueError, "stride 1", g, t(16, 8).t(), B, C, o)
    raises(ValueError, "stride 1", g, A, t(3, 4, 16).transpose(1, 2), C, o)
    raises(ValueError, "overlap", g, A, B, t(1, 4).expand(8, 4), o)
    raises(TypeError, "int32", g, A, B, C, off(4, torch.int64))
    raises(ValueError, "experts \\+ 1", g, A, B, C, off(3))
    raises(ValueError, "experts \\+ 1", g, A, B, C, off(8)[::2])
    raises(TypeError, "float32", g, A, B, C, o, scale=t(3))
    raises(ValueError, "factors", g, A, B, C, o, scale=t(2, dtype=F32))


def test_grouped_wgrad_binding():
    g = sg.grouped_gemm_wgrad
    A, D, C, o = t(8, 16), t(8, 4), t(3, 16, 4), off(4)
    raises(ValueError, ON_GPU, g, A, D, C, o)
    raises(ValueError, ON_GPU, g, A, D, t(3, 16, 4, dtype=F32), o)
    raises(TypeError, "bf16 or fp16", g, t(8, 16, dtype=F8), t(8, 4, dtype=F8), C, o)
    raises(TypeError, "D must", g, A, t(8, 4, dtype=F16), C, o)
    raises(TypeError, "C has dtype", g, A, D, t(3, 16, 4, dtype=F16), o)
    raises(ValueError, "same rows", g, A, t(7, 4), C, o)
    raises(ValueError, "C has shape", g, A, D, t(3, 15, 4), o)
    raises(ValueError, "overlap", g, A, D, t(1, 16, 4).expand(3, 16, 4), o)
    raises(ValueError, "experts \\+ 1", g, A, D, C, off(3))


def test_grouped_swiglu_binding():
    g, b = sg.grouped_swiglu_gemm, sg.grouped_swiglu_gemm_bwd
    A, W, Y, o = t(8, 16), t(3, 16, 10), t(8, 5), off(4)
    raises(ValueError, ON_GPU, g, A, W, Y, o)
    raises(ValueError, ON_GPU, b, A, W, Y, t(8, 10), o)
    raises(ValueError, "even", g, A, t(3, 16, 9), Y, o)
    raises(ValueError, "3-D", g, A, t(16, 10), Y, o)
    raises(ValueError, "Wfused has shape", g, A, t(3, 15, 10), Y, o)
    raises(ValueError, "contiguous", g, t(16, 8).t(), W, Y, o)
    raises(ValueError, "Y has shape", g, A, W, t(8, 4), o)
    raises(TypeError, "Y has dtype", g, A, W, t(8, 5, dtype=F16), o)
    raises(TypeError, "SwiGLU takes", g, t(8, 16, dtype=F32), t(3, 16, 10, dtype=F32), Y, o)
    raises(TypeError, "backward", b, t(8, 16, dtype=F8), t(3, 16, 10, dtype=F8), Y, t(8, 10), o)
    raises(ValueError, "dH has shape", b, A, W, Y, t(8, 5), o)
    raises(TypeError, "dY must", b, A, W, t(8, 5, dtype=F16), t(8, 10), o)
    raises(ValueError, "experts \\+ 1", b, A, W, Y, t(8, 10), off(5))


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def test_mxfp4_binding():
    q, d = sg.mxfp4_quantize, sg.mxfp4_dequantize
    assert sg.mxfp4_shapes(33, 260) == (144, 1024)
    raises(ValueError, ON_GPU, q, t(4, 64))
    raises(ValueError, ON_GPU, q, t(2, 4, 64), u8(2, 4, 32), u8(2, 256))
    raises(ValueError, ON_GPU, q, t(4, 64), values=t(4, 64))
    raises(TypeError, "fp32, fp16 or bf16", q, t(4, 64, dtype=F8))
    raises(ValueError, "2-D or 3-D", q, t(64))
    raises(ValueError, "codes has shape", q, t(4, 64), u8(4, 31))
    raises(TypeError, "uint8", q, t(4, 64), t(4, 32))
    raises(ValueError, "scales has shape", q, t(4, 64), u8(4, 32), u8(255))
    raises(TypeError, "X's dtype", q, t(4, 64), values=t(4, 64, dtype=F16))
    raises(ValueError, "values has shape", q, t(4, 64), values=t(4, 63))
    raises(ValueError, ON_GPU, d, u8(4, 32), u8(256), t(4, 64))
    raises(ValueError, "codes has shape", d, u8(4, 32), u8(256), t(4, 65))
    raises(ValueError, "scales has shape", d, u8(4, 32), u8(512), t(4, 64))
    raises(ValueError, "overlap", d, u8(2, 4, 32), u8(2, 256), t(1, 4, 64).expand(2, 4, 64))
    raises(ValueError, ON_GPU, sg.mxfp4_tile_scales, u8(4, 2))
    raises(TypeError, "uint8", sg.mxfp4_tile_scales, t(4, 2))


def test_mxfp4_product_binding():
    g, s, o = sg.mxfp4_gemm, sg.mxfp4_swiglu_gemm, off(4)
    A, As, B, Bs, C = u8(8, 32), u8(256), u8(40, 32), u8(512), t(8, 40)
    E, Es = u8(3, 40, 32), u8(3, 512)
    raises(ValueError, ON_GPU, g, A, As, B, Bs, C)
    raises(ValueError, ON_GPU, g, A, As, E, Es, t(8, 48, dtype=F32)[:, :40], offsets=o)
    raises(ValueError, ON_GPU, s, A, As, B, Bs, t(8, 20))
    raises(ValueError, ON_GPU, s, A, As, E, Es, t(8, 20, dtype=F16), offsets=o)
    raises(ValueError, "3-D", g, A, As, B, Bs, C, offsets=off(2))
    raises(ValueError, "2-D", g, A, As, E, Es, C)
    raises(ValueError, "of one length", g, A, As, u8(40, 48), Bs, C)
    raises(ValueError, "of one length", g, u8(8, 31), As, u8(40, 31), Bs, C)
    raises(ValueError, "scales has shape", g, A, u8(512), B, Bs, C)
    raises(ValueError, "codes has shape", g, A, As, u8(41, 32), Bs, C)
    raises(ValueError, "rows, A", g, A, As, B, Bs, t(7, 40))
    raises(TypeError, "fp32, fp16 or bf16", g, A, As, B, Bs, t(8, 40, dtype=F8))
    raises(TypeError, "fp16 or bf16", s, A, As, B, Bs, t(8, 20, dtype=F32))
    raises(ValueError, "contiguous", s, A, As, B, Bs, t(8, 24)[:, :20])
    raises(ValueError, "experts \\+ 1", g, A, As, E, Es, C, offsets=off(3))
