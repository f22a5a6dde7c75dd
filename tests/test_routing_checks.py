"""What the routing operators and 4-bit integer weights refuse, without a GPU: the C ABI's argument
checks (before any HIP call) and the binding's (CPU tensors reach every check; a call that passes
all of them ends in the "must be on the GPU" error); and the references against closed forms."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import routing_reference as ref
import swiglu_gemm_amd as sg
from swiglu_gemm_amd import build as sgbuild
from test_experts_checks import expect

ON_GPU = "on the GPU"
P, ODD, NUL = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1001), ctypes.c_void_p(0)
BF, F16, F8, F32, I32, U8 = (torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.float32,
                             torch.int32, torch.uint8)


@pytest.fixture(scope="module")
def L():
    if sgbuild.is_stale():
        sgbuild.build()
    return sg.lib()


def test_route_abi(L):
    order = "X ldx T E dt k how bias groups tg gt norm scale mask ids w st".split()
    base = dict(X=P, ldx=8, T=4, E=8, dt=0, k=2, how=0, bias=NUL, groups=1, tg=1, gt=2, norm=1,
                scale=1.0, mask=NUL, ids=P, w=P, st=NUL)
    expect(L.sg_route_experts, order, base, [
        (-1, dict(X=NUL)), (-2, dict(ldx=7)), (-3, dict(T=-1)), (-4, dict(E=0)),
        (-4, dict(E=1025, ldx=2000)), (-5, dict(dt=3)), (-6, dict(k=0)), (-6, dict(k=9)),
        (-6, dict(k=65, E=100, ldx=100)), (-7, dict(how=2)), (-9, dict(groups=0)), (-9, dict(groups=3)),
        (-9, dict(groups=128, E=128, ldx=128)), (-10, dict(groups=4, tg=5)), (-10, dict(tg=0)),
        (-11, dict(gt=3)), (-12, dict(norm=2)), (-13, dict(scale=float("inf"))), (-15, dict(ids=NUL)),
        (-16, dict(w=NUL)), (0, dict(T=0, X=NUL, ids=NUL, w=NUL))])
    order = "X ldx T E dt k how norm scale ids dw dX lddx st".split()
    base = dict(X=P, ldx=8, T=4, E=8, dt=0, k=2, how=0, norm=1, scale=1.0, ids=P, dw=P, dX=P, lddx=8,
                st=NUL)
    expect(L.sg_route_experts_bwd, order, base, [
        (-1, dict(X=NUL)), (-2, dict(ldx=7)), (-3, dict(T=-1)), (-4, dict(E=0)), (-5, dict(dt=3)),
        (-6, dict(k=9)), (-7, dict(how=-1)), (-8, dict(norm=-1)), (-9, dict(scale=float("nan"))),
        (-10, dict(ids=NUL)), (-11, dict(dw=NUL)), (-12, dict(dX=NUL)), (-13, dict(lddx=7)),
        (0, dict(T=0))])


def test_rows_abi(L):
    order = "ids n E off order place st".split()
    base = dict(ids=P, n=4, E=8, off=P, order=P, place=P, st=NUL)
    expect(L.sg_sort_experts, order, base, [
        (-1, dict(ids=NUL)), (-2, dict(n=-1)), (-2, dict(n=2**30 + 1)), (-3, dict(E=0)),
        (-3, dict(E=65537)), (-4, dict(off=NUL))])
    order = "X ldx T D dt place k w M Y ldy st".split()
    base = dict(X=P, ldx=8, T=4, D=8, dt=2, place=P, k=2, w=NUL, M=8, Y=P, ldy=8, st=NUL)
    expect(L.sg_spread_rows, order, base, [
        (-1, dict(X=NUL)), (-2, dict(ldx=7)), (-3, dict(T=-1)), (-4, dict(D=-1)), (-5, dict(dt=3)),
        (-6, dict(place=NUL)), (-7, dict(k=0)), (-9, dict(M=-1)), (-10, dict(Y=NUL)),
        (-11, dict(ldy=7)), (0, dict(T=0)), (0, dict(D=0, ldx=1, ldy=1)), (0, dict(M=0, X=NUL, Y=NUL))])
    order = "Z ldz M D T dt place k w R ldr out ldo st".split()
    base = dict(Z=P, ldz=8, M=8, D=8, T=4, dt=2, place=P, k=2, w=P, R=P, ldr=8, out=P, ldo=8, st=NUL)
    expect(L.sg_combine_rows, order, base, [
        (-1, dict(Z=NUL)), (-2, dict(ldz=7)), (-3, dict(M=-1)), (-4, dict(D=-1)), (-5, dict(T=-1)),
        (-6, dict(dt=3)), (-7, dict(place=NUL)), (-8, dict(k=0)), (-11, dict(ldr=7)),
        (-12, dict(out=NUL)), (-13, dict(ldo=7)), (0, dict(T=0)), (0, dict(D=0))])
    order = "dO lddo Z ldz M D T dt place k w dZ lddz dw st".split()
    base = dict(dO=P, lddo=8, Z=P, ldz=8, M=8, D=8, T=4, dt=2, place=P, k=2, w=P, dZ=P, lddz=8, dw=P,
                st=NUL)
    expect(L.sg_combine_rows_bwd, order, base, [
        (-1, dict(dO=NUL)), (-2, dict(lddo=7)), (-3, dict(Z=NUL)), (-4, dict(ldz=7)), (-5, dict(M=-1)),
        (-6, dict(D=-1)), (-7, dict(T=-1)), (-8, dict(dt=3)), (-9, dict(place=NUL)), (-10, dict(k=0)),
        (-11, dict(w=NUL)), (-13, dict(lddz=7)), (0, dict(T=0)), (0, dict(dZ=NUL, dw=NUL))])


def test_int4_abi(L):
    order = "W ldw sW batch N K dt g codes scales zeros sdt st".split()
    base = dict(W=P, ldw=64, sW=0, batch=1, N=4, K=64, dt=2, g=64, codes=P, scales=P, zeros=NUL, sdt=2,
                st=NUL)
    expect(L.sg_int4_quantize, order, base, [
        (-1, dict(W=NUL)), (-2, dict(ldw=63)), (-3, dict(sW=-1)), (-4, dict(batch=-1)),
        (-4, dict(batch=65536)), (-5, dict(N=-1)), (-6, dict(K=-1)), (-7, dict(dt=3)), (-8, dict(g=16)),
        (-9, dict(codes=NUL)), (-9, dict(codes=ODD)), (-10, dict(scales=ODD)), (-11, dict(zeros=ODD)),
        (-12, dict(sdt=0)), (0, dict(N=0)), (0, dict(batch=0))])
    order = "src ss sz batch N K g codes scales zeros st".split()
    base = dict(src=P, ss=P, sz=NUL, batch=1, N=4, K=64, g=64, codes=P, scales=P, zeros=NUL, st=NUL)
    expect(L.sg_int4_pack, order, base, [
        (-1, dict(src=NUL)), (-2, dict(ss=NUL)), (-2, dict(ss=ODD)), (-3, dict(sz=P)),
        (-3, dict(zeros=P)), (-4, dict(batch=-1)), (-5, dict(N=-1)), (-6, dict(K=-1)), (-7, dict(g=0)),
        (-8, dict(codes=ODD)), (-9, dict(scales=ODD)), (-10, dict(zeros=ODD, sz=P)), (0, dict(K=0))])
    order = "codes scales zeros sdt batch N K g W ldw sW dt st".split()
    base = dict(codes=P, scales=P, zeros=NUL, sdt=2, batch=2, N=4, K=64, g=32, W=P, ldw=64, sW=256, dt=0,
                st=NUL)
    expect(L.sg_int4_dequantize, order, base, [
        (-1, dict(codes=ODD)), (-2, dict(scales=NUL)), (-3, dict(zeros=ODD)), (-4, dict(sdt=3)),
        (-5, dict(batch=-1)), (-6, dict(N=-1)), (-7, dict(K=-1)), (-8, dict(g=96)), (-9, dict(W=NUL)),
        (-10, dict(ldw=63)), (-11, dict(sW=255)), (-12, dict(dt=3)), (0, dict(N=0))])
    order = "E off order k T M N K g alpha A lda codes scales zeros C ldc dt cdt st".split()
    base = dict(E=1, off=NUL, order=NUL, k=1, T=4, M=4, N=8, K=64, g=64, alpha=1.0, A=P, lda=64, codes=P,
                scales=P, zeros=NUL, C=P, ldc=8, dt=2, cdt=2, st=NUL)
    expect(L.sg_int4_gemm, order, base, [
        (-1, dict(E=0)), (-2, dict(E=2)), (-4, dict(k=0)), (-4, dict(k=2)), (-5, dict(T=3)),
        (-5, dict(T=-1, order=P)), (-5, dict(T=0, order=P)), (-6, dict(M=-1, T=-1)), (-7, dict(N=-1)),
        (-8, dict(K=-1)), (-9, dict(g=48)), (-11, dict(A=NUL)), (-12, dict(lda=63)),
        (-13, dict(codes=ODD)), (-14, dict(scales=ODD)), (-15, dict(zeros=ODD)), (-16, dict(C=NUL)),
        (-17, dict(ldc=7)), (-18, dict(dt=0)), (-19, dict(cdt=1)), (0, dict(M=0, T=0)), (0, dict(N=0))])
    order = "E off order k T M N K g A lda codes scales zeros Y ldy dt st".split()
    base = dict(E=1, off=NUL, order=NUL, k=1, T=4, M=4, N=8, K=64, g=64, A=P, lda=64, codes=P, scales=P,
                zeros=NUL, Y=P, ldy=8, dt=2, st=NUL)
    expect(L.sg_int4_swiglu_gemm, order, base, [
        (-1, dict(E=0)), (-2, dict(E=2)), (-4, dict(k=2)), (-5, dict(T=3)), (-6, dict(M=-1)),
        (-7, dict(N=-1)), (-7, dict(N=2**29 + 1)), (-8, dict(K=-1)), (-9, dict(g=48)), (-10, dict(A=NUL)),
        (-11, dict(lda=63)), (-12, dict(codes=NUL)), (-13, dict(scales=NUL)), (-14, dict(zeros=ODD)),
        (-15, dict(Y=NUL)), (-16, dict(ldy=7)), (-17, dict(dt=0)), (0, dict(M=0, T=0))])


def refuse(kind, text, fn, *args, **kw):
    with pytest.raises(kind, match=text):
        fn(*args, **kw)


def test_route_binding():
    X = torch.zeros(4, 8)
    refuse(ValueError, ON_GPU, sg.route_experts, X, 2)
    refuse(TypeError, "fp32, fp16 or bf16", sg.route_experts, X.to(F8), 2)
    refuse(TypeError, "dtype", sg.route_experts, X.double(), 2)
    refuse(ValueError, "2-D", sg.route_experts, X[0], 2)
    refuse(ValueError, "scoring", sg.route_experts, X, 2, scoring="tanh")
    refuse(ValueError, "top_k", sg.route_experts, X, 0)
    refuse(ValueError, "top_k", sg.route_experts, X, 9)
    refuse(ValueError, "1024", sg.route_experts, torch.zeros(2, 1025), 2)
    refuse(ValueError, "groups", sg.route_experts, X, 2, groups=3)
    refuse(ValueError, "groups", sg.route_experts, X, 2, groups=4, top_groups=5)
    refuse(ValueError, "group_top", sg.route_experts, X, 2, group_top=0)
    refuse(TypeError, "bias", sg.route_experts, X, 2, bias=torch.zeros(8, dtype=BF))
    refuse(ValueError, "bias", sg.route_experts, X, 2, bias=torch.zeros(7))
    refuse(TypeError, "mask", sg.route_experts, X, 2, mask=torch.zeros(4))
    refuse(ValueError, "mask", sg.route_experts, X, 2, mask=torch.zeros(3, dtype=torch.bool))
    refuse(ValueError, "mask", sg.route_experts, X, 2, mask=torch.zeros(8, dtype=torch.bool)[::2])
    refuse(ValueError, "stride 1", sg.route_experts, torch.zeros(8, 4).t(), 2)
    refuse(ValueError, "overlap", sg.route_experts, torch.zeros(1, 8).expand(4, 8), 2)
    refuse(TypeError, "ids", sg.route_experts, X, 2, ids=torch.zeros(4, 2, dtype=torch.int64))
    refuse(ValueError, "weights", sg.route_experts, X, 2, weights=torch.zeros(4, 3))
    ids, g = torch.zeros(4, 2, dtype=I32), torch.zeros(4, 2)
    refuse(ValueError, ON_GPU, sg.route_experts_bwd, X, ids, g, torch.zeros(4, 8))
    refuse(TypeError, "dX", sg.route_experts_bwd, X, ids, g, torch.zeros(4, 8, dtype=BF))
    refuse(ValueError, "dX", sg.route_experts_bwd, X, ids, g, torch.zeros(3, 8))
    refuse(ValueError, "ids", sg.route_experts_bwd, X, ids[:3], g, torch.zeros(4, 8))
    refuse(ValueError, "dweights", sg.route_experts_bwd, X, ids, g[:3], torch.zeros(4, 8))
    refuse(ValueError, "scoring", sg.route_experts_bwd, X, ids, g, torch.zeros(4, 8), scoring="")


def test_rows_binding():
    ids = torch.zeros(4, 2, dtype=I32)
    refuse(ValueError, ON_GPU, sg.sort_experts, ids, 8)
    refuse(TypeError, "int32", sg.sort_experts, ids.long(), 8)
    refuse(ValueError, "experts", sg.sort_experts, ids, 0)
    refuse(ValueError, "contiguous", sg.sort_experts, torch.zeros(2, 4, dtype=I32).t(), 8)
    X, Y, w = torch.zeros(4, 16, dtype=BF), torch.zeros(8, 16, dtype=BF), torch.zeros(4, 2)
    refuse(ValueError, ON_GPU, sg.spread_rows, X, ids, Y)
    refuse(TypeError, "Y", sg.spread_rows, X, ids, Y.float())
    refuse(ValueError, "Y", sg.spread_rows, X, ids, Y[:, :8])
    refuse(ValueError, "tokens", sg.spread_rows, X, ids[:3], Y)
    refuse(ValueError, "2-D", sg.spread_rows, X, ids.flatten(), Y)
    refuse(TypeError, "place", sg.spread_rows, X, ids.long(), Y)
    refuse(ValueError, "weights", sg.spread_rows, X, ids, Y, weights=w[:3])
    refuse(TypeError, "fp32, fp16 or bf16", sg.spread_rows, X.to(F8), ids, Y.to(F8))
    refuse(ValueError, ON_GPU, sg.combine_rows, Y, ids, X, w, X)
    refuse(TypeError, "out", sg.combine_rows, Y, ids, X.half())
    refuse(TypeError, "weights", sg.combine_rows, Y, ids, X, w.half())
    refuse(TypeError, "residual", sg.combine_rows, Y, ids, X, w, X.float())
    refuse(ValueError, "residual", sg.combine_rows, Y, ids, X, w, X[:3])
    refuse(ValueError, "tokens", sg.combine_rows, Y, ids, X[:3])
    refuse(ValueError, "overlap", sg.combine_rows, Y, ids, X[:1].expand(4, 16))
    refuse(ValueError, ON_GPU, sg.combine_rows_bwd, X, Y, ids, w, Y, w)
    refuse(ValueError, "dZ", sg.combine_rows_bwd, X, Y, ids, w, Y[:7])
    refuse(TypeError, "dZ", sg.combine_rows_bwd, X, Y, ids, w, Y.float())
    refuse(ValueError, "dweights", sg.combine_rows_bwd, X, Y, ids, w, Y, w[:3])
    refuse(TypeError, "dOut", sg.combine_rows_bwd, X.half(), Y, ids, w)


def test_int4_binding():
    W = torch.zeros(40, 300, dtype=BF)
    refuse(ValueError, ON_GPU, sg.int4_quantize, W)
    refuse(ValueError, "group", sg.int4_quantize, W, group=16)
    refuse(TypeError, "scale_dtype", sg.int4_quantize, W.float())
    refuse(TypeError, "scale_dtype", sg.int4_quantize, W, scale_dtype=F32)
    refuse(TypeError, "fp32, fp16 or bf16", sg.int4_quantize, W.to(F8))
    raw, s = torch.zeros(40, 300, dtype=U8), torch.zeros(40, 3, dtype=BF)
    refuse(ValueError, ON_GPU, sg.int4_pack, raw, s)
    refuse(ValueError, "none of 32, 64 or 128", sg.int4_pack, raw, torch.zeros(40, 4, dtype=BF))
    refuse(TypeError, "uint8", sg.int4_pack, raw.int(), s)
    refuse(TypeError, "fp16 or bf16", sg.int4_pack, raw, s.float())
    refuse(ValueError, "zeros", sg.int4_pack, raw, s, torch.zeros(40, 2, dtype=U8))
    nc, ns = sg.int4_shapes(40, 300)
    assert (nc, ns) == (3 * 3 * 1024, 3 * 64) and sg.int4_shapes(40, 300, 32) == (nc, 3 * 3 * 64)
    codes, scales, zeros = torch.zeros(nc, dtype=U8), torch.zeros(ns, dtype=BF), torch.zeros(ns, dtype=U8)
    refuse(ValueError, ON_GPU, sg.int4_dequantize, codes, scales, W, zeros)
    refuse(ValueError, "codes", sg.int4_dequantize, codes[:-16], scales, W)
    refuse(ValueError, "scales", sg.int4_dequantize, codes, scales, W, group=32)
    A, C = torch.zeros(5, 300, dtype=BF), torch.zeros(5, 40, dtype=BF)
    refuse(ValueError, ON_GPU, sg.int4_gemm, A, codes, scales, C, zeros)
    refuse(TypeError, "fp16 or bf16", sg.int4_gemm, A.float(), codes, scales, C)
    refuse(TypeError, "scales", sg.int4_gemm, A, codes, scales.half(), C)
    refuse(TypeError, "C has", sg.int4_gemm, A, codes, scales, C.half())
    refuse(ValueError, "rows", sg.int4_gemm, A, codes, scales, C[:4])
    refuse(ValueError, "zeros", sg.int4_gemm, A, codes, scales, C, zeros[:64])
    refuse(ValueError, "codes", sg.int4_gemm, A[:, :100], codes, scales, C)
    order = torch.zeros(5, dtype=I32)
    refuse(TypeError, "order", sg.int4_gemm, A, codes, scales, C, order=order.long())
    refuse(ValueError, "order", sg.int4_gemm, A, codes, scales, C, order=order[:4])
    refuse(ValueError, "top_k", sg.int4_gemm, A, codes, scales, C, order=order, top_k=0)
    refuse(ValueError, "no rows", sg.int4_gemm, A[:0], codes, scales, C, order=order)
    off = torch.zeros(3, dtype=I32)
    refuse(ValueError, "2-D", sg.int4_gemm, A, codes, scales, C, offsets=off)
    refuse(ValueError, "row numbers", sg.int4_gemm, A, codes.expand(3, nc), scales, C, offsets=off)
    refuse(ValueError, "scales", sg.int4_gemm, A, torch.zeros(2, nc, dtype=U8), scales, C, offsets=off)
    Y = torch.zeros(5, 20, dtype=BF)
    refuse(ValueError, ON_GPU, sg.int4_swiglu_gemm, A, codes, scales, Y)
    refuse(TypeError, "Y has", sg.int4_swiglu_gemm, A, codes, scales, Y.float())
    refuse(ValueError, "codes", sg.int4_swiglu_gemm, A, codes, scales, C)


def test_reference_route_closed_forms():
    X = torch.tensor([[0.0, 1.0, 1.0, -1.0], [2.0, 2.0, 2.0, 2.0], [-float("inf")] * 4])
    ids, w, _ = ref.route(X, 3)
    assert ids.tolist() == [[1, 2, 0], [0, 1, 2], [-1, -1, -1]]
    e = torch.exp(torch.tensor(1.0, dtype=torch.float64))
    assert torch.allclose(w[0], torch.stack([e, e, e / e]) / (2 * e + 1))
    assert torch.allclose(w[1], torch.full((3,), 1 / 3, dtype=torch.float64)) and (w[2] == 0).all()
    bias = torch.tensor([0.0, -5.0, 0.0, 5.0])
    ids, w, _ = ref.route(X[:1], 2, "sigmoid", bias, renormalize=False, scale=2.0)
    assert ids.tolist() == [[3, 2]]
    assert torch.allclose(w[0], 2 * torch.sigmoid(torch.tensor([-1.0, 1.0], dtype=torch.float64)))
    ids, _, _ = ref.route(torch.tensor([[3.0, 0, 2, 2, 0, 1]]), 2, groups=3, top_groups=1)
    assert ids.tolist() == [[0, 1]]          # softmax scores: the group of the 3 outweighs 2 + 2
    ids, _, _ = ref.route(torch.tensor([[3.0, 0, 2.6, 2.6, 0, 1]]), 2, groups=3, top_groups=1)
    assert ids.tolist() == [[2, 3]]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_reference_route_gradient(scoring, renormalize):
    g = torch.Generator().manual_seed(3)
    X = torch.randn(3, 7, generator=g, dtype=torch.float64)
    ids = ref.route(X, 3)[0]
    dw = torch.randn(3, 3, generator=g, dtype=torch.float64)
    x = X.clone().requires_grad_(True)
    s = torch.softmax(x, 1) if scoring == "softmax" else torch.sigmoid(x)
    w = s.gather(1, ids.long())
    w = 1.7 * (w / w.sum(1, keepdim=True) if renormalize else w)
    w.backward(dw)
    got, _ = ref.route_bwd(X, ids, dw, scoring, renormalize, 1.7)
    assert torch.allclose(got, x.grad, atol=1e-12)


def test_reference_int4_layout_and_values():
    g = torch.Generator().manual_seed(4)
    for N, K, group in ((1, 1, 32), (17, 130, 64), (33, 300, 128)):
        n = -(-K // group)
        codes = torch.randint(0, 16, (N, K), generator=g, dtype=U8)
        scales = torch.rand(N, n, generator=g).bfloat16()
        zeros = torch.randint(0, 16, (N, n), generator=g, dtype=U8)
        packed, s, z = ref.int4_layout(codes, scales, zeros, group)
        assert (len(packed), len(s)) == sg.int4_shapes(N, K, group)
        for r, c in ((0, 0), (N - 1, K - 1), (N // 2, K // 3)):
            i = c % 8
            byte = 1024 * (r // 16 * -(-K // 128) + c // 128) + 16 * (16 * (c % 32 // 8) + r % 16)
            byte += 4 * (c % 128 // 32) + (i // 2 + 4 * (i % 2)) // 2
            nib = (i // 2) % 2
            assert int(packed[byte]) >> 4 * nib & 15 == int(codes[r, c])
    W = torch.tensor([[-7.0, 0.0, 3.5, 7.0]])
    codes, scales, _ = ref.int4_quantize(W, 32, False, F16)
    assert codes.tolist() == [[1, 8, 12, 15]] and scales.item() == 1.0
    codes, scales, zeros = ref.int4_quantize(torch.tensor([[-3.0, 0.0, 12.0]]), 32, True, F16)
    assert codes.tolist() == [[0, 3, 15]] and zeros.item() == 3
