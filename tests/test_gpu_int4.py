"""4-bit integer weights against their definition in 64 bits: quantisation and packing bit for bit,
the way back, and the products: every group size, with and without zero points, odd sizes, strides,
experts without rows, rows through `order`, values at the ends of the types."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import routing_reference as ref
from experts_reference import check
from test_gpu_grouped import padded

HALF = {"f16": torch.float16, "bf16": torch.bfloat16}
FLOATS = dict(HALF, f32=torch.float32)
INF, NAN = float("inf"), float("nan")
U8 = torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import swiglu_gemm_amd as sg
    sg.lib()


def cuda(t):
    return None if t is None else t.cuda()


def same(a, b):
    """Equal, NaN with NaN."""
    a = a.cpu()
    if a.is_floating_point():
        assert torch.equal(torch.isnan(a), torch.isnan(b))
        ok = ~torch.isnan(b)
        a, b = a[ok], b[ok]
    assert torch.equal(a, b)


def check_quantize(W, group, scale_dtype, Wd=None):
    import swiglu_gemm_amd as sg
    Wd = W.cuda() if Wd is None else Wd
    for zero_points in (False, True):
        codes, scales, zeros = ref.int4_quantize(W, group, zero_points, scale_dtype)
        want = ref.int4_layout(codes, scales, zeros, group)
        got = sg.int4_quantize(Wd, group, zero_points, scale_dtype)
        packed = sg.int4_pack(codes.cuda(), scales.cuda(), cuda(zeros))
        assert (got[2] is None) == (not zero_points) and (packed[2] is None) == (not zero_points)
        for a, b, c in zip(got, packed, want):
            if c is not None:
                same(a, c)
                same(b, c)
        values = ref.int4_values(codes, scales, zeros, group)
        for dtype in FLOATS.values():
            out = torch.full(W.shape, 7.0, dtype=dtype, device="cuda:0")
            sg.int4_dequantize(got[0], got[1], out, zeros=got[2], group=group)
            same(out, values.to(dtype))


@pytest.mark.parametrize("N,K", [(1, 1), (1, 32), (16, 128), (3, 31), (17, 130), (40, 300), (33, 520), (64, 1000)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize(group, N, K):
    g = torch.Generator().manual_seed(N * 1000 + K)
    W = torch.randn(N, K, generator=g) * torch.exp(torch.randn(N, 1, generator=g))
    print("int4 quantize %d x %d, groups of %d" % (N, K, group), flush=True)
    for dtype in FLOATS.values():
        for scale_dtype in HALF.values():
            check_quantize(W.to(dtype), group, scale_dtype)


def test_quantize_extremes():
    """Zeros, the smallest and largest numbers, one-sided groups, infinities and NaN; ties."""
    for dtype in FLOATS.values():
        f = torch.finfo(dtype)
        g = torch.Generator().manual_seed(7)
        tops = [0.0, f.smallest_normal * f.eps, f.smallest_normal, 1e-6, 1.0, f.max / 4, f.max, INF, -INF, NAN]
        W = torch.zeros(3 * len(tops), 64)
        for i, t in enumerate(tops):
            part = torch.rand(64, generator=g) * 2 - 1
            part = part * (t if abs(t) < 1e38 else 1.0) if t == t and abs(t) != INF else part
            W[3 * i], W[3 * i + 1], W[3 * i + 2] = part, part.abs(), -part.abs()
            W[3 * i: 3 * i + 3, 5] = t
        half = torch.arange(-16, 16).float() / 2                # ties at scale 1
        W = torch.cat([W, torch.cat([half, half]).clamp(-7, 7)[None], torch.full((1, 64), 3.0)])
        for scale_dtype in HALF.values():
            check_quantize(W.to(dtype), 32, scale_dtype)


def test_quantize_rows_apart_and_experts():
    import swiglu_gemm_amd as sg
    g = torch.Generator().manual_seed(5)
    W = torch.randn(3, 40, 200, generator=g).bfloat16()
    for pad, shift in ((8, 8), (3, 1)):
        got = sg.int4_quantize(padded(W, pad, shift), 64, True)
        wide = padded(torch.zeros_like(W), pad, shift)
        sg.int4_dequantize(got[0], got[1], wide, zeros=got[2], group=64)
        parts = [ref.int4_quantize(W[i], 64, True, torch.bfloat16) for i in range(3)]
        packed = sg.int4_pack(*(torch.stack(p).cuda() for p in zip(*parts)))
        for i in range(3):
            for a, b, c in zip(got, packed, ref.int4_layout(*parts[i], 64)):
                same(a[i], c)
                same(b[i], c)
            same(wide[i], ref.int4_values(*parts[i], 64).bfloat16())


def weight(g, N, K, group, dtype, zeros, size=None):
    """codes, scales and zeros of one weight; scales near K^-1/2."""
    n = -(-K // group)
    codes = torch.randint(0, 16, (N, K), generator=g, dtype=U8)
    scales = ((0.5 + torch.rand(N, n, generator=g)) * (K ** -0.5 / 4 if size is None else size)).to(dtype)
    scales[::3] *= -1
    return codes, scales, torch.randint(0, 16, (N, n), generator=g, dtype=U8) if zeros else None


def layouts(weights, group, lead):
    """The kernels' form of one weight for each expert, on the GPU."""
    parts = [ref.int4_layout(*w, group) for w in weights]
    out = [None if p[0] is None else torch.stack(p).cuda() for p in zip(*parts)]
    return out if lead else [None if p is None else p[0] for p in out]


def check_product(A, weights, group, offsets=None, order=None, top_k=1, M=None, pad=0, shift=0, alpha=1.0):
    """Both products (the second if N is even) of every output type against the definition."""
    import swiglu_gemm_amd as sg
    M = len(A) if M is None else M
    N = weights[0][0].shape[0]
    codes, scales, zeros = layouts(weights, group, offsets is not None)
    Ad = padded(A, pad, shift)
    kw = dict(zeros=zeros, group=group, offsets=cuda(offsets), order=cuda(order), top_k=top_k)
    for out_dtype in (A.dtype, torch.float32):
        want, tol = ref.int4_rows(A, weights, group, offsets, order, top_k, M, out_dtype, False, alpha)
        old = torch.full((M, N), 7.0).to(out_dtype)
        C = padded(old, pad, shift)
        sg.int4_gemm(Ad, codes, scales, C, alpha=alpha, **kw)
        check(C, want, tol, "gemm -> %s" % out_dtype)
        rest = torch.isnan(want).all(1)
        if offsets is not None:
            assert torch.equal(C.cpu()[rest], old[rest])
    if N % 2 == 0:
        want, tol = ref.int4_rows(A, weights, group, offsets, order, top_k, M, A.dtype, True)
        old = torch.full((M, N // 2), 7.0).to(A.dtype)
        Y = padded(old, pad, shift)
        sg.int4_swiglu_gemm(Ad, codes, scales, Y, **kw)
        check(Y, want, tol, "swiglu")
        if offsets is not None:
            assert torch.equal(Y.cpu()[rest], old[rest])


SIZES = [(1, 1, 1), (1, 16, 128), (1, 64, 1024), (2, 33, 130), (5, 100, 257), (16, 48, 512), (17, 66, 96),
         (31, 130, 1000), (33, 72, 384), (64, 16, 2050), (70, 258, 640), (130, 64, 160), (300, 96, 256)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", sorted(HALF))
def test_product_sizes(dtype, M, N, K):
    print("int4 %s %d x %d x %d" % (dtype, M, N, K), flush=True)
    for group in (32, 64, 128):
        for zeros in (False, True):
            g = torch.Generator().manual_seed(M * 7 + N + K)
            A = torch.randn(M, K, generator=g).to(HALF[dtype])
            check_product(A, [weight(g, N, K, group, HALF[dtype], zeros)], group, alpha=0.7)


@pytest.mark.parametrize("dtype", sorted(HALF))
def test_product_strides(dtype):
    g = torch.Generator().manual_seed(11)
    for M, N, K in ((3, 50, 136), (20, 34, 300), (100, 64, 129)):
        for pad, shift in ((8, 8), (4, 0), (3, 1)):
            A = torch.randn(M, K, generator=g).to(HALF[dtype])
            check_product(A, [weight(g, N, K, 64, HALF[dtype], True)], 64, pad=pad, shift=shift)


def runs(sizes, first=0, behind=0):
    offsets = [first]
    for s in sizes:
        offsets.append(offsets[-1] + s)
    return torch.tensor(offsets, dtype=torch.int32), offsets[-1] + behind


@pytest.mark.parametrize("sizes", [[1], [0, 0, 3], [1, 0, 5, 2], [16, 17, 0, 33], [0, 130, 1, 40, 7], [2] * 70])
@pytest.mark.parametrize("dtype", sorted(HALF))
def test_product_by_expert(dtype, sizes):
    g = torch.Generator().manual_seed(len(sizes) + sum(sizes))
    for (first, behind), (N, K, group) in zip(((0, 0), (3, 5)), ((50, 160, 32), (32, 260, 128))):
        offsets, M = runs(sizes, first, behind)
        print("int4 experts %s %s" % (dtype, sizes), flush=True)
        A = torch.randn(M, K, generator=g).to(HALF[dtype])
        A[:first], A[M - behind:] = NAN, NAN
        ws = [weight(g, N, K, group, HALF[dtype], len(sizes) % 2 == 0) for _ in sizes]
        check_product(A, ws, group, offsets)


@pytest.mark.parametrize("dtype", sorted(HALF))
def test_product_through_order(dtype):
    """Rows of tokens where they lie: each token at top_k experts, some places empty."""
    g = torch.Generator().manual_seed(3)
    for T, k, E in ((1, 2, 4), (9, 3, 5), (40, 8, 16)):
        ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
        ids[T // 2, 0] = -1
        offsets, order, _ = ref.sort(ids, E)
        A = torch.randn(T, 200, generator=g).to(HALF[dtype])
        ws = [weight(g, 36, 200, 64, HALF[dtype], True) for _ in range(E)]
        check_product(A, ws, 64, offsets, order, k, T * k)
    # without experts: any rows of A in any order
    order = torch.tensor([4, 0, 4, 2, 1], dtype=torch.int32)
    check_product(A[:5].clone(), ws[:1], 64, None, order, 1, 5)


def test_product_orders_outside_stay_inside():
    """Rows whose order is out of range are undefined, the others unharmed."""
    import swiglu_gemm_amd as sg
    g = torch.Generator().manual_seed(3)
    A = torch.randn(4, 64, generator=g).half()
    w = weight(g, 32, 64, 32, torch.float16, False)
    codes, scales, _ = layouts([w], 32, False)
    order = torch.tensor([0, -1, 2**31 - 1, 3, -2**31, 1], dtype=torch.int32)
    C = sg.int4_gemm(A.cuda(), codes, scales, torch.empty(6, 32, dtype=torch.float16, device="cuda:0"),
                     group=32, order=order.cuda())
    want, tol = ref.int4_rows(A, [w], 32, None, order.clamp(0, 3), 1, 6, torch.float16, False)
    for r in (0, 3, 5):
        check(C[r], want[r], tol[r])


def test_bad_offsets_stay_inside():
    """Tables that do not ascend, or leave the rows: nothing outside C is written."""
    import swiglu_gemm_amd as sg
    g = torch.Generator().manual_seed(3)
    A = torch.randn(20, 64, generator=g).bfloat16()
    ws = [weight(g, 32, 64, 32, torch.bfloat16, False) for _ in range(3)]
    codes, scales, _ = layouts(ws, 32, True)
    for table in ([0, 30, 10, 20], [-5, 3, 2**31 - 1, 7], [20, 10, 5, 0], [2**31 - 1] * 4, [-2**31] * 4):
        room = torch.full((40, 32), 7.0, dtype=torch.bfloat16, device="cuda:0")
        sg.int4_gemm(A.cuda(), codes, scales, room[10:30], group=32,
                     offsets=torch.tensor(table, dtype=torch.int32, device="cuda:0"))
        assert (room[:10] == 7).all() and (room[30:] == 7).all()


def test_values_at_the_ends():
    """Zero points above the codes, scales of 0 and NaN, activations near the types' ends."""
    g = torch.Generator().manual_seed(13)
    for dtype in HALF.values():
        codes, scales, zeros = weight(g, 32, 256, 64, dtype, True)
        zeros[0], zeros[1], scales[2] = 255, 16, 0.0
        A = torch.randn(6, 256, generator=g).to(dtype)
        A[0] = 0.0
        A[1] *= 2.0 ** -14 if dtype == torch.float16 else 2.0 ** -90
        A[2] *= 1000.0 if dtype == torch.float16 else 2.0 ** 100
        A[3, 1::2] = 0.0
        small = weight(g, 32, 256, 64, dtype, True, 2.0 ** -14)
        check_product(A, [(codes, (scales.double() * 2.0 ** -10).to(dtype), zeros)], 64)
        check_product(A, [small], 64)


def test_nan_stays_in_its_row_and_column():
    import swiglu_gemm_amd as sg
    g = torch.Generator().manual_seed(13)
    for dtype in HALF.values():
        w = weight(g, 40, 200, 64, dtype, True)
        w[1][7, 2] = NAN
        A = torch.randn(20, 200, generator=g).to(dtype)
        A[3, 150], A[11, 0] = NAN, INF
        codes, scales, zeros = layouts([w], 64, False)
        C = sg.int4_gemm(A.cuda(), codes, scales, torch.empty(20, 40, dtype=dtype, device="cuda:0"),
                         zeros=zeros, group=64).cpu()
        assert torch.isnan(C[3]).all() and torch.isnan(C[:, 7]).all() and not torch.isfinite(C[11]).any()
        C = C[[r for r in range(20) if r not in (3, 11)]]
        assert torch.isfinite(C[:, [c for c in range(40) if c != 7]]).all()


@pytest.mark.parametrize("cfg", range(9))
@pytest.mark.parametrize("group,K", [(128, 700), (32, 513), (64, 1280)])
def test_nan_stays_in_its_row_and_column_of_every_tile(group, K, cfg, monkeypatch):
    """Rows of NaN and infinity, a NaN scale in the last group: every other output is bit for bit what it
    is without them."""
    import swiglu_gemm_amd as sg
    monkeypatch.setenv("SG_FORCE_INT4", str(cfg))
    g = torch.Generator().manual_seed(K + cfg)
    M, N = 67, 141
    for dtype in HALF.values():
        w = weight(g, N, K, group, dtype, True)
        A = torch.randn(M, K, generator=g).to(dtype)
        outs = []
        for bad in (False, True):
            if bad:
                w[1][77, -1] = NAN
                A[3, K - 1], A[30, 0], A[64, K // 2] = NAN, INF, -INF
            codes, scales, zeros = layouts([w], group, False)
            outs.append(sg.int4_gemm(A.cuda(), codes, scales, torch.empty(M, N, dtype=dtype, device="cuda:0"),
                                     zeros=zeros, group=group).cpu())
        clean, C = outs
        rows = [r for r in range(M) if r not in (3, 30, 64)]
        columns = [c for c in range(N) if c != 77]
        assert torch.isnan(C[3]).all() and torch.isnan(C[:, 77]).all() and not torch.isfinite(C[[30, 64]]).any()
        assert torch.equal(C[rows][:, columns], clean[rows][:, columns])


def test_no_depth_and_no_rows():
    import swiglu_gemm_amd as sg
    dev = dict(device="cuda:0", dtype=torch.float16)
    none = torch.empty(0, device="cuda:0", dtype=U8), torch.empty(0, **dev)
    C = sg.int4_gemm(torch.empty(3, 0, **dev), *none, torch.full((3, 16), 7.0, **dev))
    assert (C == 0).all()
    nc, ns = sg.int4_shapes(16, 128)
    codes, scales = torch.zeros(nc, device="cuda:0", dtype=U8), torch.full((ns,), NAN, **dev)
    C = sg.int4_gemm(torch.full((3, 128), INF, **dev), codes, scales, torch.full((3, 16), 7.0, **dev), alpha=0.0)
    assert (C == 0).all()
    sg.int4_gemm(torch.empty(0, 128, **dev), codes, scales, torch.empty(0, 16, **dev))
    sg.int4_swiglu_gemm(torch.empty(0, 128, **dev), codes, scales, torch.empty(0, 8, **dev))


@pytest.mark.parametrize("cfg", range(9))
@pytest.mark.parametrize("dtype", sorted(HALF))
def test_every_tile(dtype, cfg, monkeypatch):
    """Each tile forced on sizes that end inside it: rows, columns, depth, runs and groups."""
    import swiglu_gemm_amd as sg
    monkeypatch.setenv("SG_FORCE_INT4", str(cfg))
    for M, N, K, group, zeros in ((1, 16, 128, 128, False), (70, 210, 1100, 64, True), (65, 130, 2304, 128, True),
                                  (16, 98, 4000, 32, False), (3, 34, 40, 32, True),
                                  (40, 50, 640, 128, True), (33, 60, 384, 64, False)):
        g = torch.Generator().manual_seed(M + N + K)
        A = torch.randn(M, K, generator=g).to(HALF[dtype])
        print("int4 tile %d %s %d x %d x %d" % (cfg, dtype, M, N, K), flush=True)
        check_product(A, [weight(g, N, K, group, HALF[dtype], zeros)], group)
        assert "cfg=%d" % cfg in sg.last_config()
    offsets, M = runs([5, 0, 64, 1, 130, 16], 2, 3)
    A = torch.randn(M, 200, generator=g).to(HALF[dtype])
    ws = [weight(g, 150, 200, 64, HALF[dtype], True) for _ in range(6)]
    check_product(A, ws, 64, offsets)


def test_the_choice_of_tiles():
    """One piece to a work-group, then more columns, then 32-row tiles in two parts along K, 64-row ones, and
    tiles that are whole along K, as the products grow."""
    import swiglu_gemm_amd as sg
    dev = dict(device="cuda:0", dtype=torch.bfloat16)
    for M, N, want in ((1, 4096, 0), (1, 8192, 1), (1, 11008, 2), (1, 16384, 3), (16, 22016, 4), (32, 1024, 0),
                       (256, 4096, 7), (512, 4096, 6), (256, 11008, 8), (512, 11008, 5)):
        nc, ns = sg.int4_shapes(N, 4096)
        sg.int4_gemm(torch.zeros(M, 4096, **dev), torch.zeros(nc, device="cuda:0", dtype=U8), torch.zeros(ns, **dev),
                     torch.empty(M, N, **dev))
        assert "cfg=%d " % want in sg.last_config(), (M, N, sg.last_config())
