"""Microscaled 4-bit floating point against its definition in 64 bits: quantisation bit for
bit (ties, saturation, subnormal and extreme scales, infinities, odd sizes, strides), its
inverse, the scales' tiles, and the products, plain and grouped by expert."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import experts_reference as ref
from test_gpu_grouped import SIZES, padded, table

FLOATS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import swiglu_gemm_amd as sg
    sg.lib()


def bits(t):
    return t.cpu().contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def check_quantize(X, Xd=None):
    import swiglu_gemm_amd as sg
    Xd = X.cuda() if Xd is None else Xd
    vals = torch.full(X.shape, 7.0, dtype=X.dtype, device="cuda:0")
    codes, scales = sg.mxfp4_quantize(Xd)
    sg.mxfp4_quantize(Xd, values=vals)
    back = sg.mxfp4_dequantize(codes, scales, torch.empty_like(vals))
    wc, ws, wv = ref.quantize(X)
    R, nb = ws.shape
    assert torch.equal(scales.cpu(), ref.tile_scales(ws))
    assert torch.equal(codes.cpu(), wc)
    want = wv.to(X.dtype)
    for got in (vals, back):
        got = got.cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        ok = ~torch.isnan(want)
        assert torch.equal(bits(got)[ok], bits(want)[ok])
    return codes, scales


@pytest.mark.parametrize("R,K", [(1, 1), (1, 32), (3, 31), (5, 33), (32, 256), (33, 260), (70, 520),
                                 (64, 1000)])
@pytest.mark.parametrize("dtype", sorted(FLOATS))
def test_quantize_sizes(dtype, R, K):
    g = torch.Generator().manual_seed(R * 1000 + K)
    X = torch.randn(R, K, generator=g) * torch.exp(2 * torch.randn(R, 1, generator=g))
    print("quantize %s %d x %d" % (dtype, R, K), flush=True)
    check_quantize(X.to(FLOATS[dtype]))


@pytest.mark.parametrize("dtype", sorted(FLOATS))
def test_quantize_every_border(dtype):
    """Every value between two codes, and its neighbours, at each position of t in [4, 8)."""
    mids = torch.tensor([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7],
                        dtype=torch.float64)
    eps = torch.finfo(FLOATS[dtype]).eps
    near = torch.cat([mids, mids * (1 + eps), mids * (1 - eps), -mids])
    rows = []
    for top in (4.0, 5.0, 6.0, 7.0, 7.9):
        v = near[near.abs() <= top]
        v = torch.cat([v, torch.zeros(-len(v) % 31)]).view(-1, 31)
        rows.append(torch.cat([torch.full((len(v), 1), top), v], 1))
    X = torch.cat(rows)
    for e in (-10, -2, 0, 3, 8):
        check_quantize((X * 2.0 ** e).to(FLOATS[dtype]))


@pytest.mark.parametrize("dtype", sorted(FLOATS))
def test_quantize_extreme_scales(dtype):
    """Blocks from the smallest numbers of the type to the largest; zeros; NaN and infinities."""
    f = torch.finfo(FLOATS[dtype])
    tops = [0.0, -0.0, f.smallest_normal * f.eps, f.smallest_normal / 2, f.smallest_normal,
            f.smallest_normal * 3, 1.0, f.max / 2, f.max, float("inf"), float("-inf"), float("nan")]
    g = torch.Generator().manual_seed(5)
    X = torch.zeros(len(tops), 96)
    X[:, 32:] = torch.randn(len(tops), 64, generator=g)
    for i, t in enumerate(tops):
        part = torch.rand(32, generator=g) * 2 - 1
        X[i, :32] = part * (t if abs(t) < 1e38 else 1.0) if t == t and abs(t) != float("inf") else part
        X[i, i] = t
    check_quantize(X.to(FLOATS[dtype]))


def test_quantize_rows_apart_and_batches():
    import swiglu_gemm_amd as sg
    g = torch.Generator().manual_seed(5)
    for pad, shift in ((8, 8), (3, 1)):
        X = torch.randn(40, 288, generator=g).bfloat16()
        check_quantize(X, padded(X, pad, shift))
        X3 = torch.randn(3, 40, 100, generator=g).bfloat16()
        codes, scales = sg.mxfp4_quantize(padded(X3, pad, shift))
        vals = torch.empty_like(X3, device="cuda:0")
        sg.mxfp4_quantize(padded(X3, pad, shift), values=vals)
        wide = padded(torch.zeros_like(X3), pad, shift)
        sg.mxfp4_dequantize(codes, scales, wide)
        for i in range(3):
            wc, ws, wv = ref.quantize(X3[i])
            assert torch.equal(codes[i].cpu(), wc)
            assert torch.equal(scales[i].cpu(), ref.tile_scales(ws))
            assert torch.equal(vals[i].double().cpu(), wv)
            assert torch.equal(wide[i].double().cpu(), wv)


def test_tile_scales():
    import swiglu_gemm_amd as sg
    g = torch.Generator().manual_seed(5)
    for R, nb in ((1, 1), (33, 9), (64, 8), (100, 31)):
        S = torch.randint(0, 256, (2, R, nb), generator=g, dtype=torch.uint8)
        got = sg.mxfp4_tile_scales(padded(S, 3))
        one = sg.mxfp4_tile_scales(S[0].cuda())
        for i in range(2):
            assert torch.equal(got[i].cpu(), ref.tile_scales(S[i]))
        assert torch.equal(one, got[0])


# ------------------------------------------------------------------ products
def random_mx(batch, R, K, seed, spread=6):
    """Codes, tiled scales and 64-bit values of `batch` matrices with scales 2^-spread .. 2^spread."""
    g = torch.Generator().manual_seed(seed)
    nb = -(-K // 32)
    codes = torch.randint(0, 256, (batch, R, nb * 16), generator=g, dtype=torch.uint8)
    if K % 32:
        keep = torch.arange(nb * 32) < K
        keep = keep[0::2].to(torch.uint8) * 15 + keep[1::2].to(torch.uint8) * 240
        codes &= keep
    s = torch.randint(127 - spread, 128 + spread, (batch, R, nb), generator=g).to(torch.uint8)
    tiles = torch.stack([ref.tile_scales(x) for x in s])
    return codes, tiles, ref.values(codes, s)


def run_product(sizes, N, K, out="bf16", swiglu=False, alpha=1.0, pad=0, before=0, behind=0,
                spread=6):
    """sizes: rows of each expert, or one number: no offsets."""
    import swiglu_gemm_amd as sg
    grouped = isinstance(sizes, list)
    off = table(sizes if grouped else [sizes], before)
    M, E = int(off[-1]) + behind, len(off) - 1
    odt = FLOATS[out]
    A, As, a = random_mx(1, M, K, 1, spread)
    B, Bs, b = random_mx(E, 2 * N if swiglu else N, K, 2, spread)
    g = torch.Generator().manual_seed(3)
    C = torch.randn(M, N, generator=g).to(odt)
    Cd = padded(C, pad)
    dev = [t.cuda() for t in (A[0], As[0], B if grouped else B[0], Bs if grouped else Bs[0])]
    print("mx %s %s N=%d K=%d %s" % ("swiglu" if swiglu else "gemm", out, N, K, sizes), flush=True)
    offd = off.cuda() if grouped else None
    if swiglu:
        sg.mxfp4_swiglu_gemm(*dev, Cd, offsets=offd)
    else:
        sg.mxfp4_gemm(*dev, Cd, offsets=offd, alpha=alpha)
    want = torch.full((M, N), float("nan"), dtype=torch.float64)
    tol = want.clone()
    for e, p in enumerate(ref.parts(off)):
        if swiglu:
            want[p], tol[p] = ref.swiglu(*ref.gate_up(a[0, p], b[e].t()), odt)
        else:
            s, err = ref.matmul(a[0, p], b[e].t())
            want[p] = alpha * s
            tol[p] = abs(alpha) * (err + 2 * ref.STEP * s.abs()) + ref.half_step(alpha * s, odt)
    got = Cd.cpu()
    ref.check(got, want, tol)
    for rows in (slice(0, before), slice(M - behind, M)):
        assert torch.equal(bits(got[rows]), bits(C[rows]))
    if pad:
        assert torch.isnan(torch.as_strided(Cd, (M, N + pad), (N + pad, 1))[:, N:]).all()


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 40, 32), (7, 130, 96), (33, 129, 256),
                                   (64, 256, 512), (200, 300, 800), (130, 72, 33), (300, 520, 1056)])
@pytest.mark.parametrize("out", sorted(FLOATS))
def test_gemm_sizes(out, M, N, K):
    run_product(M, N, K, out, alpha=0.25, spread=1 if out == "f16" else 6)


@pytest.mark.parametrize("sizes", sorted(SIZES))
@pytest.mark.parametrize("swiglu", [False, True])
def test_grouped_row_counts(sizes, swiglu):
    run_product(SIZES[sizes], 72, 320, swiglu=swiglu, before=3, behind=5, spread=1)


@pytest.mark.parametrize("N,K", [(1, 32), (65, 96), (64, 256), (136, 544), (40, 2048)])
@pytest.mark.parametrize("out", ["bf16", "f16"])
def test_swiglu_sizes(out, N, K):
    run_product(90, N, K, out, swiglu=True, spread=0)


@pytest.mark.parametrize("pad", [8, 3])
@pytest.mark.parametrize("out", sorted(FLOATS))
def test_gemm_rows_of_c_apart(out, pad):
    run_product([40, 0, 100], 132, 288, out, pad=pad, spread=1, behind=4)


@pytest.mark.parametrize("alpha,K", [(0.0, 64), (1.0, 0)])
def test_gemm_without_products(alpha, K):
    import swiglu_gemm_amd as sg
    nan = lambda *s: torch.full(s, 255, dtype=torch.uint8, device="cuda:0")
    nb, sa = sg.mxfp4_shapes(5, K)
    sb = sg.mxfp4_shapes(40, K)[1]
    C = torch.full((5, 40), float("nan"), device="cuda:0")
    sg.mxfp4_gemm(nan(5, nb), nan(sa), nan(40, nb), nan(sb), C, alpha=alpha)
    assert torch.count_nonzero(C) == 0


def test_nan_scale_reaches_its_row_and_column_only():
    import swiglu_gemm_amd as sg
    A, As, a = random_mx(1, 70, 320, 1)
    B, Bs, b = random_mx(1, 50, 320, 2)
    sa = ref.untile_scales(As[0], 70, 10)
    sb = ref.untile_scales(Bs[0], 50, 10)
    sa[40, 9], sb[3, 0] = 255, 255
    C = torch.zeros(70, 50, device="cuda:0")
    sg.mxfp4_gemm(A[0].cuda(), ref.tile_scales(sa).cuda(), B[0].cuda(), ref.tile_scales(sb).cuda(), C)
    got = C.cpu()
    assert torch.isnan(got[40]).all() and torch.isnan(got[:, 3]).all()
    rows, cols = [i for i in range(70) if i != 40], [i for i in range(50) if i != 3]
    s, err = ref.matmul(a[0][rows], b[0][cols].t())
    ref.check(got[rows][:, cols], s, err + ref.half_step(s, torch.float32))


def test_padding_of_the_scales_is_not_read():
    """Rows and blocks outside the matrices: 255 in their bytes leaves no NaN."""
    import swiglu_gemm_amd as sg
    A, As, a = random_mx(1, 35, 288, 1)
    B, Bs, b = random_mx(1, 45, 288, 2)
    def fill(t, R):
        used = ref.tile_scales(torch.ones(R, 9, dtype=torch.uint8)) == 1
        return torch.where(used, t, 255).to(torch.uint8)
    C = torch.zeros(35, 45, device="cuda:0")
    sg.mxfp4_gemm(A[0].cuda(), fill(As[0], 35).cuda(), B[0].cuda(), fill(Bs[0], 45).cuda(), C)
    s, err = ref.matmul(a[0], b[0].t())
    ref.check(C, s, err + ref.half_step(s, torch.float32))


def test_mixture_layer_in_four_bits():
    """Quantise, gate/up SwiGLU, quantise, down projection, as a serving layer runs them; the
    second quantisation is checked from the first product's own output."""
    import swiglu_gemm_amd as sg
    off = table([20, 0, 45, 1])
    M, E, K, N = 66, 4, 160, 96
    g = torch.Generator().manual_seed(9)
    X = torch.randn(M, K, generator=g).bfloat16()
    W1, W2 = (torch.randn(E, N, K, generator=g) * K ** -0.5 for _ in range(2))
    Wf = torch.stack((W1, W2), 2).flatten(1, 2).bfloat16().cuda()
    Wd = (torch.randn(E, K, N, generator=g) * N ** -0.5).bfloat16().cuda()
    offd = off.cuda()
    qf, qd = sg.mxfp4_quantize(Wf), sg.mxfp4_quantize(Wd)
    Y = sg.mxfp4_swiglu_gemm(*sg.mxfp4_quantize(X.cuda()), *qf,
                             torch.empty(M, N, dtype=torch.bfloat16, device="cuda:0"), offsets=offd)
    Z = sg.mxfp4_gemm(*sg.mxfp4_quantize(Y), *qd, torch.empty(M, K, device="cuda:0"), offsets=offd)
    x, y = ref.quantize(X)[2], ref.quantize(Y.cpu())[2]
    for e, p in enumerate(ref.parts(off)):
        wf, wd = ref.quantize(Wf[e].cpu())[2], ref.quantize(Wd[e].cpu())[2]
        w, t = ref.swiglu(*ref.gate_up(x[p], wf.t()), torch.bfloat16)
        ref.check(Y[p], w, t)
        s, err = ref.matmul(y[p], wd.t())
        ref.check(Z[p], s, err + ref.half_step(s, torch.float32))


@pytest.mark.parametrize("cfg", range(4))
def test_every_tile(monkeypatch, cfg):
    """Ragged runs that start inside a tile of scales, rows that end in every block of a K tile,
    few and many K tiles."""
    import swiglu_gemm_amd as sg
    monkeypatch.setenv("SG_FORCE_MX4", str(cfg))
    sizes = [1, 0, 257, 64, 130]
    for nb in range(1, 18):
        run_product(sizes, 160, 32 * nb, spread=1, before=3, behind=5)
        assert "cfg=%d " % cfg in sg.last_config()
    run_product(sizes, 520, 2048, "f32", alpha=-0.5)
    run_product(300, 324, 1312, "f16", spread=0, pad=4)
    run_product(sizes, 164, 416, swiglu=True, spread=0, before=3, behind=5)
    run_product(260, 256, 1024, "f16", swiglu=True, spread=0)


def test_graph_and_two_streams():
    """Quantisation and product captured together follow new inputs and offsets; two streams at
    once give the bits of one after the other."""
    import swiglu_gemm_amd as sg
    offs = [table([100, 0, 156]).cuda(), table([1, 255, 0]).cuda()]
    g = torch.Generator().manual_seed(9)
    Xs = [torch.randn(256, 320, generator=g).bfloat16().cuda() for _ in range(2)]
    W = sg.mxfp4_quantize((torch.randn(3, 512, 320, generator=g) * 0.05).bfloat16().cuda())
    new = lambda: torch.zeros(256, 256, dtype=torch.bfloat16, device="cuda:0")
    run = lambda x, o, y: sg.mxfp4_swiglu_gemm(*sg.mxfp4_quantize(x), *W, y, offsets=o)
    alone = [run(x, o, new()) for x, o in zip(Xs, offs)]
    both, streams = [new(), new()], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(8):
        for s, x, o, y in zip(streams, Xs, offs, both):
            with torch.cuda.stream(s):
                run(x, o, y)
    torch.cuda.synchronize()
    assert torch.equal(both[0], alone[0]) and torch.equal(both[1], alone[1])
    X, off, Y = Xs[0].clone(), offs[0].clone(), new()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(X, off, Y)
    for i in (0, 1, 0, 1):
        X.copy_(Xs[i])
        off.copy_(offs[i])
        Y.zero_()
        assert torch.equal(run(Xs[i], offs[i], new()), alone[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, alone[i])


def test_quantize_past_32_bits():
    import swiglu_gemm_amd as sg
    R, K = (1 << 20) + 40, 2080
    X = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda:0")
    assert X.numel() > 1 << 31
    tail = torch.randn(72, K, generator=torch.Generator().manual_seed(1)).bfloat16()
    X[-72:] = tail.cuda()
    codes, scales = sg.mxfp4_quantize(X)
    wc, ws, wv = ref.quantize(tail)
    assert torch.equal(codes[-72:].cpu(), wc)
    nb = ws.shape[1]
    rows = scales.view(-1, (nb + 7) // 8 * 256)[-3:].flatten().cpu()     # the last 96 rows' tiles
    first = (R - 72) % 32                                  # the tail's first row in them
    assert torch.equal(ref.untile_scales(rows, first + 72, nb)[first:], ws)
    assert torch.count_nonzero(codes[:-72]) == 0
    B, Bs, b = random_mx(1, 64, K, 2, 1)
    C = torch.empty(R, 64, device="cuda:0")
    sg.mxfp4_gemm(codes, scales, B[0].cuda(), Bs[0].cuda(), C)
    s, err = ref.matmul(wv, b[0].t())
    ref.check(C[-72:], s, err + ref.half_step(s, torch.float32))


def test_far_scales_meet():
    """The smallest scales of one matrix against the largest of the other: the exponents add
    before anything is rounded away.  2^-127 * 2^127, codes up to 6: sums of at most 36 K."""
    import swiglu_gemm_amd as sg
    K = 320
    A, _, _ = random_mx(1, 40, K, 1)
    B, _, _ = random_mx(1, 72, K, 2)
    low = torch.arange(40 * 10).view(40, 10) % 3
    sa, sb = low.to(torch.uint8), (254 - torch.arange(72 * 10).view(72, 10) % 3).to(torch.uint8)
    for x, sx, y, sy in ((A, sa, B, sb), (A, 254 - sa, B, 254 - sb)):
        a, b = ref.values(x[0], sx), ref.values(y[0], sy)
        C = torch.empty(40, 72, device="cuda:0")
        sg.mxfp4_gemm(x[0].cuda(), ref.tile_scales(sx).cuda(), y[0].cuda(), ref.tile_scales(sy).cuda(), C)
        s, err = ref.matmul(a, b.t())
        ref.check(C, s, err + ref.half_step(s, torch.float32))
