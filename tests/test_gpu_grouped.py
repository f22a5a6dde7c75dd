"""Products grouped by expert against their definition in 64 bits: runs of rows of every
length (none, one, odd, longer than a tile), rows that belong to no expert, one expert and
many, both weight layouts, all operand types, padded and unaligned strides, alpha, beta and
the experts' scales."""
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import experts_reference as ref

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import swiglu_gemm_amd as sg
    sg.lib()


def out_of(dtype):
    return torch.bfloat16 if dtype == "e4m3" else DT[dtype]


def table(sizes, before=0):
    o = [before]
    for s in sizes:
        o.append(o[-1] + s)
    return torch.tensor(o, dtype=torch.int32)


def rand(shape, dtype, std, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(DT.get(dtype, dtype))


def padded(x, pad, shift=0):
    """x on the GPU as a view whose rows are `pad` elements longer and that starts `shift`
    elements into its storage; the padding is NaN (0x7f for e4m3)."""
    r, c = x.shape[-2:]
    lead = x.shape[:-2]
    n = r * (c + pad)
    for d in lead:
        n *= d
    buf = torch.full((n + shift,), float("nan"), dtype=torch.float32).to(x.dtype).to("cuda:0")
    v = buf[shift:].view(*lead, r, c + pad)[..., :c]
    v.copy_(x.to("cuda:0"))
    return v


SIZES = {
    "none": [0, 0, 0], "one": [1], "ones": [1] * 9, "ragged": [5, 0, 33, 1, 64, 0, 70],
    "long": [300, 0, 129], "many": [i % 4 for i in range(150)], "single": [257],
}


def run_gemm(dtype, trans, sizes, N, K, alpha=1.0, beta=0.0, scaled=False, pad=(0, 0, 0),
             shift=0, before=0, behind=0):
    import swiglu_gemm_amd as sg
    off = table(sizes, before)
    M, E = int(off[-1]) + behind, len(sizes)
    A, B = rand((M, K), dtype, 1.0, 1), rand((E, N, K) if trans == "T" else (E, K, N), dtype,
                                             max(K, 1) ** -0.5, 2)
    C = rand((M, N), out_of(dtype), 1.0, 3)
    scale = torch.rand(E, generator=torch.Generator().manual_seed(4)) + 0.5 if scaled else None
    Ad, Bd, Cd = padded(A, pad[0], shift), padded(B, pad[1], shift), padded(C, pad[2], shift)
    print("grouped_gemm %s %s N=%d K=%d %s" % (dtype, trans, N, K, sizes[:9]), flush=True)
    sg.grouped_gemm(Ad, Bd, Cd, off.cuda(), alpha=alpha, beta=beta, transB=trans,
                    scale=scale.cuda() if scaled else None)
    want, tol = ref.gemm_rows(A, B, off, trans, alpha, scale, C, beta, out_of(dtype))
    got = Cd.cpu()
    ref.check(got, want, tol)
    for rows in (slice(0, before), slice(M - behind, M)):
        assert torch.equal(got[rows].view(torch.int16), C[rows].view(torch.int16))
    if pad[2]:
        assert torch.isnan(torch.as_strided(Cd, (M, N + pad[2]), (N + pad[2], 1))[:, N:]).all()


@pytest.mark.parametrize("sizes", sorted(SIZES))
@pytest.mark.parametrize("trans", "NT")
@pytest.mark.parametrize("dtype", ["bf16", "f16", "e4m3"])
def test_gemm_row_counts(dtype, trans, sizes):
    run_gemm(dtype, trans, SIZES[sizes], 144, 96, scaled=dtype == "e4m3")


@pytest.mark.parametrize("N,K", [(1, 1), (8, 16), (129, 33), (136, 72), (320, 1040), (31, 200)])
@pytest.mark.parametrize("trans", "NT")
@pytest.mark.parametrize("dtype", ["bf16", "f16", "e4m3"])
def test_gemm_sizes(dtype, trans, N, K):
    run_gemm(dtype, trans, [3, 0, 140, 17], N, K)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("trans", "NT")
def test_gemm_alpha_beta_and_strangers(dtype, trans):
    run_gemm(dtype, trans, [40, 0, 90, 1], 160, 128, alpha=-0.5, beta=0.75, scaled=True, before=7,
             behind=9)


@pytest.mark.parametrize("pad,shift", [((16, 32, 8), 16), ((1, 3, 5), 1), ((16, 16, 3), 0)])
@pytest.mark.parametrize("dtype,trans", [("bf16", "N"), ("bf16", "T"), ("e4m3", "T")])
def test_gemm_strides(dtype, trans, pad, shift):
    run_gemm(dtype, trans, [20, 150, 0, 2], 144, 64, beta=0.5, pad=pad, shift=shift, behind=3)


@pytest.mark.parametrize("alpha,K", [(0.0, 32), (1.0, 0)])
@pytest.mark.parametrize("beta", [0.0, 0.5])
def test_gemm_without_products(alpha, K, beta):
    """alpha = 0 reads neither operand: infinities there leave no mark."""
    import swiglu_gemm_amd as sg
    off = table([2, 0, 3], 1)
    C = rand((8, 24), "bf16", 1.0, 3)
    Cd = C.cuda()
    A = torch.full((8, K), float("inf"), dtype=torch.bfloat16, device="cuda:0")
    B = torch.full((3, K, 24), float("nan"), dtype=torch.bfloat16, device="cuda:0")
    sg.grouped_gemm(A, B, Cd, off.cuda(), alpha=alpha, beta=beta)
    got = Cd.cpu()
    assert torch.equal(got[1:6], (beta * C[1:6].float()).bfloat16())
    assert torch.equal(got[:1], C[:1]) and torch.equal(got[6:], C[6:])


def test_gemm_beta_zero_does_not_read_c():
    import swiglu_gemm_amd as sg
    off = table([70, 3])
    A, B = rand((73, 64), "bf16", 1.0, 1), rand((2, 64, 40), "bf16", 0.1, 2)
    C = torch.full((73, 40), float("nan"), dtype=torch.bfloat16, device="cuda:0")
    sg.grouped_gemm(A.cuda(), B.cuda(), C, off.cuda())
    want, tol = ref.gemm_rows(A, B, off, "N", 1.0, None, None, 0.0, torch.bfloat16)
    ref.check(C, want, tol)


def test_gemm_one_weight_for_all_and_other_stream():
    import swiglu_gemm_amd as sg
    off = table([33, 60, 7])
    A, B = rand((100, 64), "f16", 1.0, 1), rand((1, 64, 48), "f16", 0.1, 2)
    Ad, Bd = A.cuda(), B.cuda().expand(3, 64, 48)
    C = torch.zeros(100, 48, dtype=torch.float16, device="cuda:0")
    offd = off.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sg.grouped_gemm(Ad, Bd, C, offd)
    side.synchronize()
    want, tol = ref.gemm_rows(A, B.expand(3, 64, 48), off, "N", 1.0, None, None, 0.0, torch.float16)
    ref.check(C, want, tol)


def test_gemm_infinite_rows_stay_in_their_rows():
    import swiglu_gemm_amd as sg
    off = table([40, 30])
    A, B = rand((70, 64), "bf16", 1.0, 1), rand((2, 64, 40), "bf16", 0.1, 2)
    A[39], A[41] = float("inf"), float("nan")
    C = torch.zeros(70, 40, dtype=torch.bfloat16, device="cuda:0")
    sg.grouped_gemm(A.cuda(), B.cuda(), C, off.cuda())
    clean = A.clone()
    clean[39], clean[41] = 0, 0
    want, tol = ref.gemm_rows(clean, B, off, "N", 1.0, None, None, 0.0, torch.bfloat16)
    got = C.cpu()
    assert not torch.isfinite(got[[39, 41]]).any()
    keep = [i for i in range(70) if i not in (39, 41)]
    ref.check(got[keep], want[keep], tol[keep])


# ------------------------------------------------------------------ weight gradient
def run_wgrad(dtype, out, sizes, N, K, alpha=1.0, beta=0.0, pad=(0, 0, 0), shift=0, before=0,
              behind=0):
    import swiglu_gemm_amd as sg
    off = table(sizes, before)
    M, E = int(off[-1]) + behind, len(sizes)
    A, D = rand((M, K), dtype, 1.0, 1), rand((M, N), dtype, 0.1, 2)
    odt = torch.float32 if out == "f32" else DT[dtype]
    C = rand((E, K, N), odt, 1.0, 3)
    Ad, Dd, Cd = padded(A, pad[0], shift), padded(D, pad[1], shift), padded(C, pad[2], shift)
    print("wgrad %s->%s N=%d K=%d %s" % (dtype, out, N, K, sizes[:9]), flush=True)
    sg.grouped_gemm_wgrad(Ad, Dd, Cd, off.cuda(), alpha=alpha, beta=beta)
    want, tol = ref.wgrad(A, D, off, alpha, C, beta, odt)
    ref.check(Cd.cpu(), want, tol)
    if pad[2]:
        whole = torch.as_strided(Cd, (E, K, N + pad[2]), (K * (N + pad[2]), N + pad[2], 1))
        assert torch.isnan(whole[..., N:]).all()


@pytest.mark.parametrize("sizes", sorted(SIZES))
@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("bf16", "same"), ("f16", "f32"),
                                       ("f16", "same")])
def test_wgrad_row_counts(dtype, out, sizes):
    run_wgrad(dtype, out, SIZES[sizes], 72, 136)


@pytest.mark.parametrize("N,K", [(1, 1), (8, 264), (129, 33), (264, 8), (7, 260)])
@pytest.mark.parametrize("out", ["f32", "same"])
def test_wgrad_sizes(out, N, K):
    run_wgrad("bf16", out, [3, 0, 140, 17], N, K, alpha=0.5, beta=-1.0, before=5, behind=6)


@pytest.mark.parametrize("pad,shift", [((16, 8, 8), 8), ((1, 3, 5), 1), ((8, 8, 3), 0)])
@pytest.mark.parametrize("out", ["f32", "same"])
def test_wgrad_strides(out, pad, shift):
    run_wgrad("f16", out, [20, 150, 0, 2], 144, 64, beta=0.5, pad=pad, shift=shift)


def test_wgrad_strangers_do_not_count():
    """NaN in rows of no expert leaves every gradient finite; alpha = 0 reads nothing."""
    import swiglu_gemm_amd as sg
    off = table([10, 0, 25], 3)
    A, D = rand((45, 64), "bf16", 1.0, 1), rand((45, 48), "bf16", 1.0, 2)
    for t in (A, D):
        t[:3], t[38:] = float("nan"), float("inf")
    C = torch.empty(3, 64, 48, device="cuda:0")
    sg.grouped_gemm_wgrad(A.cuda(), D.cuda(), C, off.cuda())
    want, tol = ref.wgrad(A, D, off, 1.0, None, 0.0, torch.float32)
    ref.check(C, want, tol)
    A.fill_(float("nan"))
    C.fill_(2.0)
    sg.grouped_gemm_wgrad(A.cuda(), D.cuda(), C, off.cuda(), alpha=0.0, beta=0.5)
    assert torch.equal(C, torch.ones_like(C))


# ------------------------------------------------------------------ SwiGLU
def run_swiglu(dtype, sizes, N, K, bwd=False, before=0, behind=0, alpha=1.0, scaled=False):
    import swiglu_gemm_amd as sg
    off = table(sizes, before)
    M, E = int(off[-1]) + behind, len(sizes)
    A, W = rand((M, K), dtype, 1.0, 1), rand((E, K, 2 * N), dtype, 1.5 * max(K, 1) ** -0.5, 2)
    scale = torch.rand(E, generator=torch.Generator().manual_seed(4)) + 0.5 if scaled else None
    odt = out_of(dtype)
    Y = rand((M, N), odt, 1.0, 3)
    print("swiglu%s %s N=%d K=%d %s" % (" bwd" if bwd else "", dtype, N, K, sizes[:9]), flush=True)
    if bwd:
        H = rand((M, 2 * N), odt, 1.0, 5)
        Hd = H.cuda()
        sg.grouped_swiglu_gemm_bwd(A.cuda(), W.cuda(), Y.cuda(), Hd, off.cuda())
        want, tol = ref.swiglu_bwd_rows(A, W, Y, off, odt)
        got, old = Hd.cpu(), H
    else:
        Yd = Y.cuda()
        sg.grouped_swiglu_gemm(A.cuda(), W.cuda(), Yd, off.cuda(), alpha=alpha,
                               scale=scale.cuda() if scaled else None)
        want, tol = ref.swiglu_rows(A, W, off, alpha, scale, odt)
        got, old = Yd.cpu(), Y
    ref.check(got, want, tol)
    for rows in (slice(0, before), slice(M - behind, M)):
        assert torch.equal(got[rows].view(torch.int16), old[rows].view(torch.int16))


@pytest.mark.parametrize("sizes", sorted(SIZES))
@pytest.mark.parametrize("dtype,bwd", [("bf16", False), ("f16", False), ("e4m3", False),
                                       ("bf16", True), ("f16", True)])
def test_swiglu_row_counts(dtype, bwd, sizes):
    run_swiglu(dtype, SIZES[sizes], 72, 96, bwd)


@pytest.mark.parametrize("N,K", [(1, 1), (8, 16), (65, 33), (68, 72), (160, 1040), (33, 200),
                                 (40, 0)])
@pytest.mark.parametrize("dtype,bwd", [("bf16", False), ("e4m3", False), ("f16", True)])
def test_swiglu_sizes(dtype, bwd, N, K):
    run_swiglu(dtype, [3, 0, 140, 17], N, K, bwd, before=2, behind=5)


def test_swiglu_e4m3_scales():
    run_swiglu("e4m3", [64, 0, 70, 5], 144, 128, alpha=0.5, scaled=True)


def test_swiglu_far_gates():
    """Gates at which e^-g overflows or vanishes: SiLU is 0 (or g), its slope 0 (or 1)."""
    import swiglu_gemm_amd as sg
    off = table([6])
    A = torch.zeros(6, 32, dtype=torch.bfloat16)
    A[:, 0] = torch.tensor([-1000.0, -100.0, -20.0, 20.0, 100.0, 1000.0])
    A[:, 1] = 1.0
    W = torch.zeros(1, 32, 16, dtype=torch.bfloat16)
    W[0, 0, 0::2] = 1.0                              # gate = A[:, 0]
    W[0, 1, 1::2] = 3.0                              # up = 3
    dY = torch.ones(6, 8, dtype=torch.bfloat16)
    Y, H = torch.empty(6, 8), torch.empty(6, 16)
    Y, H = (t.to(torch.bfloat16).cuda() for t in (Y, H))
    sg.grouped_swiglu_gemm(A.cuda(), W.cuda(), Y, off.cuda())
    sg.grouped_swiglu_gemm_bwd(A.cuda(), W.cuda(), dY.cuda(), H, off.cuda())
    y, t = ref.swiglu_rows(A, W, off, 1.0, None, torch.bfloat16)
    ref.check(Y, y, t)
    h, t = ref.swiglu_bwd_rows(A, W, dY, off, torch.bfloat16)
    ref.check(H, h, t)


# ------------------------------------------------------------------ together, as in a layer
def test_mixture_layer_training_step():
    """Route, gate/up SwiGLU, down projection, weighted sum; then backward through all of it.
    Gradients against autograd of the same layer in 64 bits on the stored 16-bit intermediate
    values, and the weights' gradient against differences of the 64-bit loss."""
    import swiglu_gemm_amd as sg
    T, E, k, K, N = 90, 6, 2, 64, 48
    g = torch.Generator().manual_seed(7)
    X = torch.randn(T, K, generator=g).bfloat16()
    Wf = (torch.randn(E, K, 2 * N, generator=g) * K ** -0.5).bfloat16()
    Wd = (torch.randn(E, N, K, generator=g) * N ** -0.5).bfloat16()
    logits = torch.randn(T, E, generator=g)
    logits[:, 4] = -100.0                                  # an expert nobody picks
    gate, idx = logits.softmax(1).topk(k)
    order = idx.flatten().argsort(stable=True)
    token = order // k
    off = torch.cat([torch.zeros(1, dtype=torch.long),
                     torch.bincount(idx.flatten(), minlength=E).cumsum(0)]).int()
    w = gate.flatten()[order][:, None]
    A = X[token]
    dOut = torch.randn(T, K, generator=g).bfloat16()
    # forward
    Ad, Wfd, Wdd, offd = A.cuda(), Wf.cuda(), Wd.cuda(), off.cuda()
    M = A.shape[0]
    new = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda:0")
    Y = sg.grouped_swiglu_gemm(Ad, Wfd, new(M, N), offd)
    Z = sg.grouped_gemm(Y, Wdd, new(M, K), offd)
    out = torch.zeros(T, K, device="cuda:0").index_add_(0, token.cuda(), Z.float() * w.cuda())
    # backward
    dZ = (dOut[token].float() * w).bfloat16()
    dZd = dZ.cuda()
    dY = sg.grouped_gemm(dZd, Wdd, new(M, N), offd, transB="T")
    dWd = sg.grouped_gemm_wgrad(Y, dZd, torch.empty(E, N, K, device="cuda:0"), offd)
    dH = sg.grouped_swiglu_gemm_bwd(Ad, Wfd, dY, new(M, 2 * N), offd)
    dA = sg.grouped_gemm(dH, Wfd, new(M, K), offd, transB="T")
    dWf = sg.grouped_gemm_wgrad(Ad, dH, torch.empty(E, K, 2 * N, device="cuda:0"), offd)

    def layer(a, wf, wd):
        ys, zs = [], []
        for e, p in enumerate(ref.parts(off)):
            h = a[p] @ wf[e]
            ys.append(torch.nn.functional.silu(h[:, 0::2]) * h[:, 1::2])
            zs.append(ys[-1] @ wd[e])
        return torch.cat(ys), torch.cat(zs)
    a, wf, wd = (t.double().requires_grad_() for t in (A, Wf, Wd))
    y, z = layer(a, wf, wd)
    z.backward(dZ.double())
    # Y, dY and dH are rounded to bf16 on the way (2^-8 each at most, relative to the value):
    # in the 2-norm a chain of n such roundings is off by at most n * 2^-8 of its largest link
    far = lambda x, ref_: float((x.double().cpu() - ref_).norm() / ref_.norm())
    eps = 2.0 ** -8
    assert far(Y, y.detach()) < 2 * eps
    assert far(Z, z.detach()) < 3 * eps
    want = torch.zeros(T, K, dtype=torch.float64).index_add_(0, token, z.detach() * w.double())
    assert far(out, want) < 3 * eps
    assert far(dWd, wd.grad) < 3 * eps
    assert far(dA, a.grad) < 4 * eps and far(dWf, wf.grad) < 4 * eps
    assert torch.count_nonzero(dWf[4]) == 0 and torch.count_nonzero(dWd[4]) == 0
    # differences: along a direction, the loss <z, dZ> changes by <dWf, direction>
    step = 1e-5
    d = torch.randn(wf.shape, generator=g, dtype=torch.float64)
    with torch.no_grad():
        up, down = (float((layer(a, wf + s * step * d, wd)[1] * dZ.double()).sum())
                    for s in (1, -1))
    slope = float((dWf.double().cpu() * d).sum())
    assert abs((up - down) / (2 * step) - slope) < 4 * eps * float(wf.grad.norm() * d.norm())


def test_calls_overlap_on_two_streams_and_replay_in_a_graph():
    """No workspace: two streams at once give the bits of one after the other; a captured call
    follows new offsets written to the same tensor."""
    import swiglu_gemm_amd as sg
    offs = [table([100, 0, 156]).cuda(), table([1, 255, 0]).cuda()]
    A, W = rand((256, 128), "bf16", 1.0, 1).cuda(), rand((3, 128, 512), "bf16", 0.1, 2).cuda()
    new = lambda: torch.zeros(256, 256, dtype=torch.bfloat16, device="cuda:0")
    alone = [sg.grouped_swiglu_gemm(A, W, new(), o) for o in offs]
    streams = [torch.cuda.Stream() for _ in offs]
    both = [new() for _ in offs]
    torch.cuda.synchronize()
    for _ in range(8):
        for s, o, y in zip(streams, offs, both):
            with torch.cuda.stream(s):
                sg.grouped_swiglu_gemm(A, W, y, o)
    torch.cuda.synchronize()
    for x, y in zip(alone, both):
        assert torch.equal(x, y)
    off, Y, C = offs[0].clone(), new(), torch.zeros(3, 128, 512, device="cuda:0")
    D = rand((256, 512), "bf16", 1.0, 5).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sg.grouped_swiglu_gemm(A, W, Y, off)
        sg.grouped_gemm_wgrad(A, D, C, off)
    for i in (0, 1, 0, 1):
        off.copy_(offs[i])
        Y.zero_()
        C.fill_(float("nan"))
        want = sg.grouped_gemm_wgrad(A, D, torch.empty_like(C), offs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, alone[i]) and torch.equal(C, want)


# ------------------------------------------------------------------ every tile
@pytest.fixture
def force():
    yield lambda cfg: os.environ.__setitem__("SG_FORCE_GROUPED", str(cfg))
    os.environ.pop("SG_FORCE_GROUPED", None)


def took(cfg):
    import swiglu_gemm_amd as sg
    return "cfg=%d " % cfg in sg.last_config()


LONG = [1, 0, 257, 64, 130]


@pytest.mark.parametrize("cfg", [0, 1, 3, 4, 5])
@pytest.mark.parametrize("dtype,trans", [("bf16", "N"), ("f16", "T")])
def test_every_tile_rows(force, cfg, dtype, trans):
    """Ragged runs, a K tail, N inside a chunk, C aligned and not, beta."""
    force(cfg)
    for N, K, pad, beta in ((328, 200, (0, 0, 0), 0.0), (260, 136, (8, 12 if trans == "N" else 8, 4), 0.5),
                            (300, 64, (8, 4 if trans == "N" else 8, 3), 0.0),
                            (512, 512, (0, 0, 0), 0.0)):
        run_gemm(dtype, trans, LONG, N, K, beta=beta, pad=pad, before=3, behind=5, scaled=True)
        assert took(cfg)
    run_swiglu(dtype, LONG, 164, 200, before=3, behind=5)
    assert took(cfg)
    run_swiglu(dtype, LONG, 256, 128)
    run_swiglu(dtype, LONG, 164, 200, bwd=True, before=3, behind=5)
    assert took(cfg)
    run_swiglu(dtype, LONG, 256, 128, bwd=True)


@pytest.mark.parametrize("cfg", [6, 7, 8])
@pytest.mark.parametrize("trans", "NT")
def test_every_tile_e4m3(force, cfg, trans):
    force(cfg)
    for N, K, pad in ((336, 208, (0, 0, 0)), (272, 144, (16, 16, 4))):
        run_gemm("e4m3", trans, LONG, N, K, pad=pad, before=3, behind=5, scaled=True, beta=0.5)
        assert took(cfg)
    run_swiglu("e4m3", LONG, 168, 208, before=3, behind=5, alpha=0.5, scaled=True)
    assert took(cfg)


@pytest.mark.parametrize("cfg", [2, 4, 5])
@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("f16", "same")])
def test_every_tile_depth(force, cfg, dtype, out):
    force(cfg)
    for N, K, pad, beta in ((328, 264, (0, 0, 0), 0.0), (260, 300, (4, 4, 4), 0.5),
                            (512, 512, (0, 0, 0), 0.0)):
        run_wgrad(dtype, out, LONG, N, K, beta=beta, pad=pad, before=3, behind=5)
        assert took(cfg)


# ------------------------------------------------------------------ what lies behind K, far offsets
@pytest.mark.parametrize("trans", "NT")
@pytest.mark.parametrize("K", [8, 72, 200])
def test_neighbours_behind_k_do_not_count(trans, K):
    """A partial K tile may be loaded whole: the next row of A, the next row or the next
    expert's weight come in with it.  NaN and infinities there leave no mark."""
    import swiglu_gemm_amd as sg
    off = table([64, 64, 64, 64])
    A, B = rand((256, K), "bf16", 1.0, 1), rand((4, 160, K) if trans == "T" else (4, K, 160), "bf16",
                                                0.1, 2)
    bad = torch.arange(256) % 2 == 1
    A[bad] = float("nan")
    B[1] = float("inf")
    B[3] = float("nan")
    C = torch.zeros(256, 160, dtype=torch.bfloat16, device="cuda:0")
    sg.grouped_gemm(A.cuda(), B.cuda(), C, off.cuda(), transB=trans)
    assert "cfg=-1" not in sg.last_config()
    got = C.cpu()
    clean = [r for r in range(256) if not bad[r] and r // 64 in (0, 2)]
    A[bad] = 0
    B[1], B[3] = 0, 0
    want, tol = ref.gemm_rows(A, B, off, trans, 1.0, None, None, 0.0, torch.bfloat16)
    ref.check(got[clean], want[clean], tol[clean])


def test_rows_past_32_bits():
    """Rows whose offset in A passes 2^31 elements, and an expert's weight that does."""
    import swiglu_gemm_amd as sg
    K, N, far = 2048, 64, (1 << 20) + 3
    off = table([far, 0, 70])
    M = far + 70
    A = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda:0")
    assert A.numel() > 1 << 31
    tail = rand((200, K), "bf16", 1.0, 1)
    A[-200:] = tail.cuda()
    stride = (1 << 30) + 64
    store = torch.zeros(2 * stride + K * N, dtype=torch.bfloat16, device="cuda:0")
    B = torch.as_strided(store, (3, K, N), (stride, N, 1))
    w = rand((3, K, N), "bf16", 0.02, 2)
    B.copy_(w.cuda())
    C = torch.ones(M, N, dtype=torch.bfloat16, device="cuda:0")
    sg.grouped_gemm(A, B, C, off.cuda())
    near = table([130, 0, 70])
    want, tol = ref.gemm_rows(tail, w, near, "N", 1.0, None, None, 0.0, torch.bfloat16)
    ref.check(C[-200:], want, tol)
    assert torch.count_nonzero(C[:-200]) == 0
    # the weight gradient sums the far rows
    G = torch.empty(3, K, N, device="cuda:0")
    D = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda:0")
    d = rand((200, N), "bf16", 1.0, 3)
    D[-200:] = d.cuda()
    sg.grouped_gemm_wgrad(A, D, G, off.cuda())
    want, tol = ref.wgrad(tail, d, near, 1.0, None, 0.0, torch.float32)
    ref.check(G, want, tol)


def test_offsets_that_do_not_ascend_stay_inside():
    """A bad table: unspecified rows, but only rows of C and whole calls (the offsets are cut to
    [0, M])."""
    import swiglu_gemm_amd as sg
    A, B = rand((100, 64), "bf16", 1.0, 1).cuda(), rand((3, 64, 48), "bf16", 0.1, 2).cuda()
    whole = torch.full((300, 48), 7.0, dtype=torch.bfloat16, device="cuda:0")
    for bad in ([0, 90, 20, 100], [-50, 40, 1 << 30, 100], [100, 50, 0, 0], [-(1 << 31), 5, -3, 99]):
        o = torch.tensor(bad, dtype=torch.int32, device="cuda:0")
        sg.grouped_gemm(A, B, whole[100:200], o)
        sg.grouped_gemm_wgrad(A, A[:, :48].contiguous(), torch.empty(3, 64, 48, device="cuda:0"), o)
        torch.cuda.synchronize()
        assert (whole[:100] == 7).all() and (whole[200:] == 7).all()


def test_factors_of_no_products_do_not_count():
    """alpha = 0 or K = 0 with infinite or NaN scales, and infinite alpha for an expert without
    rows: beta * C_old all the same."""
    import swiglu_gemm_amd as sg
    off = table([3, 0, 2]).cuda()
    inf = float("inf")
    C = torch.full((5, 24), 2.0, dtype=torch.bfloat16, device="cuda:0")
    scale = torch.tensor([inf, float("nan"), -inf], device="cuda:0")
    A, B = rand((5, 32), "bf16", 1.0, 1).cuda(), rand((3, 32, 24), "bf16", 1.0, 2).cuda()
    sg.grouped_gemm(A, B, C, off, alpha=0.0, beta=0.5, scale=scale)
    assert (C == 1).all()
    sg.grouped_gemm(A[:, :0].contiguous(), B[:, :0].contiguous(), C, off, alpha=inf, beta=0.5,
                    scale=scale)
    assert (C == 0.5).all()
    G = torch.full((3, 32, 24), 2.0, device="cuda:0")
    sg.grouped_gemm_wgrad(A, rand((5, 24), "bf16", 1.0, 3).cuda(), G, off, alpha=inf, beta=0.5)
    assert (G[1] == 1).all()


def test_a_bad_table_of_many_experts_stays_inside():
    import swiglu_gemm_amd as sg
    g = torch.Generator().manual_seed(3)
    A, B = rand((100, 64), "bf16", 1.0, 1).cuda(), rand((100, 64, 48), "bf16", 0.1, 2).cuda()
    whole = torch.full((300, 48), 7.0, dtype=torch.bfloat16, device="cuda:0")
    for _ in range(4):
        o = torch.randint(-(1 << 31), (1 << 31) - 1, (101,), generator=g).int().cuda()
        sg.grouped_gemm(A, B, whole[100:200], o)
        sg.grouped_gemm_wgrad(A, A[:, :48].contiguous(), torch.empty(100, 64, 48, device="cuda:0"), o)
        torch.cuda.synchronize()
        assert (whole[:100] == 7).all() and (whole[200:] == 7).all()
