"""The routing operators against their definitions in 64 bits: the choice and its ties, biases,
groups, masks that leave nothing, NaN and infinities, gradients by the formula and by differences;
the sort and the rows to their places and back, at odd sizes, strides and empty places."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import routing_reference as ref
from experts_reference import check
from test_gpu_grouped import padded

FLOATS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import swiglu_gemm_amd as sg
    sg.lib()


def cuda(t):
    return None if t is None else t.cuda()


def logits(T, E, dtype, seed, size=2.0):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn(T, E, generator=g)).to(FLOATS[dtype]), g


def check_route(X, top_k, Xd=None, **how):
    import swiglu_gemm_amd as sg
    want, w, tol = ref.route(X, top_k, **how)
    dev = {k: cuda(v) if torch.is_tensor(v) else v for k, v in how.items()}
    ids, weights = sg.route_experts(X.cuda() if Xd is None else Xd, top_k, **dev)
    assert ids.dtype == torch.int32 and weights.dtype == torch.float32
    assert torch.equal(ids.cpu(), want), "ids"
    check(weights, w, tol, "weights")
    return want, w


SHAPES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (7, 60, 6), (130, 64, 8), (9, 128, 8), (5, 160, 6), (33, 256, 8),
          (2, 500, 64), (3, 1024, 33), (6, 100, 9), (5, 300, 17), (3, 200, 12)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype", sorted(FLOATS))
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_sizes(scoring, dtype, T, E, k):
    X, g = logits(T, E, dtype, 17 * E + T)
    bias = 0.3 * torch.randn(E, generator=g)
    print("route %s %s %d x %d, top %d" % (scoring, dtype, T, E, k), flush=True)
    for renormalize in (False, True):
        check_route(X, k, scoring=scoring, renormalize=renormalize)
        check_route(X, k, scoring=scoring, renormalize=renormalize, bias=bias, scale=2.5)


@pytest.mark.parametrize("E,groups,top_groups,k", [(8, 2, 1, 4), (8, 8, 3, 3), (60, 4, 2, 6), (64, 64, 9, 7),
                                                    (256, 8, 4, 8), (160, 8, 3, 6), (1024, 32, 4, 16),
                                                    (96, 3, 3, 5)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_groups(scoring, E, groups, top_groups, k):
    for dtype in ("f32", "bf16"):
        X, g = logits(21, E, dtype, E + groups)
        bias = 0.3 * torch.randn(E, generator=g)
        for top in (1, 2):
            for b in (None, bias):
                check_route(X, k, scoring=scoring, bias=b, groups=groups, top_groups=top_groups,
                            group_top=top)


def test_route_ties_go_to_the_lowest_index():
    g = torch.Generator().manual_seed(2)
    for E, k in ((8, 4), (64, 8), (256, 8), (300, 20)):
        X = torch.randint(-2, 3, (40, E), generator=g).float()
        X[0] = 0.0
        for dtype in FLOATS.values():
            for bias in (None, torch.zeros(E), torch.randint(0, 2, (E,), generator=g).float()):
                check_route(X.to(dtype), k, bias=bias)
                check_route(X.to(dtype), k, scoring="sigmoid", bias=bias, renormalize=False)
                if E % 4 == 0:
                    check_route(X.to(dtype), min(k, E // 4), bias=bias, groups=4, top_groups=2,
                                scoring="sigmoid")


def test_route_near_ties():
    """Scores that differ by less than fp32 shows, with a bias: compared in 64 bits."""
    g = torch.Generator().manual_seed(9)
    for scoring in ("softmax", "sigmoid"):
        X = 1.0 + torch.randint(0, 64, (200, 64), generator=g).float() * 2.0 ** -23
        check_route(X, 8, scoring=scoring, bias=torch.full((64,), 0.5))
        check_route(X, 8, scoring=scoring, bias=torch.full((64,), 0.5), groups=8, top_groups=4)
        # biases that undo the scores' differences
        s = torch.softmax(X[0].double(), 0) if scoring == "softmax" else torch.sigmoid(X[0].double())
        check_route(X, 8, scoring=scoring, bias=(1.0 - s).float())


def test_route_extremes():
    """Logits of the type's largest and lowest values, and scores that underflow."""
    for name, dtype in FLOATS.items():
        f = torch.finfo(dtype)
        X = torch.tensor([[f.min, f.min, 1.0, f.min], [f.max, 0.0, f.max, f.min], [f.min] * 4,
                          [-200.0, -300.0, -250.0, -1000.0], [60.0, 61.0, 100.0, 90.0]]).to(dtype)
        for k in (1, 3, 4):
            check_route(X, k)
            check_route(X, k, renormalize=False)
            check_route(X, k, scoring="sigmoid", renormalize=False)
        check_route(X[:3], 2, groups=2, top_groups=1)
        check_route(X[3:], 4, scoring="sigmoid")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_masks(scoring):
    X, g = logits(60, 24, "f32", 4)
    mask = torch.rand(60, generator=g) < 0.5
    Xn = X.clone()
    Xn[~mask] = NAN                               # rows of masked tokens are not read
    check_route(Xn, 4, scoring=scoring, mask=mask)
    check_route(Xn, 4, scoring=scoring, mask=torch.zeros(60, dtype=torch.bool))
    # experts taken out: some, all but two, all
    X[:20, ::2] = -INF
    X[20:40, 2:] = -INF
    X[40:] = -INF
    X[50, 7] = 1.0
    bias = 0.3 * torch.randn(24, generator=g)
    for renormalize in (False, True):
        for b in (None, bias):
            check_route(X, 4, scoring=scoring, bias=b, renormalize=renormalize)
            check_route(X, 4, scoring=scoring, bias=b, groups=6, top_groups=2, renormalize=renormalize)
    bias[3], bias[5] = -INF, NAN
    check_route(X, 4, scoring=scoring, bias=bias)


def test_route_nan_shows():
    import swiglu_gemm_amd as sg
    X, _ = logits(4, 40, "f32", 4)
    X[1, 3], X[2, 7], X[3] = NAN, INF, NAN
    X[1, 5] = -INF
    for how in (dict(), dict(renormalize=False), dict(groups=4, top_groups=2), dict(bias=torch.zeros(40))):
        ids, w = sg.route_experts(X.cuda(), 6, **{k: cuda(v) if torch.is_tensor(v) else v
                                                  for k, v in how.items()})
        ids, w = ids.cpu(), w.cpu()
        assert torch.isfinite(w[0]).all() and torch.isnan(w[1:]).all()
        for t in range(4):
            assert len(set(ids[t].tolist())) == 6 and (ids[t] >= 0).all() and (ids[t] < 40).all()
        assert 3 not in ids[1].tolist() and 5 not in ids[1].tolist() and ids[2, 0] == 7
    ids, w = sg.route_experts(X.cuda(), 6, scoring="sigmoid", renormalize=False)
    assert ids[2, 0] == 7 and w[2, 0] == 1.0 and torch.isnan(w[1]).all()


def test_route_rows_apart_and_given_outputs():
    import swiglu_gemm_amd as sg
    for dtype in FLOATS:
        X, _ = logits(37, 60, dtype, 6)
        for pad, shift in ((4, 0), (3, 1)):
            check_route(X, 6, padded(X, pad, shift))
    ids = torch.full((37, 6), 99, dtype=torch.int32, device="cuda:0")
    w = torch.full((37, 6), 99.0, device="cuda:0")
    a, b = sg.route_experts(X.cuda(), 6, ids=ids, weights=w)
    assert a is ids and b is w and torch.equal(ids.cpu(), ref.route(X, 6)[0])
    empty, _ = sg.route_experts(torch.zeros(0, 60, device="cuda:0"), 6)
    assert empty.shape == (0, 6)


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_backward(scoring, T, E, k):
    import swiglu_gemm_amd as sg
    for dtype in sorted(FLOATS):
        X, g = logits(T, E, dtype, E + T)
        dw = torch.randn(T, k, generator=g)
        ids = ref.route(X, k)[0]
        if T > 2:
            ids[1], ids[2, k // 2:] = -1, -1                  # a masked token, and a row partly empty
        for renormalize in (False, True):
            want, tol = ref.route_bwd(X, ids, dw, scoring, renormalize, 2.5)
            for pad in (0, 3):
                dX = padded(torch.full((T, E), 7.0).to(X.dtype), pad, 1 if pad else 0)
                sg.route_experts_bwd(padded(X, pad, 0), ids.cuda(), dw.cuda(), dX, scoring=scoring,
                                     renormalize=renormalize, scale=2.5)
                check(dX, want, tol, "%s %s" % (dtype, renormalize))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient_against_differences(scoring, renormalize):
    """dX against central differences of the kernel's own weights: a step h of one logit, with the
    choice as it was; off by h^2 / 6 of the third derivative (at most 1 for these scores, summed over
    k weights) and by the weights' rounding, 2^-20, over h."""
    import swiglu_gemm_amd as sg
    X, g = logits(6, 16, "f32", 8, 1.0)
    X = X.sort(1, descending=True).values - torch.arange(16) * 0.25   # no choice is near another
    k, h = 4, 2.0 ** -5
    dw = torch.randn(6, k, generator=g)
    how = dict(scoring=scoring, renormalize=renormalize)
    ids, _ = sg.route_experts(X.cuda(), k, **how)
    dX = sg.route_experts_bwd(X.cuda(), ids, dw.cuda(), torch.empty(6, 16, device="cuda:0"), **how).cpu()
    for e in range(16):
        ends = []
        for sign in (1, -1):
            Xs = X.clone()
            Xs[:, e] += sign * h
            i, w = sg.route_experts(Xs.cuda(), k, **how)
            assert torch.equal(i, ids)
            ends.append((w.cpu().double() * dw).sum(1))
        diff = (ends[0] - ends[1]) / (2 * h)
        bound = (h * h / 6 + 2.0 ** -20 / h) * dw.abs().sum(1)
        assert ((diff - dX[:, e]).abs() <= bound).all(), e


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_of_negative_logits(scoring):
    """Logits all far below zero: what a lane without a place holds must not pass for a logit."""
    import swiglu_gemm_amd as sg
    for T, E, k in ((5, 16, 4), (3, 64, 8), (4, 256, 8), (3, 300, 20)):
        X, g = logits(T, E, "f32", E)
        X -= 300.0 if scoring == "softmax" else 60.0
        dw = torch.randn(T, k, generator=g)
        for renormalize in (False, True):
            ids, _ = check_route(X, k, scoring=scoring, renormalize=renormalize)
            want, tol = ref.route_bwd(X, ids, dw, scoring, renormalize, 1.0)
            dX = sg.route_experts_bwd(X.cuda(), ids.cuda(), dw.cuda(), torch.empty(T, E, device="cuda:0"),
                                      scoring=scoring, renormalize=renormalize)
            check(dX, want, tol)


def test_route_backward_of_odd_ids():
    """The same expert twice, ids outside the experts, and a row that no place reads."""
    import swiglu_gemm_amd as sg
    X, g = logits(3, 10, "f32", 3)
    X[2] = NAN
    ids = torch.tensor([[4, 4, 1], [11, 2, -5], [-1, -1, 10]], dtype=torch.int32)
    dw = torch.randn(3, 3, generator=g)
    for scoring in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            want, tol = ref.route_bwd(X, ids, dw, scoring, renormalize, 1.0)
            dX = sg.route_experts_bwd(X.cuda(), ids.cuda(), dw.cuda(), torch.empty(3, 10, device="cuda:0"),
                                      scoring=scoring, renormalize=renormalize)
            check(dX, want, tol)
            assert (dX[2] == 0).all()


# ------------------------------------------------------------------ sort
@pytest.mark.parametrize("n,E", [(0, 3), (1, 1), (5, 4), (64, 64), (256, 64), (1000, 8), (1025, 300),
                                 (4096, 20), (5000, 60), (20000, 256), (70001, 7)])
def test_sort(n, E):
    import swiglu_gemm_amd as sg
    g = torch.Generator().manual_seed(n + E)
    print("sort %d places of %d experts" % (n, E), flush=True)
    for low, high in ((0, E), (-2, E + 2), (E // 2, E // 2 + 1), (-1, 0)):
        ids = torch.randint(low, high, (n,), generator=g, dtype=torch.int32)
        got = sg.sort_experts(ids.cuda(), E)
        for a, b, what in zip(got, ref.sort(ids, E), ("offsets", "order", "place")):
            assert a.dtype == torch.int32 and torch.equal(a.cpu(), b), what


def test_sort_shape_and_extreme_ids():
    import swiglu_gemm_amd as sg
    ids = torch.tensor([[2**31 - 1, 0], [-2**31, 65535], [65536, 65535]], dtype=torch.int32)
    offsets, order, place = sg.sort_experts(ids.cuda(), 65536)
    assert order[:3].tolist() == [1, 3, 5] and order[3:].tolist() == [-1] * 3
    assert place.tolist() == [[-1, 0], [-1, 1], [-1, 2]]
    assert offsets[0] == 0 and offsets[1] == 1 and offsets[65535] == 1 and offsets[65536] == 3


# ------------------------------------------------------------------ rows
ROWS = [(1, 1, 1), (3, 2, 7), (5, 4, 8), (17, 8, 130), (64, 2, 2048), (9, 3, 1001), (1, 8, 4104), (300, 6, 64)]


def places(T, k, M, seed, empty=0.2):
    g = torch.Generator().manual_seed(seed)
    p = torch.randperm(max(M, T * k), generator=g)[:T * k].view(T, k).to(torch.int32)
    p[torch.rand(T, k, generator=g) < empty] = -1
    if T > 1:
        p[T // 2] = -1                                       # a token without a place
    return p, g                                              # places from M on are empty too


@pytest.mark.parametrize("T,k,D", ROWS)
@pytest.mark.parametrize("dtype", sorted(FLOATS))
def test_spread(dtype, T, k, D):
    import swiglu_gemm_amd as sg
    M = T * k + 3
    place, g = places(T, k, M, T + D)
    X = torch.randn(T, D, generator=g).to(FLOATS[dtype])
    Y = torch.randn(M, D, generator=g).to(FLOATS[dtype])
    w = torch.randn(T, k, generator=g)
    for pad, shift in ((0, 0), (8, 8), (3, 1)):
        for weights in (None, w):
            got = padded(Y, pad, shift)
            sg.spread_rows(padded(X, pad, shift), place.cuda(), got, weights=cuda(weights))
            want = ref.spread(X, place, Y, weights)
            if weights is None:
                assert torch.equal(got.cpu(), want)
            else:
                # fp32 product, then the type's rounding: for fp32 the two are one
                check(got, want.double(), ref.U * want.double().abs() + 2 * ref.half_step(want.double(), X.dtype))
                rest = torch.ones(M, dtype=torch.bool)
                rest[place[(place >= 0) & (place < M)].long()] = False
                assert torch.equal(got.cpu()[rest], Y[rest])


@pytest.mark.parametrize("T,k,D", ROWS)
@pytest.mark.parametrize("dtype", sorted(FLOATS))
def test_combine_and_backward(dtype, T, k, D):
    import swiglu_gemm_amd as sg
    M = max(1, T * k - 2)                                    # some places fall outside Z
    place, g = places(T, k, M, T * D)
    place[0, 0] = 0 if not (place == 0).any() else place[0, 0]
    dt = FLOATS[dtype]
    Z, R, dO = (torch.randn(n, D, generator=g).to(dt) for n in (M, T, T))
    w = torch.randn(T, k, generator=g)
    empty = (place < 0) | (place >= M)
    wn = torch.where(empty, NAN, w)                          # weights of empty places do not count
    for pad, shift in ((0, 0), (8, 8), (3, 1)):
        Zd, pd = padded(Z, pad, shift), place.cuda()
        for weights, residual in ((None, None), (wn, None), (wn, R)):
            out = padded(torch.full((T, D), 7.0).to(dt), pad, shift)
            sg.combine_rows(Zd, pd, out, cuda(weights), None if residual is None else padded(R, pad, shift))
            check(out, *ref.combine(Z, place, weights, residual), "out")
        old = torch.randn(M, D, generator=g).to(dt)
        dZ, dw = padded(old, pad, shift), torch.full((T, k), 7.0, device="cuda:0")
        sg.combine_rows_bwd(padded(dO, pad, shift), Zd, pd, cuda(wn), dZ, dw)
        want, tol, want_w, tol_w = ref.combine_bwd(dO, Z, place, w)
        check(dZ, want, tol, "dZ")
        check(dw, want_w, tol_w, "dweights")
        rest = torch.isnan(want[:, 0])
        assert torch.equal(dZ.cpu()[rest], old[rest])
        only = padded(old, pad, shift)
        assert sg.combine_rows_bwd(dO.cuda(), Zd, pd, cuda(wn), dZ=only)[1] is None
        assert torch.equal(only, dZ)
        alone = sg.combine_rows_bwd(dO.cuda(), Zd, pd, cuda(wn), dweights=torch.empty_like(dw))[1]
        assert torch.equal(alone, dw)


@pytest.mark.parametrize("dtype", sorted(FLOATS))
def test_combine_onto_its_residual(dtype):
    """out may be the residual itself."""
    import swiglu_gemm_amd as sg
    T, k, D, M = 37, 3, 2500, 90
    place, g = places(T, k, M, 5)
    Z, R = (torch.randn(n, D, generator=g).to(FLOATS[dtype]) for n in (M, T))
    w = torch.randn(T, k, generator=g)
    out = R.cuda()
    sg.combine_rows(Z.cuda(), place.cuda(), out, w.cuda(), out)
    check(out, *ref.combine(Z, place, w, R), "out")


def test_rows_of_nothing():
    import swiglu_gemm_amd as sg
    dev = dict(device="cuda:0")
    place = torch.full((3, 2), -1, dtype=torch.int32, **dev)
    R = torch.randn(3, 16, **dev)
    out = sg.combine_rows(torch.empty(0, 16, **dev), place, torch.full((3, 16), 7.0, **dev))
    assert (out == 0).all()
    out = sg.combine_rows(torch.empty(0, 16, **dev), place, torch.full((3, 16), 7.0, **dev), residual=R)
    assert torch.equal(out, R)
    dw = sg.combine_rows_bwd(R, torch.empty(0, 16, **dev), place, torch.ones(3, 2, **dev),
                             dweights=torch.full((3, 2), 7.0, **dev))[1]
    assert (dw == 0).all()
    sg.spread_rows(torch.empty(0, 16, **dev), place[:0], R)
    sg.spread_rows(R, place, torch.empty(0, 16, **dev))


def test_gradient_of_spread_is_combine():
    """<dY, spread(X)> == <combine(dY), X>: on whole numbers both are exact."""
    import swiglu_gemm_amd as sg
    g = torch.Generator().manual_seed(1)
    place, _ = places(20, 4, 80, 5)
    X = torch.randint(-4, 5, (20, 96), generator=g).float()
    dY = torch.randint(-4, 5, (80, 96), generator=g).float()
    w = torch.randint(-2, 3, (20, 4), generator=g).float()
    for weights in (None, w.cuda()):
        Y = sg.spread_rows(X.cuda(), place.cuda(), torch.zeros(80, 96, device="cuda:0"), weights=weights)
        dX = sg.combine_rows(dY.cuda(), place.cuda(), torch.empty(20, 96, device="cuda:0"), weights=weights)
        assert (Y.cpu() * dY).sum() == (dX.cpu() * X).sum()
