"""The router's choice where a row has NaN logits, or with softmax infinite ones: the biases, those that
take an expert out among them, and the groups hold there as anywhere, and NaN logits come last.  The
weights of these rows are NaN, so the ids are all that can be compared, and they are exact."""
import pytest

torch = pytest.importorskip("torch")

INF, NAN = float("inf"), float("nan")
LAST = -1e300                                       # a group of NaN logits alone


def choice(X, top_k, scoring="softmax", bias=None, groups=1, top_groups=1, group_top=2):
    """(ids, whether the row's weights are NaN) row by row, in 64 bits."""
    T, E = X.shape
    per = E // groups
    ids = torch.full((T, top_k), -1, dtype=torch.int32)
    shows = torch.zeros(T, dtype=torch.bool)
    for t in range(T):
        x = X[t].double()
        nan = torch.isnan(x)
        shows[t] = nan.any() or (scoring == "softmax" and (x == INF).any())
        b = torch.zeros(E, dtype=torch.float64) if bias is None else bias.double()
        open_ = (x != -INF) & (b != -INF) & ~torch.isnan(b)
        n = torch.where(nan, -INF, x)                # the row without its NaN logits
        if scoring == "sigmoid":
            s = 1 / (1 + torch.exp(-n))
        elif (n == INF).any():
            s = (n == INF).double() / (n == INF).sum()
        else:
            s = torch.softmax(n, 0) if (n != -INF).any() else torch.zeros(E, dtype=torch.float64)
        c = s + b
        key = n if bias is None else c
        on = open_.clone()
        if groups > 1 and top_groups < groups:
            value = []
            for g in range(groups):
                at = [e for e in range(g * per, g * per + per) if open_[e]]
                best = sorted((float(c[e]) for e in at if not nan[e]), reverse=True)[:group_top]
                value.append(sum(best) if best else LAST if at else -INF)
            kept = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
            on &= torch.tensor([e // per in kept for e in range(E)])
        numbers = sorted((e for e in range(E) if on[e] and not nan[e]), key=lambda e: (-float(key[e]), e))
        pick = (numbers + [e for e in range(E) if on[e] and nan[e]])[:top_k]
        ids[t, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
    return ids, shows


def test_choice_closed_forms():
    X = torch.tensor([[1.0, NAN, 3.0, 2.0], [NAN] * 4, [INF, 5.0, INF, -INF]])
    ids, shows = choice(X, 4)
    assert ids.tolist() == [[2, 3, 0, 1], [0, 1, 2, 3], [0, 2, 1, -1]] and shows.all()
    bias = torch.tensor([0.0, 0.0, -INF, NAN])
    assert choice(X, 4, bias=bias)[0].tolist() == [[0, 1, -1, -1], [0, 1, -1, -1], [0, 1, -1, -1]]
    # sigmoid: 0.73 + 0.5 outweighs 0.95 and 0.88
    ids, shows = choice(X, 2, "sigmoid", bias=torch.tensor([0.5, 0.0, 0.0, 0.0]))
    assert ids[0].tolist() == [0, 2] and shows.tolist() == [True, True, False]
    # groups of two: of NaN alone behind one with a number, in front of one without any expert
    X = torch.tensor([[NAN, NAN, -9.0, NAN, -INF, -INF]])
    for top, want in ((1, [2, 3, -1]), (2, [2, 0, 1])):
        assert choice(X, 3, groups=3, top_groups=top)[0][0].tolist() == want


def check(X, k, **how):
    import swiglu_gemm_amd as sg
    want, shows = choice(X, k, **how)
    dev = {n: v.cuda() if torch.is_tensor(v) else v for n, v in how.items()}
    for renormalize in (True, False):
        ids, w = sg.route_experts(X.cuda(), k, renormalize=renormalize, **dev)
        assert torch.equal(ids.cpu(), want), "ids"
        w = w.cpu()
        assert (w[want < 0] == 0).all()
        assert torch.isnan(w[shows[:, None] & (want >= 0)]).all() and torch.isfinite(w[~shows]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("E,groups,top_groups,k", [(16, 4, 2, 4), (64, 8, 4, 8), (256, 8, 3, 8), (60, 4, 1, 8),
                                                   (96, 8, 8, 20), (300, 6, 2, 10), (1024, 16, 5, 33)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_choice_with_nan(scoring, E, groups, top_groups, k):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator().manual_seed(E + k)
    for dtype in (torch.float32, torch.bfloat16):
        X = torch.randn(24, E, generator=g)
        for t in range(1, 23):                       # the first and the last row are as usual
            some = torch.randperm(E, generator=g)
            X[t, some[:1 + t % 3]] = NAN
            if t % 4 == 1:
                X[t, some[3:3 + E // 2]] = -INF
            if t % 5 == 2:
                X[t, some[-1:]] = INF
            if t % 7 == 3:
                X[t, some[:E - 2]] = NAN             # two numbers are left
        X[20] = NAN
        X[21, :E // groups] = NAN                    # one group of NaN alone, the others without an expert
        X[21, E // groups:] = -INF
        X[22, :] = -INF
        X[22, E - 1] = NAN
        X = X.to(dtype)
        bias = torch.randn(E, generator=g)
        out = bias.clone()
        out[::3], out[1::5] = -INF, NAN
        print("route with NaN: %s, %d experts, %s" % (scoring, E, dtype), flush=True)
        for b in (None, torch.zeros(E), bias, out):
            check(X, k, scoring=scoring, bias=b)
            for top in (1, 2):
                check(X, k, scoring=scoring, bias=b, groups=groups, top_groups=top_groups, group_top=top)


@pytest.mark.gpu
@pytest.mark.parametrize("E,k", [(40, 4), (300, 10)])
def test_gradient_with_nan(E, k):
    """Renormalised and sigmoid gradients read the chosen logits alone; the softmax's own reads the row."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import routing_reference as ref
    from experts_reference import check
    import swiglu_gemm_amd as sg
    g = torch.Generator().manual_seed(E)
    X = torch.randn(6, E, generator=g)
    dw = torch.randn(6, k, generator=g)
    ids = ref.route(X, k)[0]
    bad = X.clone()
    for t in range(1, 6):
        free = [e for e in range(E) if e not in ids[t].tolist()]
        bad[t, free[t]] = NAN
    for scoring, renormalize in (("softmax", True), ("sigmoid", True), ("sigmoid", False), ("softmax", False)):
        dX = sg.route_experts_bwd(bad.cuda(), ids.cuda(), dw.cuda(), torch.empty(6, E, device="cuda:0"),
                                  scoring=scoring, renormalize=renormalize)
        want, tol = ref.route_bwd(X, ids, dw, scoring, renormalize, 1.0)
        if scoring == "softmax" and not renormalize:
            assert torch.isnan(dX[1:]).all()
            dX, want, tol = dX[:1], want[:1], tol[:1]
        check(dX, want, tol, "%s %s" % (scoring, renormalize))
