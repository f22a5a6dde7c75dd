"""The experts' layer as a whole: routing, sort, rows to their experts, the experts' products, rows back,
and all gradients in training; the same with 4-bit weights in serving, eager and as a captured graph.
Every stage is held against 64 bits from the values that the stage before it stored, so each bound is
that stage's own."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import experts_reference as eref
import routing_reference as ref
from experts_reference import check

BF, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import swiglu_gemm_amd as sg
    sg.lib()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,D,N", [(40, 8, 2, 96, 64), (33, 16, 4, 128, 40), (1, 8, 2, 64, 32)])
def test_training_step(T, E, k, D, N, scoring):
    import swiglu_gemm_amd as sg
    g = torch.Generator().manual_seed(T + E)
    dev = dict(device="cuda:0")
    X = torch.randn(T, D, generator=g).to(BF)
    Wr = (torch.randn(D, E, generator=g) * D ** -0.5).to(BF)
    Wf = (torch.randn(E, D, 2 * N, generator=g) * D ** -0.5).to(BF)
    Wd = (torch.randn(E, N, D, generator=g) * N ** -0.5).to(BF)
    dOut = torch.randn(T, D, generator=g).to(BF)
    mask = torch.rand(T, generator=g) < 0.8 if T > 1 else None
    Xd, Wrd, Wfd, Wdd, dOutd = (t.cuda() for t in (X, Wr, Wf, Wd, dOut))
    logits = sg.gemm(Xd, Wrd, torch.empty(T, E, dtype=BF, **dev))
    how = dict(scoring=scoring, scale=1.5)
    ids, w = sg.route_experts(logits, k, mask=None if mask is None else mask.cuda(), **how)
    want = ref.route(logits.cpu(), k, mask=mask, **how)
    assert torch.equal(ids.cpu(), want[0])
    check(w, want[1], want[2], "weights")
    offsets, order, place = sg.sort_experts(ids, E)
    for a, b in zip((offsets, order, place), ref.sort(ids.cpu(), E)):
        assert torch.equal(a.cpu(), b)
    off, pl = offsets.cpu(), place.cpu()
    M, live = T * k, int(off[-1])
    A = sg.spread_rows(Xd, place, torch.full((M, D), 7.0, dtype=BF, **dev))
    assert torch.equal(A.cpu(), ref.spread(X, pl, torch.full((M, D), 7.0, dtype=BF)))
    Y = sg.grouped_swiglu_gemm(A, Wfd, torch.zeros(M, N, dtype=BF, **dev), offsets)
    check(Y[:live], *(t[:live] for t in eref.swiglu_rows(A.cpu(), Wf, off, 1.0, None, BF)), "Y")
    Z = sg.grouped_gemm(Y, Wdd, torch.zeros(M, D, dtype=BF, **dev), offsets)
    zw, zt = eref.gemm_rows(Y.cpu(), Wd, off, "N", 1.0, None, None, 0.0, BF)
    check(Z[:live], zw[:live], zt[:live], "Z")
    out = sg.combine_rows(Z, place, torch.empty(T, D, dtype=BF, **dev), weights=w, residual=Xd)
    check(out, *ref.combine(Z.cpu(), pl, w.cpu(), X), "out")
    # backward
    dZ, dw = sg.combine_rows_bwd(dOutd, Z, place, w, torch.zeros_like(Z), torch.empty_like(w))
    rz, rt, rw, rwt = ref.combine_bwd(dOut, Z.cpu(), pl, w.cpu())
    check(dZ[:live], rz[:live], rt[:live], "dZ")
    check(dw, rw, rwt, "dw")
    dY = sg.grouped_gemm(dZ, Wdd, torch.zeros_like(Y), offsets, transB="T")
    yw, yt = eref.gemm_rows(dZ.cpu(), Wd, off, "T", 1.0, None, None, 0.0, BF)
    check(dY[:live], yw[:live], yt[:live], "dY")
    dWd = sg.grouped_gemm_wgrad(Y, dZ, torch.empty_like(Wdd), offsets)
    check(dWd, *eref.wgrad(Y.cpu(), dZ.cpu(), off, 1.0, None, 0.0, BF), "dWd")
    dH = sg.grouped_swiglu_gemm_bwd(A, Wfd, dY, torch.zeros(M, 2 * N, dtype=BF, **dev), offsets)
    hw, ht = eref.swiglu_bwd_rows(A.cpu(), Wf, dY.cpu(), off, BF)
    check(dH[:live], hw[:live], ht[:live], "dH")
    dA = sg.grouped_gemm(dH, Wfd, torch.zeros_like(A), offsets, transB="T")
    dWf = sg.grouped_gemm_wgrad(A, dH, torch.empty_like(Wfd), offsets)
    check(dWf, *eref.wgrad(A.cpu(), dH.cpu(), off, 1.0, None, 0.0, BF), "dWf")
    dX = sg.combine_rows(dA, place, torch.empty(T, D, dtype=BF, **dev), residual=dOutd)
    check(dX, *ref.combine(dA.cpu(), pl, None, dOut), "dX")
    dlogits = sg.route_experts_bwd(logits, ids, dw, torch.empty_like(logits), **how)
    check(dlogits, *ref.route_bwd(logits.cpu(), ids.cpu(), dw.cpu(), scoring, True, 1.5), "dlogits")


class Serving:
    """A decode batch through one layer with 4-bit experts, into buffers of its own."""

    def __init__(self, T, E, k, D, N, group, seed, dtype=BF):
        import swiglu_gemm_amd as sg
        g = torch.Generator().manual_seed(seed)
        self.k, self.E, self.group, self.D, self.N = k, E, group, D, N
        self.X = torch.randn(T, D, generator=g).to(dtype).cuda()
        self.logits = torch.randn(T, E, generator=g).cuda()
        self.bias = (0.1 * torch.randn(E, generator=g)).cuda()
        gu = torch.randn(E, 2 * N, D, generator=g).to(dtype) * D ** -0.5
        dn = torch.randn(E, D, N, generator=g).to(dtype) * N ** -0.5
        self.up = sg.int4_quantize(gu.cuda(), group, True)
        self.down = sg.int4_quantize(dn.cuda(), group)
        self.Y = torch.zeros(T * k, N, dtype=dtype, device="cuda:0")
        self.Z = torch.zeros(T * k, D, dtype=dtype, device="cuda:0")
        self.out = torch.zeros(T, D, dtype=dtype, device="cuda:0")

    def run(self):
        import swiglu_gemm_amd as sg
        ids, w = sg.route_experts(self.logits, self.k, scoring="sigmoid", bias=self.bias, groups=4, top_groups=2)
        offsets, order, place = sg.sort_experts(ids, self.E)
        sg.int4_swiglu_gemm(self.X, *self.up[:2], self.Y, zeros=self.up[2], group=self.group, offsets=offsets,
                            order=order, top_k=self.k)
        sg.int4_gemm(self.Y, *self.down[:2], self.Z, group=self.group, offsets=offsets)
        sg.combine_rows(self.Z, place, self.out, weights=w, residual=self.X)
        return ids, w, offsets, order, place

    def renew(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.X.copy_(torch.randn(self.X.shape, generator=g).to(self.X.dtype))
        self.logits.copy_(torch.randn(self.logits.shape, generator=g))

    def state(self):
        return [t.clone() for t in (self.Y, self.Z, self.out)]


def unpacked(w, N, K, group):
    """codes, scales, zeros of each expert, element by element, from the kernels' layout."""
    out = []
    for e in range(w[0].shape[0]):
        r, c = torch.meshgrid(torch.arange(N), torch.arange(K), indexing="ij")
        i = c % 8
        nib = i // 2 + 4 * (i % 2)
        at = ((r // 16) * -(-K // 128) + c // 128) * 1024 + 16 * (16 * (c % 32 // 8) + r % 16) + 4 * (c % 128 // 32)
        byte = w[0][e].cpu()[at + nib // 2]
        codes = torch.where(nib % 2 == 1, byte >> 4, byte & 15)
        n = -(-K // group)
        r, f = torch.meshgrid(torch.arange(N), torch.arange(n), indexing="ij")
        at = ((r // 16) * -(-n // 4) + f // 4) * 64 + 4 * (r % 16) + f % 4
        out.append((codes, w[1][e].cpu()[at], None if w[2] is None else w[2][e].cpu()[at]))
    return out


@pytest.mark.parametrize("T,dtype", [(1, BF), (13, F16), (50, BF)])
def test_serving_step(T, dtype):
    s = Serving(T, 16, 4, 160, 96, 32, T, dtype)
    ids, w, offsets, order, place = s.run()
    want = ref.route(s.logits.cpu(), 4, "sigmoid", s.bias.cpu(), 4, 2)
    assert torch.equal(ids.cpu(), want[0])
    check(w, want[1], want[2], "weights")
    off, od, pl = ref.sort(ids.cpu(), 16)
    assert torch.equal(offsets.cpu(), off) and torch.equal(order.cpu(), od) and torch.equal(place.cpu(), pl)
    check(s.Y, *ref.int4_rows(s.X.cpu(), unpacked(s.up, 192, 160, 32), 32, off, od, 4, 4 * T, dtype, True), "Y")
    check(s.Z, *ref.int4_rows(s.Y.cpu(), unpacked(s.down, 160, 96, 32), 32, off, None, 1, 4 * T, dtype, False),
          "Z")
    check(s.out, *ref.combine(s.Z.cpu(), pl, w.cpu(), s.X.cpu()), "out")


def test_serving_step_as_a_graph():
    """Captured once, replayed on other tokens and routes, with eager work between the replays."""
    eager, held = Serving(24, 16, 4, 256, 128, 64, 5), Serving(24, 16, 4, 256, 128, 64, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        held.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = held.run()
    for seed in (11, 12, 13, 14):
        eager.renew(seed)
        held.renew(seed)
        for t in (held.Y, held.Z, held.out):
            t.zero_()
        want = [t.clone() for t in eager.run()] + eager.state()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(list(kept) + held.state(), want):
            assert torch.equal(a, b), seed


def test_two_graphs_and_two_streams_at_once():
    """Two layers of different sizes whose calls interleave on two streams, eager and replayed."""
    one, two = Serving(40, 16, 4, 256, 128, 64, 5), Serving(9, 32, 2, 384, 64, 128, 6)
    want = []
    for s in (one, two):
        s.run()
        torch.cuda.synchronize()
        want.append(s.state())
        s.out.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, st in zip((one, two), streams):
            with torch.cuda.stream(st):
                s.run()
    torch.cuda.synchronize()
    for s, w in zip((one, two), want):
        for a, b in zip(s.state(), w):
            assert torch.equal(a, b)
    graphs = []
    for s in (one, two):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            s.run()
    for _ in range(3):
        for s in (one, two):
            s.out.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for s, w in zip((one, two), want):
            for a, b in zip(s.state(), w):
                assert torch.equal(a, b)


def test_runs_repeat_bit_for_bit():
    import swiglu_gemm_amd as sg
    s = Serving(200, 32, 4, 256, 128, 64, 8)
    first = [t.clone() for t in s.run()] + s.state()
    for _ in range(3):
        for a, b in zip(list(s.run()) + s.state(), first):
            assert torch.equal(a, b)
    g = torch.Generator().manual_seed(2)
    ids, w, _, _, place = s.run()
    dw = torch.randn(200, 4, generator=g).cuda()
    for _ in range(2):
        dX = [sg.route_experts_bwd(s.logits, ids, dw, torch.empty_like(s.logits), scoring="sigmoid")
              for _ in range(2)]
        grads = [sg.combine_rows_bwd(s.X, s.Z, place, w, torch.zeros_like(s.Z), torch.empty_like(w))
                 for _ in range(2)]
        assert torch.equal(*dX)
        assert torch.equal(grads[0][0], grads[1][0]) and torch.equal(grads[0][1], grads[1][1])
