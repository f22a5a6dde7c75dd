"""Sizes whose offsets pass 32 bits: logits, rows and 4-bit weights beyond 2^31 elements or bytes, and
many places.  The far end is compared, from inputs made on the GPU."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import routing_reference as ref
from experts_reference import check


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import swiglu_gemm_amd as sg
    sg.lib()


def test_logits_past_32_bits():
    import swiglu_gemm_amd as sg
    T, E = 2**23 + 5, 256                                  # 2^31 elements and some
    X = torch.empty(T, E, dtype=torch.bfloat16, device="cuda:0").normal_()
    ids, w = sg.route_experts(X, 8, renormalize=False)
    want, ww, tol = ref.route(X[-40:].cpu(), 8, renormalize=False)
    assert torch.equal(ids[-40:].cpu(), want)
    check(w[-40:], ww, tol)
    dw = torch.ones_like(w)
    dX = sg.route_experts_bwd(X, ids, dw, torch.empty_like(X), renormalize=False)
    check(dX[-40:], *ref.route_bwd(X[-40:].cpu(), want, dw[-40:].cpu(), "softmax", False, 1.0))


def test_rows_past_32_bits():
    import swiglu_gemm_amd as sg
    M, D = 600000, 4096                                    # 4.9 GB of rows
    Z = torch.zeros(M, D, dtype=torch.bfloat16, device="cuda:0")
    g = torch.Generator().manual_seed(1)
    X = torch.randn(6, D, generator=g).bfloat16()
    place = torch.tensor([[M - 1, 5], [M - 7, 2**18], [3, M - 2], [M // 2, M - 3], [0, M - 5], [M, -1]],
                         dtype=torch.int32)
    sg.spread_rows(X.cuda(), place.cuda(), Z)
    for t in range(5):
        for r in place[t].tolist():
            assert torch.equal(Z[r].cpu(), X[t])
    w = torch.rand(6, 2, generator=g)
    small = torch.stack([Z[min(max(r, 0), M - 1)] for r in place.flatten().tolist()]).cpu()
    at = torch.arange(12, dtype=torch.int32).view(6, 2)
    at[5] = -1
    out = sg.combine_rows(Z, place.cuda(), torch.empty(6, D, dtype=torch.bfloat16, device="cuda:0"), weights=w.cuda())
    check(out, *ref.combine(small, at, w))
    dZ, dw = sg.combine_rows_bwd(X.cuda(), Z, place.cuda(), w.cuda(), torch.zeros_like(Z), torch.empty(6, 2, device="cuda:0"))
    _, _, ww, wt = ref.combine_bwd(X, small, at, w)
    check(dw, ww, wt)
    for t in range(5):
        for j in range(2):
            want = w[t, j].double() * X[t].double()
            check(dZ[int(place[t, j])], want, ref.U * want.abs() + ref.half_step(want, torch.bfloat16))


def test_many_places():
    import swiglu_gemm_amd as sg
    for n, E in ((2**22 + 77, 100), (2**20, 5000)):
        ids = torch.randint(-1, E, (n,), dtype=torch.int32, device="cuda:0")
        offsets, order, place = sg.sort_experts(ids, E)
        key = torch.where(ids < 0, E, ids.long())
        want = torch.argsort(key, stable=True)
        live = int((ids >= 0).sum())
        assert torch.equal(order[:live].long(), want[:live]) and (order[live:] == -1).all()
        counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda:0").scatter_add_(0, key, torch.ones_like(key))
        assert torch.equal(offsets[1:].long(), counts[:E].cumsum(0)) and offsets[0] == 0
        assert torch.equal(place[order[:live].long()].long(), torch.arange(live, device="cuda:0"))
        assert (place[ids < 0] == -1).all()


def test_weights_past_32_bits():
    """Five experts of 16384 x 65536, 512 MiB of codes each; the last expert's last columns."""
    import swiglu_gemm_amd as sg
    E, N, K = 5, 16384, 65536
    nc, ns = sg.int4_shapes(N, K)
    codes = torch.randint(0, 256, (E, nc), dtype=torch.uint8, device="cuda:0")
    scales = (torch.rand(E, ns, device="cuda:0") + 0.5).mul_(2.0 ** -9).half()
    A = torch.randn(3, K, device="cuda:0").half()
    offsets = torch.tensor([0, 0, 0, 0, 1, 3], dtype=torch.int32, device="cuda:0")
    C = sg.int4_gemm(A, codes, scales, torch.empty(3, N, dtype=torch.float16, device="cuda:0"), offsets=offsets)
    r, c = torch.meshgrid(torch.arange(N - 20, N), torch.arange(K), indexing="ij")
    nib = c % 8 // 2 + 4 * (c % 2)
    at = ((r // 16) * (K // 128) + c // 128) * 1024 + 16 * (16 * (c % 32 // 8) + r % 16) + 4 * (c % 128 // 32)
    f = torch.arange(K // 128)[None]
    rows = torch.arange(N - 20, N)[:, None]
    fat = ((rows // 16) * (K // 512) + f // 4) * 64 + 4 * (rows % 16) + f % 4
    for e, row in ((3, 0), (4, 1), (4, 2)):
        byte = codes[e][(at + nib // 2).cuda()].cpu()
        held = torch.where(nib % 2 == 1, byte >> 4, byte & 15), scales[e].cpu()[fat], None
        want, tol = ref.int4_rows(A[row:row + 1].cpu(), [held], 128, None, None, 1, 1, torch.float16, False)
        check(C[row:row + 1, -20:], want, tol)
