"""The largest calls of the routing operators and of 4-bit integer weights: one launch has fewer than 2^32
threads along a side, and a product at most 2^22 work-groups, so a call that needs more is refused before it
starts (no GPU is used for that), and the largest that fits runs."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import swiglu_gemm_amd as sg
from swiglu_gemm_amd import build as sgbuild

P, NUL = ctypes.c_void_p(0x1000), ctypes.c_void_p(0)
TOO_MANY = 9                                          # hipErrorInvalidConfiguration
TOKENS = 2**26 - 4


@pytest.fixture(scope="module")
def L():
    if sgbuild.is_stale():
        sgbuild.build()
    return sg.lib()


def test_calls_past_the_largest_launch_are_refused(L):
    for T in (TOKENS + 1, 2**26, 2**30):
        assert L.sg_route_experts(P, 8, T, 8, 0, 2, 0, NUL, 1, 1, 2, 1, 1.0, NUL, P, P, NUL) == TOO_MANY
        assert L.sg_route_experts_bwd(P, 8, T, 8, 0, 2, 0, 1, 1.0, P, P, P, 8, NUL) == TOO_MANY
    # rows of more than 1024 elements take 256 threads, of 513 to 1024 half of them, ...
    for D, T in ((1025, 2**24), (70000, 2**24), (1024, 2**25 - 1), (512, 2**26 - 3), (129, 2**27 - 7)):
        assert L.sg_spread_rows(P, D, T, D, 2, P, 2, NUL, 8, P, D, NUL) == TOO_MANY
        assert L.sg_combine_rows(P, D, 8, D, T, 2, P, 2, P, NUL, 1, P, D, NUL) == TOO_MANY
    # the gradient of combining: 64 threads a place
    for T, k in ((2**24, 4), (TOKENS + 1, 1), (2**20, 64), (2**30, 65536)):
        assert L.sg_combine_rows_bwd(P, 8, P, 8, 8, 8, T, 2, P, k, P, P, 8, P, NUL) == TOO_MANY


def test_products_past_the_largest_launch_are_refused(L):
    for M, N in ((2**20, 2**16), (2**18 + 1, 2**17), (2**30, 2**30), (64, 2**30)):
        args = [1, NUL, NUL, 1, M, M, N, 128, 128]
        ends = [P, 128, P, P, NUL, P, N]
        assert L.sg_int4_gemm(*args, 1.0, *ends, 2, 2, NUL) == TOO_MANY
        args[6] = N // 2
        assert L.sg_int4_swiglu_gemm(*args, *ends, 2, NUL) == TOO_MANY


@pytest.mark.gpu
def test_the_most_tokens():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    X = torch.empty(TOKENS, 3, dtype=torch.bfloat16, device="cuda:0").normal_()
    ids, w = sg.route_experts(X, 1, renormalize=False)
    for lo in range(0, TOKENS, 2**23):
        part = slice(lo, lo + 2**23)
        want = X[part].float()
        top = want.amax(1, keepdim=True)
        first = torch.where(want == top, torch.arange(3, device="cuda:0"), 3).amin(1, keepdim=True)
        assert torch.equal(ids[part].long(), first)
        s = 1 / torch.exp(want.double() - top.double()).sum(1, keepdim=True)
        assert ((w[part] - s).abs() <= 2.0 ** -19 * s).all()   # exponentials, two sums and a division: 32 half steps
    dw = torch.ones(TOKENS, 1, device="cuda:0")
    dX = sg.route_experts_bwd(X, ids, dw, torch.full_like(X, 7.0))
    assert (dX == 0).all()                             # one expert renormalised: its weight is 1 whatever X


@pytest.mark.gpu
def test_the_most_places():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    k = 4
    T = TOKENS // k
    dev = dict(device="cuda:0")
    place = (torch.arange(T * k, dtype=torch.int32, **dev) % 97 - 1).view(T, k)
    Z = torch.arange(1.0, 96.0, **dev)[:, None].contiguous()           # 95 rows: places 95 are outside
    dOut = (torch.arange(T, **dev) % 13 - 6).float()[:, None].contiguous()
    dw = sg.combine_rows_bwd(dOut, Z, place, torch.ones(T, k, **dev), dweights=torch.full((T, k), 7.0, **dev))[1]
    want = torch.where((place >= 0) & (place < 95), dOut * (place + 1), 0.0)
    assert torch.equal(dw, want)
