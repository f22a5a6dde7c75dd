"""Partial K tiles beside rows of no expert and gaps between the experts' matrices, both full of
NaN: the products are those of the experts' own elements, whichever way the tile's tail is loaded."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import experts_reference as ref
from test_gpu_grouped import force, rand, table, took

SIZES = [70, 0, 3, 130, 64]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import swiglu_gemm_amd as sg
    sg.lib()


def apart(B, gap):
    """B's matrices `gap` elements apart, NaN between them."""
    e, r, c = B.shape
    store = torch.full((e * (r * c + gap),), float("nan"), dtype=B.dtype, device="cuda:0")
    out = torch.as_strided(store, (e, r, c), (r * c + gap, c, 1))
    out.copy_(B.cuda())
    return out


@pytest.mark.parametrize("cfg", [1, 3, 4, 5])
@pytest.mark.parametrize("gap", [0, 8, 64 * 136])
@pytest.mark.parametrize("trans", "NT")
def test_gemm(force, cfg, gap, trans):
    import swiglu_gemm_amd as sg
    force(cfg)
    N, K, off = 136, 72, table(SIZES, 3)
    M = int(off[-1]) + 9
    A = rand((M, K), "bf16", 1.0, 1)
    A[:3], A[-9:] = float("nan"), float("nan")
    B = rand((5, N, K) if trans == "T" else (5, K, N), "bf16", 0.1, 2)
    C = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda:0")
    print("tail cfg=%d gap=%d %s" % (cfg, gap, trans), flush=True)
    sg.grouped_gemm(A.cuda(), apart(B, gap), C, off.cuda(), transB=trans)
    assert took(cfg)
    want, tol = ref.gemm_rows(A, B, off, trans, 1.0, None, None, 0.0, torch.bfloat16)
    ref.check(C, want, tol)
    assert (C[:3] == 7).all() and (C[-9:] == 7).all()


@pytest.mark.parametrize("cfg", [2, 4, 5])
def test_wgrad(force, cfg):
    import swiglu_gemm_amd as sg
    force(cfg)
    N, K, off = 136, 264, table(SIZES, 3)
    M = int(off[-1]) + 61
    A, D = rand((M, K), "bf16", 1.0, 1), rand((M, N), "bf16", 0.1, 2)
    for t in (A, D):
        t[:3], t[-61:] = float("nan"), float("inf")
    C = torch.empty(5, K, N, device="cuda:0")
    print("tail wgrad cfg=%d" % cfg, flush=True)
    sg.grouped_gemm_wgrad(A.cuda(), D.cuda(), C, off.cuda())
    assert took(cfg)
    want, tol = ref.wgrad(A, D, off, 1.0, None, 0.0, torch.float32)
    ref.check(C, want, tol)
