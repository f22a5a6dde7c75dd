"""More experts than a wave has lanes: a lane then counts several of them and the item's expert is
found by a second walk; weight gradients come in the experts' own order.  At the counts where that
begins and at those of large mixtures, with uneven runs, experts without rows at either end and
rows of no expert, every output against 64 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_grouped import run_gemm, run_swiglu, run_wgrad
from test_gpu_mxfp4 import run_product


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import swiglu_gemm_amd as sg
    sg.lib()


def uneven(experts):
    """Runs of 0 to 150 rows, most of them short; none for the first and the last two experts."""
    g = torch.Generator().manual_seed(experts)
    n = (150 * torch.rand(experts, generator=g) ** 4).int()
    n[0], n[-2:] = 0, 0
    n[experts // 2] = 150
    return n.tolist()


@pytest.mark.parametrize("experts", [64, 65, 128, 129, 256])
@pytest.mark.parametrize("what", ["gemm", "e4m3", "swiglu", "bwd", "wgrad", "wgrad fp32", "mx"])
def test_uneven_experts(what, experts):
    sizes = uneven(experts)
    if what == "gemm":
        run_gemm("bf16", "N", sizes, 264, 136, before=3, behind=5)
    elif what == "e4m3":
        run_gemm("e4m3", "T", sizes, 272, 144, before=3, behind=5, scaled=True)
    elif what in ("swiglu", "bwd"):
        run_swiglu("f16", sizes, 136, 72, bwd=what == "bwd", before=3, behind=5)
    elif what == "mx":
        run_product(sizes, 136, 288, swiglu=True, before=3, behind=5, spread=0)
    else:
        run_wgrad("bf16", "f32" if "fp32" in what else "same", sizes, 264, 136, beta=0.5, before=3,
                  behind=5)
