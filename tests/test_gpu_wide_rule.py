"""A few rows each against weights stored K x N: where the cost model takes 32 x 128 tiles and ones
256 wide would make 3/4 of a round of the CUs to a whole one, those are taken in their place; outside
of that window the model's choice stands.  At both ends and next to them: which tile runs, and every
output against 64 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_grouped import run_gemm, run_swiglu, took

# 32 x 128; 128 x 256, 32 deep, by the rule; the model's own at 264 tiles of K = 512: 128 x 256, 64 deep
FEW_ROWS, WIDE, DEEP = 1, 4, 3


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import swiglu_gemm_amd as sg
    sg.lib()


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("experts,rows,cfg", [(23, 4, FEW_ROWS), (24, 4, WIDE), (32, 4, WIDE),
                                              (33, 4, DEEP), (24, 16, WIDE)])
def test_window(experts, rows, cfg, swiglu):
    sizes = [rows] * experts                # eight tiles of 256 columns each
    if swiglu:
        run_swiglu("bf16", sizes, 1024, 512)
    else:
        run_gemm("bf16", "N", sizes, 2048, 512)
    assert took(cfg)
