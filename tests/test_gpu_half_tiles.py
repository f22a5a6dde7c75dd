"""Where the items of an XCD leave its last round of work-groups at most half full, that round's
tiles run as two halves of their rows each.  That takes hundreds of tiles; here small K keeps
them cheap, every XCD splits some, and among the split ones are tiles whose lower half is whole,
partly filled and empty, as the rule in find_rows() places them.  Every row is compared with the
definition in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_grouped import force, run_gemm, run_swiglu, took
from test_gpu_mxfp4 import run_product

XCDS, CUS = 8, 32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import swiglu_gemm_amd as sg
    sg.lib()


def split_rows(sizes, cols, bm, bn, occ):
    """For every item that is split: how many rows of its tile there are.  The order of the tiles
    is the kernels': an expert's tiles together, four rows of tiles walked at a time."""
    tiles_n, left = -(-cols // bn), []
    for n in sizes:
        tm = -(-n // bm)
        for g in range(0, tm, 4):
            group = list(range(g, min(g + 4, tm)))
            left += [min(bm, n - m * bm) for _ in range(tiles_n) for m in group]
    out, first, slots = [], 0, CUS * occ
    for x in range(XCDS):
        n = len(left) // XCDS + (x < len(left) % XCDS)
        split = n % slots
        if n <= slots or 2 * split > slots:
            split = 0
        out.append(left[first + n - split:first + n])
        first += n
    return out


def runs(bm, cols, bn, occ, experts):
    """Ragged runs whose tiles fill each XCD's rounds by a third of a round too many."""
    tiles_n = -(-cols // bn)
    want = XCDS * (CUS * occ + CUS * occ // 3) // tiles_n           # rows of tiles
    kinds = [3 * bm + bm // 2 + 17, 2 * bm + bm // 2 - 20, 0, bm, 1, 4 * bm, bm - 1, bm + bm // 2]
    if experts > 64:
        kinds = [n % (2 * bm) for n in kinds]
    sizes = []
    while len(sizes) < experts - 1:
        n = kinds[len(sizes) % len(kinds)]
        n = min(n, max(0, want - 1) * bm)
        sizes.append(n)
        want -= -(-n // bm)
    return sizes + [want * bm - bm // 4]


def check_plan(sizes, cols, bm, bn, occ):
    plan = split_rows(sizes, cols, bm, bn, occ)
    assert all(plan), "every XCD splits some"
    rows = [r for x in plan for r in x]
    assert any(r <= bm // 2 for r in rows) and any(r == bm for r in rows)
    assert any(bm // 2 < r < bm for r in rows)


# tile: its rows, columns and work-groups a CU (src: kGroupCfg, kMxCfg)
GROUPED = {4: (128, 256, 2), 5: (256, 256, 1)}
FOUR_BIT = {2: (128, 128, 2), 3: (256, 256, 1)}
COLS = 1300                                                    # six tiles of 256, eleven of 128


@pytest.mark.parametrize("experts", [24, 90])
@pytest.mark.parametrize("what", ["gemm N", "gemm T", "swiglu", "swiglu bwd"])
@pytest.mark.parametrize("cfg", sorted(GROUPED))
def test_grouped_halves(force, cfg, what, experts):
    bm, bn, occ = GROUPED[cfg]
    sizes = runs(bm, COLS, bn, occ, experts)
    check_plan(sizes, COLS, bm, bn, occ)
    force(cfg)
    K = 136                                                    # K tiles and a tail
    if what.startswith("gemm"):
        run_gemm("bf16", what[-1], sizes, COLS if what[-1] == "T" else COLS - 4, K, before=3, behind=5)
    else:
        run_swiglu("f16", sizes, COLS // 2 - 2, K, bwd=what.endswith("bwd"), before=3, behind=5)
    assert took(cfg)


@pytest.mark.parametrize("what", ["gemm", "fp32", "swiglu"])
@pytest.mark.parametrize("grouped", [True, False])
@pytest.mark.parametrize("cfg", sorted(FOUR_BIT))
def test_four_bit_halves(monkeypatch, cfg, grouped, what):
    import swiglu_gemm_amd as sg
    bm, bn, occ = FOUR_BIT[cfg]
    sizes = runs(bm, COLS, bn, occ, 24)
    if grouped:
        check_plan(sizes, COLS, bm, bn, occ)
    else:
        # one run: its last tile-row is the only ragged one, in the last XCD
        sizes = [sum(-(-n // bm) for n in sizes) * bm - bm // 4]
        plan = split_rows(sizes, COLS, bm, bn, occ)
        assert all(plan) and bm - bm // 4 in plan[-1]
        sizes = sizes[0]
    monkeypatch.setenv("SG_FORCE_MX4", str(cfg))
    around = dict(before=3, behind=5) if grouped else {}
    if what == "swiglu":
        run_product(sizes, COLS // 2, 288, "bf16", swiglu=True, spread=0, **around)
    else:
        run_product(sizes, COLS, 288, "f32" if what == "fp32" else "bf16", alpha=0.5, spread=1, **around)
    assert "cfg=%d " % cfg in sg.last_config()
