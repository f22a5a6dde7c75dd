"""Quotients halfway between two codes: w / scale is rounded to the nearest integer, ties to even, and the
zero point added, so that an odd zero point does not turn a tie round."""
import pytest

torch = pytest.importorskip("torch")

import routing_reference as ref

# scale 1: the ends are 15 apart; halves in between, around an odd and an even zero point
ENDS = [(-3.0, 12.0), (-4.0, 11.0), (-15.0, 0.0), (0.0, 15.0)]


def rows():
    out = []
    for lo, hi in ENDS:
        half = torch.arange(30) / 2
        out.append(torch.cat([torch.tensor([lo, hi]), (lo + half).clamp(lo, hi)]))
    return torch.stack(out)


def by_hand(W):
    even = lambda x: int(x) if x == int(x) else min((int(x - 0.5), int(x + 0.5)), key=lambda n: n % 2)
    codes = []
    for (lo, _), row in zip(ENDS, W.tolist()):
        zero = int(-lo)
        codes.append([min(max(even(abs(w)) * (1 if w >= 0 else -1) + zero, 0), 15) for w in row])
    return codes


def test_ties_by_hand():
    W = rows()
    codes, scales, zeros = ref.int4_quantize(W, 32, True, torch.float16)
    assert (scales == 1).all() and zeros.flatten().tolist() == [3, 4, 15, 0]
    assert codes.tolist() == by_hand(W)
    at = W[0].tolist().index(0.5), W[0].tolist().index(1.5)
    assert [codes[0, i].item() for i in at] == [3, 5]          # 0 + 3 and 2 + 3


@pytest.mark.gpu
@pytest.mark.parametrize("size", [1.0, 2.0 ** -9, 2.0 ** 12])
def test_ties(size):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import swiglu_gemm_amd as sg
    W = rows()
    want = ref.int4_layout(torch.tensor(by_hand(W), dtype=torch.uint8), torch.full((4, 1), size).half(),
                           torch.tensor([[3], [4], [15], [0]], dtype=torch.uint8), 32)
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        got = sg.int4_quantize((size * W).to(dtype).cuda(), 32, True, torch.float16)
        for a, b in zip(got, want):
            assert torch.equal(a.cpu(), b)
