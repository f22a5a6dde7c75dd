"""uint8 is what the 4-bit matrices' codes are held in, so the grouped products do not take it for
e4m3 codes: a pair of 4-bit matrices given to them would be multiplied as something else, without
an error.  e4m3 operands come as torch.float8_e4m3fn (a view of the same bytes)."""
import pytest

torch = pytest.importorskip("torch")

import swiglu_gemm_amd as sg

F8, U8, BF = torch.float8_e4m3fn, torch.uint8, torch.bfloat16


def t(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def off(n):
    return torch.zeros(n, dtype=torch.int32)


@pytest.mark.parametrize("a,b", [(U8, U8), (U8, F8), (F8, U8)])
def test_grouped_products_refuse_bytes(a, b):
    A = t(8, 16, dtype=a)
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        sg.grouped_gemm(A, t(3, 4, 16, dtype=b), t(8, 4), off(4), transB="T")
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        sg.grouped_swiglu_gemm(A, t(3, 16, 10, dtype=b), t(8, 5), off(4))


def test_four_bit_codes_do_not_pass_as_e4m3():
    codes, weight = t(8, 32, dtype=U8), t(3, 40, 32, dtype=U8)       # K = 64
    with pytest.raises(TypeError, match="mxfp4_gemm"):
        sg.grouped_gemm(codes, weight, t(8, 40), off(4), transB="T")


def test_the_same_bytes_as_e4m3():
    A, B = t(8, 16, dtype=U8).view(F8), t(3, 4, 16, dtype=U8).view(F8)
    with pytest.raises(ValueError, match="on the GPU"):
        sg.grouped_gemm(A, B, t(8, 4), off(4), transB="T")
    with pytest.raises(ValueError, match="on the GPU"):
        sg.grouped_swiglu_gemm(A, t(3, 16, 10, dtype=U8).view(F8), t(8, 5), off(4))
