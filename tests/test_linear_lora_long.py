"""convrot_linear_lora where a token is longer than the row kernel's registers (K >= 8192) and
than the token-block kernel's LDS (K > 32768), as few tokens, as a list and in slices: against the
64-bit formula and its tolerance of test_linear_lora (the fp32 sum over K is in it).  Some K have
pieces that do not divide evenly among the parts of the first product."""
import pytest

from tests.test_linear_lora import check, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from w8a8_rotated_int8_convrot_amd import binding
    binding.lib()
    return binding


@pytest.mark.parametrize("io,row,bias", [("bf16", True, True), ("fp16", False, False)])
@pytest.mark.parametrize("M,K,N,ranks,run,group", [
    (1, 131072, 40, [16], None, 128), (3, 40960, 24, [8, 40], 1, 256), (16, 8192, 100, [16] * 16, 1, 128),
    (100, 12288, 64, [16, 8, 40, 64, 3, 1, 20, 33], 5, 256), (40, 8448, 100, [33, 64], 20, 128),
    (200, 12288, 104, [16, 5, 70], 60, 128), (150, 33024, 80, [24, 100], 70, 256), (30, 32768, 64, [16, 16], 9, 128),
    (700, 8192, 200, [40, 16], 150, 256), (300, 16640, 520, [128, 9, 64], 40, 128), (1100, 9088, 2050, [32, 16], 500, 128)])
def test_long_tokens(B, M, K, N, ranks, run, group, io, row, bias):
    check(B, problem(M, K, N, io, ranks, row, bias, M + K + N, run), group)
