"""What a refused shape of the operators around the linears means, and where the sizes end."""
import ctypes

import pytest

P = ctypes.c_void_p
d, odd4 = P(1 << 20), P((1 << 20) + 4)


@pytest.fixture(scope="module")
def lib():
    from w4a8_block_quantized_gb300 import binding, build
    build.build()
    return binding.load()


def test_the_shape_text_covers_every_refusal_of_a_shape(lib):
    """K of whole 64s or 16s, a row stride below K, a size past the limit."""
    from w4a8_block_quantized_gb300 import binding as b
    assert lib.w4a8_quant_fp8(d, 0, d, d, 4, 120, None) == b.W4A8_ERR_SHAPE
    assert lib.w4a8_swiglu_quant_fp8(d, d, 64, 1, d, d, 4, 128, None) == b.W4A8_ERR_SHAPE
    text = b.status_string(b.W4A8_ERR_SHAPE)
    assert all(word in text for word in ("64", "16", "stride", "limited")), text


@pytest.mark.parametrize("M,N,K,fits", [
    (32 << 15, 128 << 15, 128, True), (32 << 15, (128 << 15) + 1, 256, False), ((32 << 15) + 1, 128 << 15, 256, False),
    (32 << 15, 128 << 15, 256, False), (32 << 15, 128 << 15, 144, False), (32 << 15, (128 << 15) - 128, 256, True)])
def test_the_size_limit_of_the_e4m3_linear(lib, M, N, K, fits):
    """ceil(M / 32) ceil(N / 128) ceil(K / 128) < 2^31; a size that fits is then refused for the pointer given here."""
    from w4a8_block_quantized_gb300 import binding as b
    rc = lib.w4a8_fp8_linear(odd4, d, d, d, None, d, 0, M, N, K, None)
    assert rc == (b.W4A8_ERR_ALIGN if fits else b.W4A8_ERR_SHAPE)
