"""The example runs the operators together: its MLP agrees with fp32 on the dequantized weights within
the formats' rounding, in both weight formats, for a prompt and for one token."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a8_block_quantized_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("decoder_mlp", os.path.join(ROOT, "examples", "decoder_mlp.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens,hidden,inner", [(1, 512, 1024), (7, 1024, 896), (96, 512, 1024), (300, 1024, 1344)])
def test_decoder_mlp(example, tokens, hidden, inner):
    """Two activations are quantized on the way.  INT8 per row: a step of at most 1/127 of the row's
    largest value, 4 to 5 standard deviations of its values here, so a relative error near 0.04 / sqrt(12)
    each; e4m3: at most 2^-4 of each value, near 0.026 in norm.  Gate and up errors meet in a product:
    under 0.1 in all."""
    for name, err, exact, same, _ in example.run(tokens, hidden, inner, replays=1):
        assert exact and same, name
        assert err < 0.1, (name, err)
