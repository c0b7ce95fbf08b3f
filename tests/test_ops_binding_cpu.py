"""The binding's calls around the linears, without a GPU: what reaches the library."""
import os
import subprocess
import sys
import types

import pytest
import torch

BF, E8 = torch.bfloat16, torch.float8_e4m3fn


class OnDevice:
    """What the binding looks at in a tensor on device 0."""
    is_cuda, device = True, torch.device("cuda", 0)

    def __init__(self, t, address=4096):
        self.t, self.address = t, address
        self.dtype, self.shape = t.dtype, t.shape

    def stride(self):
        return self.t.stride()

    def is_contiguous(self):
        return self.t.is_contiguous()

    def get_device(self):
        return 0

    def data_ptr(self):
        return self.address


@pytest.fixture
def calls(monkeypatch):
    """The binding over a library that records its arguments and accepts them."""
    from w4a8_block_quantized_gb300 import binding
    seen = []
    monkeypatch.setattr(binding, "_lib", types.SimpleNamespace(
        w4a8_swiglu_quant_fp8=lambda *a: seen.append(a) or 0))
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(binding, "_raw_stream", lambda index: 0)
    return seen


@pytest.mark.parametrize("M,width,want", [(1, 515, 256), (1, 512, 256), (3, 512, 512), (3, 1024, 1024)])
def test_row_stride_of_gate_and_up(calls, M, width, want):
    """One row has no stride to speak of: a row of an array of any width passes, as where the call allocates its
    outputs; several rows pass theirs."""
    from w4a8_block_quantized_gb300 import binding
    gu = torch.zeros((M, width), dtype=BF)
    gate, up = OnDevice(gu[:, :256]), OnDevice(gu[:, 256:512])
    binding.swiglu_quant_fp8(gate, up, a_q=OnDevice(torch.zeros((M, 256)).to(E8)), a_scale=OnDevice(torch.zeros((2, M))))
    assert [c[2] for c in calls] == [want]


def test_import_without_torch_private_names():
    """A torch that lacks the private names of the short host path (one without CUDA, say): the module imports, and the
    public calls stand in."""
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "from w4a8_block_quantized_gb300 import binding as b\n"
            "torch.cuda.current_stream = lambda index: type('S', (), dict(cuda_stream=index + 40))\n"
            "assert b._current_device is torch.cuda.current_device and b._raw_stream(2) == 42\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr
