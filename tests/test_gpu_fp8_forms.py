"""GPU tests of the forms of the e4m3 linear, each called by name: its bounded waits."""
import time

import pytest
import torch

import fp8_forms as F

pytestmark = pytest.mark.gpu
E8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    F.lib()


def integers(seed, M, N, K):
    """Operands of small integers with unit scales (every partial sum below 2^24: exact in fp32, in any order), and
    their product in fp64."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = torch.randint(-8, 9, (M, K), generator=g, device="cuda").float()
    w = torch.randint(-8, 9, (N, K), generator=g, device="cuda").float()
    nb, nt = -(-K // 128), -(-N // 128)
    sa, sw = torch.ones((nb, M), device="cuda"), torch.ones((nt, nb), device="cuda")
    return (a.to(E8), sa, w.to(E8), sw), a.double() @ w.double().T


# form, M, N, K, SMs (few: several tiles to a CTA or pair), the block of a CTA before which its copies stop
STOPS = [((0, 1), 600, 600, 2048, 152, 0), ((0, 1), 600, 600, 2048, 152, 5), ((0, 1), 600, 600, 2048, 4, 21),
         ((0, 1), 600, 601, 1168, 4, 14), ((16, 1), 40, 700, 2048, 4, 3), ((16, 1), 40, 700, 2048, 4, 37),
         ((16, 4), 16, 700, 2048, 152, 2), ((32, 1), 200, 300, 2048, 4, 18), ((32, 8), 32, 300, 2048, 152, 1),
         ((64, 1), 200, 300, 2048, 4, 18), ((64, 2), 200, 300, 2048, 152, 7), ((128, 1), 300, 300, 1168, 2, 10),
         ((128, 2), 300, 300, 2048, 152, 0), ((128, 4), 300, 300, 2048, 152, 3)]


@pytest.mark.parametrize("form,M,N,K,sms,stop", STOPS)
def test_waits_run_out(form, M, N, K, sms, stop):
    """Copies that never come: every wait on them gives up, the launch ends with the timeout in the status word and
    nothing written outside y, and the next launch is right."""
    ops, want = integers(stop + M, M, N, K)
    buf = torch.full((M * N + 64,), 7.0, device="cuda")
    y = buf[32:-32].view(M, N)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    _, status = F.run(form, *ops, y=y, limit_us=20_000, copy_blocks=stop, num_sms=sms)
    torch.cuda.synchronize()
    # one wait gives up after 20 ms and up to 64 tries of 0.1 ms more, the rest of its CTA soon after it; a pair's two
    # CTAs and a split's may do so one after the other
    assert time.perf_counter() - t0 < 2.0
    assert int(status) == 1
    assert (buf[:32] == 7).all() and (buf[-32:] == 7).all()
    y, status = F.run(form, *ops, num_sms=sms)
    assert torch.equal(y.double(), want) and int(status) == 0
