"""GPU tests of the forms of the e4m3 linear, each called by name (pairs of CTAs; 16-, 32-, 64- and 128-token tiles,
K on one, two, four or eight CTAs): exact products, NaN and the largest codes, calls without waits between them,
the bounded waits; and the forms that public calls take."""
import math
import random
import time

import pytest
import torch

import fp8_forms as F
import ops_ref as R

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


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def problems(form):
    """Sizes for a form, the smallest first: odd rows and columns, a last block of 16, K of fewer blocks than a batch of
    factors and of more, for a split CTAs with one block, with several, and with none (nine blocks on eight CTAs)."""
    tn, split = form
    if tn == 0:
        sizes = [(1, 1, 16), (257, 130, 144), (600, 521, 1168), (513, 768, 2064), (300, 264, 128), (2100, 2500, 1040)]
    elif split == 1:
        sizes = [(1, 1, 16), (tn, 128, 128), (tn + 1, 257, 144), (3 * tn - 1, 300, 1168), (7 * tn + 3, 2570, 1040)]
    else:
        sizes = [(1, 1, 128 * split), (tn, 128, 128 * split - 112), (tn - 1, 130, 1040), (tn, 257, 1152), (tn + 1, 300, 2064),
                 (2 * tn - 3, 520, 2304)]
    return [z for z in sizes if F.fits(tn, split, *z, sms())]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("form", F.FORMS)
def test_exact_products(form, dt):
    """Integers whose sums fp32 holds, scaled by powers of two that differ from block to block, row to row and weight
    tile to weight tile: exact whatever the order, so a lost, doubled or misplaced part shows."""
    done = problems(form)
    assert len(done) >= 3, done
    for M, N, K in done:
        (a, sa, w, sw), _ = integers(M + N + K, M, N, K)
        g = torch.Generator(device="cuda").manual_seed(K)
        sa *= 2.0 ** torch.randint(-1, 2, sa.shape, generator=g, device="cuda")
        sw *= 2.0 ** torch.randint(-1, 2, sw.shape, generator=g, device="cuda")
        bias = torch.randint(-64, 65, (N,), generator=g, device="cuda").float()
        want = R.fp8_linear(a, sa, w, sw, bias)[0]  # below 64 * 4 * 2304 + 64 in quarters: 22 bits
        out = torch.full((M * N + 64,), 7.0, dtype=dt, device="cuda")
        y, status = F.run(form, a, sa, w, sw, bias, y=out[32:-32].view(M, N))
        assert torch.equal(y, want.float().to(dt)) and int(status) == 0, (M, N, K)
        assert (out[:32] == 7).all() and (out[-32:] == 7).all()


@pytest.mark.parametrize("form", F.FORMS)
def test_nan_and_the_largest_codes(form):
    """A NaN code reaches its own row or column alone; sums of the largest products; zero scales leave the bias."""
    M, N, K = problems(form)[-1]
    (a, sa, w, sw), want = integers(5, M, N, K)
    w.view(torch.uint8)[N // 2, K - 3] = 0x7F
    y, _ = F.run(form, a, sa, w, sw)
    assert y[:, N // 2].isnan().all() and int(y.isnan().sum()) == M
    assert torch.equal(y[:, :N // 2].double(), want[:, :N // 2]) and torch.equal(y[:, N // 2 + 1:].double(), want[:, N // 2 + 1:])
    w.view(torch.uint8)[N // 2, K - 3] = 0
    a.view(torch.uint8)[M - 1, 3] = 0xFF
    y, _ = F.run(form, a, sa, w, sw)
    assert y[M - 1].isnan().all() and int(y.isnan().sum()) == N
    big = torch.full((M, K), 448.0, device="cuda").to(E8), torch.full((N, K), -448.0, device="cuda").to(E8)
    y, _ = F.run(form, big[0], sa, big[1], sw)
    # 448^2 = 49 * 2^12 times at most 2304: 17 bits of it, every partial sum exact
    assert torch.equal(y, torch.full_like(y, -448.0 * 448.0 * K))
    bias = torch.randn(N, generator=torch.Generator().manual_seed(3)).cuda()
    y, _ = F.run(form, big[0], torch.zeros_like(sa), big[1], sw, bias)
    assert torch.equal(y, bias.expand(M, N))


@pytest.mark.parametrize("form", F.FORMS)
def test_calls_without_waits_between_them(form):
    """Each launch may start before the one ahead of it has ended (programmatic launches) but reads only what that
    has finished: a chain through one pair of buffers equals the same calls one at a time."""
    tn, split = form
    M, K = (700 if tn == 0 else 2 * tn if split == 1 else tn), 1152 if split > 1 else 640
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randint(-8, 9, (K, K), generator=g, device="cuda").float().to(E8)
    nb = -(-K // 128)
    sw = torch.ones((nb, nb), device="cuda")
    from w4a8_block_quantized_gb300 import binding as b
    x0 = torch.randn((M, K), generator=g, device="cuda")
    assert F.fits(tn, split, M, K, K, sms())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def chain(wait):
        x = x0.clone()
        a, sa = b.quant_fp8(x)
        for _ in range(30):
            F.run(form, a, sa, w, sw, y=x, status=status)
            if wait:
                torch.cuda.synchronize()
            x.mul_(2.0 ** -8)
            b.quant_fp8(x, a_q=a, a_scale=sa)
            F.run(form, a, sa, w, sw, y=x, status=status)  # directly behind the library's kernel, itself launched early
            if wait:
                torch.cuda.synchronize()
            b.quant_fp8(x, a_q=a, a_scale=sa)
            if wait:
                torch.cuda.synchronize()
            sa.mul_(2.0 ** -8)
        return x

    want = chain(True)
    assert want.isfinite().all() and want.abs().max() > 0
    for _ in range(4):
        assert torch.equal(chain(False), want) and int(status) == 0


def test_public_calls_take_each_form():
    """Over tokens 1 to 8192, outputs 64 to 14336 and inputs 128 to 14336: the smallest problem found for each form that
    the rule picks on this GPU, called publicly, gives the bits of that form and the right values."""
    from w4a8_block_quantized_gb300 import binding as b
    fit = {(t, s): F.lib().forms_clusters(t, s) for t in F.TILES for s in F.SPLITS}
    rng = random.Random(0)

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    found = {}
    for _ in range(20000):
        M, N, K = log(1, 8192), log(64, 14336), 16 * log(8, 896)
        form = F.pick(M, N, K, sms(), lambda t, s: fit[t, s])
        found[form] = min(found.get(form, (math.inf,)), (M * N * K, M, N, K))
    assert {t for t, _ in found} == {0, *F.TILES} and {s for _, s in found} == set(F.SPLITS), found
    for form, (_, M, N, K) in found.items():
        assert F.fits(*form, M, N, K, sms()), (form, M, N, K)
        g = torch.Generator(device="cuda").manual_seed(M + N + K)
        a, sa = b.quant_fp8(torch.randn((M, K), generator=g, device="cuda"))
        w = (torch.randn((N, K), generator=g, device="cuda") * 120).clamp(-448, 448).to(E8)
        sw = (torch.rand((-(-N // 128), -(-K // 128)), generator=g, device="cuda") + 0.1) * 1e-3
        y = b.fp8_linear(a, sa, w, sw)
        assert torch.equal(y, F.run(form, a, sa, w, sw)[0]), (form, M, N, K)
        ref, mag = R.fp8_linear(a, sa, w, sw, None)
        assert ((y.double() - ref).abs() <= R.fp8_linear_allowed(ref, mag, K, False)).all(), (form, M, N, K)
    assert b.sync_status() == 0
