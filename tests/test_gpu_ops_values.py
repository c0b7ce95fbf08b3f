"""GPU tests of the gated activation's values, against fp64 within its derived error: every number of chunks a
lane, rows that end inside a half warp, strided halves, outputs between guards."""
import numpy as np
import pytest
import torch

import ops_ref as R

pytestmark = pytest.mark.gpu
BF, F32, E8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a8_block_quantized_gb300 import binding, build
    build.build()
    binding.load()
    torch.cuda.set_device(0)
    yield
    assert binding.sync_status() == 0


def B():
    from w4a8_block_quantized_gb300 import binding
    return binding


def silu_mul(g, u):
    """fp64 silu(g) u on the tensors' device, and its relative error in fp32 as the header states it: the power's argument
    (1.224 |g| units of 2^-24), the power (2^-22) and what either moves the sum by, a sum, a reciprocal (2^-23), two
    products; all of it where the kernel's reciprocal is 0."""
    g, u = g.double(), u.double()
    part = 1.0 / (1.0 + torch.exp(g))
    err = (5.1 + (4.1 + 1.23 * g.abs()) * part) * R.U
    return g / (1.0 + torch.exp(-g)) * u, torch.where(g < -87.3, torch.ones_like(g), err)


def guarded(shape, dtype):
    n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
    buf = torch.full((n + 128,), 0x5A, dtype=torch.uint8, device="cuda")
    return buf[64:64 + n].view(dtype).view(shape), lambda: bool((buf[:64] == 0x5A).all() and (buf[64 + n:] == 0x5A).all())


@pytest.mark.parametrize("dt", [BF, F32])
def test_each_value(dt):
    """One live value a row, which the row's scale then shows to within its own division: gates over the whole range."""
    g = torch.cat([torch.linspace(-100, 100, 8001), torch.linspace(-2, 2, 4001), torch.tensor([-89.0, -88.5, -87.0, 88.0, 89.0]),
                   torch.logspace(-30, 2, 500), -torch.logspace(-30, 2, 500)]).cuda().to(dt)
    u = (torch.randn(g.shape, generator=torch.Generator().manual_seed(1)).cuda() + 2).to(dt)
    gate, up = torch.zeros((len(g), 64), dtype=dt, device="cuda"), torch.ones((len(g), 64), dtype=dt, device="cuda")
    gate[:, 9], up[:, 9] = g, u
    t, err = silu_mul(g, u)
    q, s, _ = B().swiglu_quant(gate, up)
    seen = (s.double() * 127 / t.abs() - 1).abs()
    gone = g.double() < -87.3
    assert (seen <= err + R.U)[~gone].all(), float((seen / (err + R.U))[~gone].max())
    assert (s[g.double() < -89] == 0).all() and ((s.double() * 127)[gone] <= 1.1e-36 * u.double().abs()[gone]).all()
    live = s > 0
    assert (q[live, 9].float() == 127 * torch.sign(t[live]).float()).all() and not q[:, 10:].any() and not q[:, :9].any()
    # e4m3: the group's scale, where it is not too small for one
    q, s = B().swiglu_quant_fp8(gate, up)
    ok = t.abs() > 2.0 ** -99
    assert ((s[0].double() * 448 / t.abs() - 1).abs() <= err + R.U)[ok].all()


# rows x columns: one chunk a lane, two, four (by the rows and the type), and last parts that end inside a half warp
SHAPES = [(3, 272), (40, 6160), (512, 6144), (700, 6000), (300, 14320), (1900, 14320), (2600, 1040), (8192, 2064)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,K", SHAPES)
def test_e4m3_codes(M, K, dt):
    """Each code is the rounding of some value within the error of t and of the group's scale."""
    gen = torch.Generator(device="cuda").manual_seed(M + K)
    wide = torch.empty((M, 2 * K + 24), dtype=dt, device="cuda")
    wide[:] = torch.randn(wide.shape, generator=gen, device="cuda") * 2
    wide[:, 11] = -200.0
    gate, up = wide[:, 8:8 + K], wide[:, 16 + K:16 + 2 * K]  # 16-byte aligned halves with a gap
    nb = -(-K // 128)
    a_q, ok_q = guarded((M, K), E8)
    a_scale, ok_s = guarded((nb, M), F32)
    q, s = B().swiglu_quant_fp8(gate, up, a_q=a_q, a_scale=a_scale)
    assert ok_q() and ok_s()
    t, err = silu_mul(gate, up)
    pad = torch.nn.functional.pad
    tg, eg = pad(t, (0, nb * 128 - K)).view(M, nb, 128), pad(err, (0, nb * 128 - K)).view(M, nb, 128)
    top, at = tg.abs().max(-1)
    # the group's largest: that of the values whose range reaches past the lowest end of the ranges' largest
    near = (tg.abs() * (1 + eg)) >= (tg.abs() * (1 - eg)).max(-1, keepdim=True).values
    terr = torch.where(near, eg, torch.zeros_like(eg)).max(-1).values
    seen = (s.t().double() * 448 / top - 1).abs()
    assert (seen <= terr + R.U).all(), float((seen / (terr + R.U)).max())
    # code = e4m3(t * fl(448 / max)): the error of t, of the largest, of the division and the product
    v = tg / top[..., None] * 448
    slack = eg + terr[..., None] + 2.1 * R.U
    lo = R.e4m3((v.abs() * (1 - slack)).clamp(min=0).cpu().numpy())
    hi = R.e4m3((v.abs() * (1 + slack)).cpu().numpy())
    code = pad(q.view(torch.uint8), (0, nb * 128 - K)).view(E8).view(M, nb, 128).double()
    mag, sign = code.abs().cpu().numpy(), (code * tg).cpu().numpy()
    assert (mag >= lo).all() and (mag <= hi).all() and (sign >= 0).all()


@pytest.mark.parametrize("given", [True, False])
def test_one_row_of_an_odd_width(given):
    """A row of an array whose width no 16 bytes divide, with outputs given and not."""
    K = 256
    wide = torch.randn((1, 2 * K + 3), generator=torch.Generator().manual_seed(2)).cuda().to(BF)
    gate, up = wide[:, :K], wide[:, K:2 * K]
    want = B().swiglu_quant_fp8(gate.clone(), up.clone())
    out = dict(a_q=torch.empty((1, K), dtype=torch.uint8, device="cuda").view(E8),
               a_scale=torch.empty((2, 1), device="cuda")) if given else {}
    got = B().swiglu_quant_fp8(gate, up, **out)
    assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1])
