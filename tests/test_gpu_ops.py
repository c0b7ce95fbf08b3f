"""GPU tests of the operators around the linears: norm + residual and gated activation with an
8-bit output, and the e4m3 linear, against plain restatements (tests/ops_ref.py)."""
import numpy as np
import pytest
import torch

import ops_ref as R

pytestmark = pytest.mark.gpu
EPS = 1e-6
BF, F32 = torch.bfloat16, torch.float32


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


def normal(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda") * scale


def hidden(seed, M, K, dt):
    x = normal(seed, M, K)
    x[:, torch.randperm(K, generator=torch.Generator().manual_seed(seed))[:4].cuda()] *= 20
    return x.to(dt)


def f32(t):
    return None if t is None else t.float().cpu().numpy()


def code_values(q):
    return q.float().cpu().numpy().astype(np.float64)


def guarded(shape, dtype, fill=0x5A):
    """A tensor of `shape` with 64 guard bytes on each side, and a check that they are untouched."""
    n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
    buf = torch.full((n + 128,), fill, dtype=torch.uint8, device="cuda")
    t = buf[64:64 + n].view(dtype).view(shape)
    return t, lambda: bool((buf[:64] == fill).all()) and bool((buf[64 + n:] == fill).all())


ROWS = [(1, 64), (3, 128), (5, 192), (1, 4096), (7, 2048), (129, 1024), (300, 320), (33, 6144), (9, 14336),
        (200, 8256), (3, 32768), (2, 33024), (153, 40960),
        (7400, 2048), (3700, 2112), (1900, 14336)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("with_res", [True, False])
@pytest.mark.parametrize("M,K", ROWS)
def test_norm_int8(M, K, with_res, dt):
    x = hidden(M + K, M, K, dt)
    res = normal(M * K, M, K, scale=2).to(dt) if with_res else None
    w = 1 + 0.1 * normal(K, K)
    a_q, ok_q = guarded((M, K), torch.int8)
    q, s, rs, out = B().rmsnorm_quant(x, w, EPS, residual=res, a_q=a_q)
    h = R.norm_sum(f32(x), f32(res))
    cq, cs, crs = R.int8_rows((h * f32(w)).astype(np.float32))
    r, tol = R.norm_factor(h, EPS)
    assert np.array_equal(q.cpu().numpy(), cq) and np.array_equal(rs.cpu().numpy(), crs) and ok_q()
    np.testing.assert_allclose(s.cpu().numpy(), cs * r, rtol=tol, atol=0)
    if with_res:
        assert torch.equal(out, (x.float() + res.float()).to(dt))
    else:
        assert out is None


E_ROWS = [(1, 16), (3, 48), (2, 128), (1, 4096), (7, 2064), (129, 1024), (300, 336), (33, 6160), (9, 14336),
          (3, 32768), (2, 33040), (153, 40960), (3700, 2064), (1900, 14320)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,K", E_ROWS)
def test_norm_e4m3(M, K, dt):
    x, res, w = hidden(M + K, M, K, dt), normal(M * K, M, K, scale=2).to(dt), 1 + 0.1 * normal(K, K)
    a_q, ok_q = guarded((M, K), torch.float8_e4m3fn)
    sc, ok_s = guarded(((K + 127) // 128, M), F32)
    q, s, out = B().rmsnorm_quant_fp8(x, w, EPS, residual=res, a_q=a_q, a_scale=sc)
    h = R.norm_sum(f32(x), f32(res))
    cq, cs = R.e4m3_rows((h * f32(w)).astype(np.float32))
    r, tol = R.norm_factor(h, EPS)
    assert np.array_equal(code_values(q), cq) and ok_q() and ok_s()
    np.testing.assert_allclose(s.cpu().numpy(), cs * r[None, :], rtol=tol, atol=0)
    assert torch.equal(out, (x.float() + res.float()).to(dt))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,K", E_ROWS)
def test_quant_e4m3(M, K, dt):
    x = hidden(M * 3 + K, M, K, dt)
    a_q, ok_q = guarded((M, K), torch.float8_e4m3fn)
    sc, ok_s = guarded(((K + 127) // 128, M), F32)
    q, s = B().quant_fp8(x, a_q=a_q, a_scale=sc)
    cq, cs = R.e4m3_rows(f32(x))
    assert np.array_equal(code_values(q), cq) and np.array_equal(s.cpu().numpy(), cs) and ok_q() and ok_s()


@pytest.mark.parametrize("K", [256, 4096, 33024])
def test_degenerate_rows(K):
    """Zero rows, one live value, rows of tiny values (scales in the subnormal range), a group of
    zeros in a live row, the largest sums of a bf16 stream that fp32 squares still hold."""
    x = torch.zeros((7, K), device="cuda")
    x[1, 5] = 3.0
    x[2] = normal(1, K, scale=1e-38)
    x[3] = normal(2, K, scale=1e-30)
    x[4, 128:] = normal(3, K - 128)
    x[5] = 1e17 * torch.sign(normal(4, K))
    x[6] = normal(5, K)
    w = torch.ones(K, device="cuda")
    h = f32(x)
    r, tol = R.norm_factor(h, EPS)
    q, s, rs, _ = B().rmsnorm_quant(x, w, EPS)
    cq, cs, crs = R.int8_rows(h)
    assert np.array_equal(q.cpu().numpy(), cq) and np.array_equal(rs.cpu().numpy(), crs)
    np.testing.assert_allclose(s.cpu().numpy(), cs * r, rtol=tol, atol=1e-44)
    q, s, _ = B().rmsnorm_quant_fp8(x, w, EPS)
    cq, cs = R.e4m3_rows(h)
    assert np.array_equal(code_values(q), cq)
    np.testing.assert_allclose(s.cpu().numpy(), cs * r[None, :], rtol=tol, atol=0)


def test_e4m3_ties_go_to_even():
    """A group whose largest value is 448 has scale 1 and factor 1: codes are the plain rounding of
    the values, ties to even, in the normal and subnormal range."""
    vals = np.zeros(128, np.float32)
    vals[:12] = [448, 1.0625, 1.1875, -1.0625, 17, 19, 2.0 ** -10, 3 * 2.0 ** -10, 5 * 2.0 ** -10, 240, 0.0146484375, -0.0]
    q, s = B().quant_fp8(torch.from_numpy(vals[None]).cuda())
    assert s.cpu().numpy().tolist() == [[1.0]]
    want = [448, 1.0, 1.25, -1.0, 16, 20, 0.0, 2.0 ** -8, 2.0 ** -8, 240, 0.015625, 0.0]
    assert code_values(q)[0, :12].tolist() == want


def between(q, v, err, rounding):
    """Codes q are the rounding of some value within the relative error of v."""
    lo, hi = rounding(v * (1 - np.sign(v) * err)), rounding(v * (1 + np.sign(v) * err))
    return np.all((q >= lo) & (q <= hi))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,K", [(1, 64), (1, 6144), (5, 192), (129, 1024), (33, 14336), (2, 33024)])
def test_swiglu(M, K, dt):
    gu = normal(M + K, M, 2 * K, scale=2).to(dt)
    gu[:, 3] = -200.0  # silu's left limit
    gate, up = gu[:, :K], gu[:, K:]
    t, err = R.swiglu(f32(gate), f32(up))
    # INT8: the row's scale comes from its largest |t|
    q, s, rs = B().swiglu_quant(gate, up)
    sc, serr = np.abs(t).max(1) / 127, (err.max() + 2 * R.U)
    np.testing.assert_allclose(s.cpu().numpy(), sc, rtol=serr)
    v, verr = t / sc[:, None], err + serr + 2 * R.U
    qn = q.cpu().numpy()
    assert between(qn, v, verr, lambda z: np.clip(R.half_away(z), -127, 127))
    assert np.array_equal(rs.cpu().numpy(), qn.reshape(M, -1, 64).astype(np.int32).sum(2))
    # e4m3
    q, s = B().swiglu_quant_fp8(gate, up)
    nb = (K + 127) // 128
    qv = code_values(q)
    for b in range(nb):
        cut = slice(128 * b, 128 * b + 128)
        sg = np.abs(t[:, cut]).max(1) / 448
        np.testing.assert_allclose(s[b].cpu().numpy(), sg, rtol=serr)
        assert between(qv[:, cut], t[:, cut] / sg[:, None], verr[:, cut], R.e4m3)


def test_swiglu_strides_and_single_row():
    """gate and up as halves, as rows of a wider array, and as two arrays of their own."""
    M, K = 37, 512
    wide = normal(1, M, 3 * K + 64).to(BF)
    g, u = wide[:, 64:64 + K], wide[:, 64 + 2 * K:64 + 3 * K]
    ref = B().swiglu_quant_fp8(g.contiguous(), u.contiguous())
    got = B().swiglu_quant_fp8(g, u)
    assert torch.equal(got[0].view(torch.uint8), ref[0].view(torch.uint8)) and torch.equal(got[1], ref[1])
    one = B().swiglu_quant(g[5:6], u[5:6])
    full = B().swiglu_quant(g, u)
    assert torch.equal(one[0], full[0][5:6]) and torch.equal(one[1], full[1][5:6]) and torch.equal(one[2], full[2][5:6])


@pytest.mark.parametrize("M", [1, 8, 9, 300, 4100])
def test_prepared_operand_equals_codes(M):
    """The operand form holds what the INT8 form returns: contractions from either agree bit for bit
    (above 8 tokens, where both take the tensor-core form) or within the linear's tolerance."""
    from w4a8_block_quantized_gb300 import synth
    K, N = 1024, 320
    d = synth.make_weights(synth.LinearSpec("w", M, K, N, True, 20.0, 5, 0))
    wq, sw, zw, bias = (torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in d[1:])
    x, res, w = hidden(M, M, K, BF), normal(M, M, K).to(BF), 1 + 0.1 * normal(3, K)
    gu = normal(M + 1, M, 2 * K)
    pw = B().prepare_weights(wq, sw, zw)
    act, out = B().rmsnorm_prepare(x, w, EPS, residual=res)
    for act, codes in ((act, B().rmsnorm_quant(x, w, EPS, residual=res)),
                       (B().swiglu_prepare(gu[:, :K], gu[:, K:]), B().swiglu_quant(gu[:, :K], gu[:, K:]))):
        y0 = B().linear(*codes[:3], wq, sw, zw, bias)
        for y1 in (B().linear_prepared(act, pw, M, N, K, bias), B().linear_act(act, wq, sw, zw, M, N, K, bias)):
            if M > 8:
                assert torch.equal(y0, y1)
            else:
                # each output is a sum of 16 block terms taken in another order, in fp32
                mag = y0.abs().max()
                assert (y0 - y1).abs().max() <= 1e-5 * mag
    assert torch.equal(out, (x.float() + res.float()).to(BF))


@pytest.mark.parametrize("dt,with_res", [(BF, True), (BF, False), (F32, True)])
def test_prepared_operand_of_many_rows(dt, with_res):
    from w4a8_block_quantized_gb300 import synth
    M, K, N = 7400, 2048, 128
    d = synth.make_weights(synth.LinearSpec("w", M, K, N, True, 20.0, 6, 0))
    wq, sw, zw, bias = (torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in d[1:])
    x, w = hidden(M, M, K, dt), 1 + 0.1 * normal(3, K)
    res = normal(4, M, K).to(dt) if with_res else None
    act, out = B().rmsnorm_prepare(x, w, EPS, residual=res)
    codes = B().rmsnorm_quant(x, w, EPS, residual=res)
    y = B().linear(*codes[:3], wq, sw, zw, bias)
    assert torch.equal(y, B().linear_prepared(act, B().prepare_weights(wq, sw, zw), M, N, K, bias))
    assert out is None if res is None else torch.equal(out, codes[3])


def test_a_row_has_the_same_bits_in_any_batch():
    """Scales too: the sum of squares is taken in an order that depends on the row's length alone."""
    K = 4160
    x, res, w = hidden(1, 4000, K, BF), normal(2, 4000, K).to(BF), 1 + 0.1 * normal(3, K)
    big = B().rmsnorm_quant(x, w, EPS, residual=res)
    for m0, m1 in ((0, 1), (7, 10), (100, 400), (0, 1500)):
        part = B().rmsnorm_quant(x[m0:m1].contiguous(), w, EPS, residual=res[m0:m1].contiguous())
        for a, b in zip(part, big):
            assert torch.equal(a, b[m0:m1])


def test_residual_in_place():
    M, K = 65, 2048
    x, res, w = hidden(1, M, K, BF), normal(2, M, K).to(BF), 1 + 0.1 * normal(3, K)
    q0, s0, out0 = B().rmsnorm_quant_fp8(x, w, EPS, residual=res)
    r1 = res.clone()
    q1, s1, out1 = B().rmsnorm_quant_fp8(x, w, EPS, residual=r1, residual_out=r1)
    assert out1 is r1 and torch.equal(out0, out1) and torch.equal(s0, s1)
    x2 = x.clone()
    q2, s2, out2 = B().rmsnorm_quant_fp8(x2, w, EPS, residual=res, residual_out=x2)
    assert torch.equal(out2, out0) and torch.equal(q2.view(torch.uint8), q0.view(torch.uint8))
    # many rows, which come through shared memory ahead of their turn
    x, res, w = hidden(1, 3700, 4096, BF), normal(2, 3700, 4096).to(BF), 1 + 0.1 * normal(3, 4096)
    q0, s0, out0 = B().rmsnorm_quant_fp8(x, w, EPS, residual=res)
    r1, x2 = res.clone(), x.clone()
    for xx, rr, into in ((x, r1, r1), (x2, res, x2)):
        q1, s1, out1 = B().rmsnorm_quant_fp8(xx, w, EPS, residual=rr, residual_out=into)
        assert torch.equal(out0, out1) and torch.equal(s0, s1) and torch.equal(q0.view(torch.uint8), q1.view(torch.uint8))
    # a row past the register-resident depth
    x, res, w = hidden(1, 3, 33024, F32), normal(2, 3, 33024), 1 + 0.1 * normal(3, 33024)
    q0, _, out0 = B().rmsnorm_quant_fp8(x, w, EPS, residual=res)
    q1, _, out1 = B().rmsnorm_quant_fp8(x, w, EPS, residual=res, residual_out=res)
    assert torch.equal(out0, out1) and torch.equal(q0.view(torch.uint8), q1.view(torch.uint8))


# ------------------------------------------------------------------ e4m3 linear
def operands(seed, M, N, K, big=False):
    a, sa = B().quant_fp8(hidden(seed, M, K, F32))
    nb, nt = (K + 127) // 128, (N + 127) // 128
    w = (normal(seed + 1, N, K) * 120).clamp(-448, 448).to(torch.float8_e4m3fn)
    sw = (normal(seed + 2, nt, nb).abs() + 0.1) * 1e-3
    return a, sa, w, sw, 0.1 * normal(seed + 3, N)


def check_linear(y, a, sa, w, sw, bias, K):
    ref, mag = R.fp8_linear(a, sa, w, sw, bias)
    tol = R.fp8_linear_allowed(ref, mag, K, y.dtype == BF)
    err = (y.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float((err / tol).nan_to_num(1e9).max()))


SHAPES = [(1, 1, 16), (1, 64, 128), (1, 1024, 1024), (2, 130, 144), (8, 3072, 1024), (9, 257, 528), (16, 512, 2048),
          (17, 1000, 1040), (31, 129, 4096), (33, 640, 640), (63, 384, 896), (64, 2048, 6144), (65, 1001, 1040),
          (127, 127, 272), (128, 128, 128), (129, 255, 400), (200, 512, 512), (256, 256, 256), (257, 770, 1040),
          (512, 1024, 2048), (513, 3073, 656), (777, 1001, 1040), (1024, 2048, 1024), (1500, 1111, 272),
          (2050, 4100, 528), (4097, 2571, 1040), (2600, 4104, 16), (1, 14336, 4096), (4, 4096, 14336)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_fp8_linear(M, N, K, dt):
    a, sa, w, sw, bias = operands(M + N + K, M, N, K)
    y, ok = guarded((M, N), dt)
    B().fp8_linear(a, sa, w, sw, bias, y=y)
    check_linear(y, a, sa, w, sw, bias, K)
    assert ok()
    y2 = B().fp8_linear(a, sa, w, sw, out_dtype=dt)
    check_linear(y2, a, sa, w, sw, None, K)
    assert torch.equal(y2, B().fp8_linear(a, sa, w, sw, out_dtype=dt))  # equal calls, equal bits


@pytest.mark.parametrize("M", [1, 40, 300, 2048])
def test_fp8_linear_exact_products(M):
    """Small integers and unit scales: every partial sum is an integer below 2^24, so the result is exact."""
    N, K = 300, 1168
    g = torch.Generator(device="cuda").manual_seed(M)
    a = torch.randint(-8, 9, (M, K), generator=g, device="cuda").float()
    w = torch.randint(-8, 9, (N, K), generator=g, device="cuda").float()
    nb = (K + 127) // 128
    sa, sw = torch.ones((nb, M), device="cuda"), torch.ones((3, nb), device="cuda")
    y = B().fp8_linear(a.to(torch.float8_e4m3fn), sa, w.to(torch.float8_e4m3fn), sw)
    assert torch.equal(y.double(), a.double() @ w.double().T)


@pytest.mark.parametrize("M", [1, 40, 300, 2048])
def test_fp8_linear_nan_and_extremes(M):
    """A NaN code reaches its own row or column alone; the largest codes do not overflow; zero
    scales give the bias."""
    N, K = 260, 512
    a, sa, w, sw, bias = operands(M, M, N, K)
    w.view(torch.uint8)[7, 300] = 0x7F
    y = B().fp8_linear(a, sa, w, sw, bias)
    assert y[:, 7].isnan().all() and int(y.isnan().sum()) == M
    w.view(torch.uint8)[7, 300] = 0
    a.view(torch.uint8)[M - 1, 3] = 0xFF
    y = B().fp8_linear(a, sa, w, sw, bias)
    assert y[M - 1].isnan().all() and int(y.isnan().sum()) == N
    a = torch.full((M, K), 448.0, device="cuda").to(torch.float8_e4m3fn)
    w = torch.full((N, K), -448.0, device="cuda").to(torch.float8_e4m3fn)
    one = torch.ones_like(sa)
    y = B().fp8_linear(a, one, w, torch.ones_like(sw))
    assert torch.equal(y, torch.full_like(y, -448.0 * 448.0 * K))
    y = B().fp8_linear(a, torch.zeros_like(sa), w, sw, bias)
    assert torch.equal(y, bias.expand(M, N))


def test_empty_problems():
    e8 = torch.float8_e4m3fn
    x, w = torch.empty((0, 256), device="cuda"), torch.ones(256, device="cuda")
    assert B().rmsnorm_quant(x, w, EPS)[0].shape == (0, 256)
    assert B().swiglu_quant_fp8(x, x)[1].shape == (2, 0)
    a, sa = B().quant_fp8(x)
    y = B().fp8_linear(a, sa, torch.empty((5, 256), device="cuda").to(e8), torch.ones((1, 2), device="cuda"))
    assert y.shape == (0, 5)
    a, sa = B().quant_fp8(torch.ones((3, 256), device="cuda"))
    assert B().fp8_linear(a, sa, torch.empty((0, 256), device="cuda").to(e8), torch.empty((0, 2), device="cuda")).shape == (3, 0)


def test_offsets_past_32_bits():
    """More than 2^31 elements in the inputs and in the output: the last rows are right."""
    M, K = 525000, 4096 + 64
    x = torch.zeros((M, K), dtype=BF, device="cuda")
    x[-3:] = hidden(1, 3, K, BF)
    w = 1 + 0.1 * normal(2, K)
    q, s, rs, _ = B().rmsnorm_quant(x, w, EPS)
    q3, s3, rs3, _ = B().rmsnorm_quant(x[-3:].clone(), w, EPS)
    assert torch.equal(q[-3:], q3) and torch.equal(s[-3:], s3) and torch.equal(rs[-3:], rs3)
    assert not q[:-3].any()
    a, sa, _ = B().rmsnorm_quant_fp8(x, w, EPS)
    del x, q
    N = 4200
    _, _, wq, sw, bias = operands(3, 1, N, K)
    y = B().fp8_linear(a, sa, wq, sw, bias, out_dtype=BF)  # 2.2e9 outputs from 2.2e9 codes
    a3, sa3 = a[-3:].clone(), sa[:, -3:].contiguous()
    check_linear(y[-3:], a3, sa3, wq, sw, bias, K)
    assert torch.equal(y[0], bias.to(BF)) and torch.equal(y[M // 2], bias.to(BF))


def test_other_streams_and_tapes():
    """The calls run on the stream that they are given, in order, and record into a tape."""
    M, K, N = 96, 1024, 640
    x0, w = hidden(1, M, K, BF), 1 + 0.1 * normal(3, K)
    res = normal(2, M, K).to(BF)
    _, _, wq, sw, bias = operands(3, 1, N, K)
    a, sa, _ = B().rmsnorm_quant_fp8(x0, w, EPS, residual=res)
    want = B().fp8_linear(a, sa, wq, sw, bias)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x, y = torch.zeros_like(x0), torch.zeros_like(want)
    q, sc, out = torch.empty_like(a), torch.empty_like(sa), torch.empty_like(res)
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        x.copy_(x0)
        B().rmsnorm_quant_fp8(x, w, EPS, residual=res, residual_out=out, a_q=q, a_scale=sc, stream=s)
        B().fp8_linear(q, sc, wq, sw, bias, y=y, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    with B().Tape(s) as tape:
        B().rmsnorm_quant_fp8(x, w, EPS, residual=res, residual_out=out, a_q=q, a_scale=sc, stream=s)
        B().fp8_linear(q, sc, wq, sw, bias, y=y, stream=s)
    assert tape.kernels() == 2
    y.zero_()
    x.copy_(x0.flip(0))
    torch.cuda.synchronize()
    tape.replay(s)
    s.synchronize()
    a, sa, _ = B().rmsnorm_quant_fp8(x, w, EPS, residual=res)
    assert torch.equal(y, B().fp8_linear(a, sa, wq, sw, bias))
    tape.free()


@pytest.mark.parametrize("M,K", [(40, 1024), (700, 1024), (2600, 2048), (7400, 2048)])
def test_back_to_back_calls_keep_their_order(M, K):
    """A chain of dependent calls without a wait between them, many times over: each kernel may start
    early (programmatic launch) but reads only finished results.  The sizes reach every form of the
    linear and both kernels of the norm."""
    w = 1 + 0.1 * normal(3, K)
    _, _, wq, sw, _ = operands(3, 1, K, K)
    def chain():
        h = hidden(1, M, K, BF)
        res = normal(2, M, K).to(BF)
        for _ in range(40):
            a, sa, res = B().rmsnorm_quant_fp8(h, w, EPS, residual=res, residual_out=res)
            h = B().fp8_linear(a, sa, wq, sw, out_dtype=BF)
        return h, res
    h0, r0 = chain()
    for _ in range(5):
        h1, r1 = chain()
        assert torch.equal(h0, h1) and torch.equal(r0, r1)
