"""GPU tests of the cache and of attention over it at the edges of what a call may hold: shared memory that earlier
kernels left full, numbers that are none, extremes of the types, streams."""
import math

import pytest
import torch

import attention_ref as R
from test_gpu_attention import BF, E8, F32, I8, B, _lib, attend, near, normal, problem, reference  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,G", [(1, 2), (4, 4), (4, 8)])
@pytest.mark.parametrize("D", [64, 128])
def test_clusters_after_full_shared_memory(D, n, G):
    """One launch for short keys, again and again behind kernels that leave shared memory full of numbers: what a CTA
    sets up there is set up before any of its warps looks at it."""
    p = problem(n + G, [(n, 500), (n, 90), (n, 300)], 2, G, D, 16, I8)
    wide = problem(1, [(300, 300)], 2, 4, D, 16, I8)
    assert B().attention_workspace_bytes(p["q"], p["cache"], 3, p["max_q"], p["max_kv"]) == 0
    want, allowed = reference(p)
    first = attend(p)
    near(first, want, allowed)
    for _ in range(100):
        attend(wide)
        assert torch.equal(attend(p), first)


def over_freed_blocks(call, *sizes):
    """`call` on another stream while the current one still reads blocks of these many bytes that it has freed: what was
    read of them."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.full((n,), 0x3C, dtype=torch.uint8, device="cuda") for n in sizes]
    seen = [torch.empty_like(t) for t in held]
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    for s, t in zip(seen, held):
        s.copy_(t)
    del held, t
    got = call(side)
    side.synchronize()
    torch.cuda.synchronize()
    return got, all(bool((s == 0x3C).all()) for s in seen)


def test_another_streams_outputs_leave_memory_in_use_alone():
    """A call on another stream allocates its outputs and workspaces where that stream may write at once, not in blocks
    that the current stream has just freed and still reads."""
    cache = B().KVCache.empty(64, 8, 64, 128)
    x, slots = normal(2, 1024, 8, 128).to(BF), torch.arange(1024, device="cuda")
    pos, table = slots.int(), B().rope_table(128)
    size = x.numel() * 2
    want = B().kv_write(cache, x, x, slots, pos, table, q=x)
    back = B().kv_read(cache, slots)
    p = problem(5, [(300, 700)] * 2, 2, 4, 128, 32, I8)
    need = B().attention_workspace_bytes(p["q"], p["cache"], 2, p["max_q"], p["max_kv"])
    out = attend(p)
    for call, expect, sizes in ((lambda s: B().rope(x, pos, table, stream=s), want, (size,)),
                                (lambda s: B().kv_write(cache, x, x, slots, pos, table, q=x, stream=s), want, (size,)),
                                (lambda s: torch.stack(B().kv_read(cache, slots, stream=s)), torch.stack(back), (size, size)),
                                (lambda s: attend(p, stream=s), out, (out.numel() * 2, need))):
        got, kept = over_freed_blocks(call, *sizes)
        assert kept and torch.equal(got, expect)


def test_another_streams_outputs_of_the_linears():
    """The same of the calls around the attention."""
    x, w = normal(1, 512, 1024), torch.ones(1024, device="cuda")
    codes = torch.randint(0, 256, (640, 512), dtype=torch.uint8, device="cuda")
    ws, wz = torch.full((640, 16), 0.01, dtype=torch.float16, device="cuda"), torch.full((640, 16), 8.0, dtype=torch.float16, device="cuda")
    a, s, r = B().quant_pack(x)
    act, pw = B().prepare_activations(x), B().prepare_weights(codes, ws, wz)
    e, es = B().quant_fp8(x)
    we, wes = normal(2, 640, 1024).to(E8), torch.ones((5, 8), device="cuda")
    y, M, N, K = 512 * 640 * 4, 512, 640, 1024
    for name, call, sizes in (
            ("quant_pack", lambda st: B().quant_pack(x, stream=st), (M * K, M * 4, M * K // 16)),
            ("linear", lambda st: B().linear(a, s, r, codes, ws, wz, stream=st), (y, B().linear_workspace_bytes(M, N, K))),
            ("prefill_linear", lambda st: B().prefill_linear(x, codes, ws, wz, stream=st), (y, B().prefill_workspace_bytes(M, N, K))),
            ("batch", lambda st: B().prefill_linear_batch([dict(x=x, wq=codes, s_w=ws, z_w=wz)], stream=st), (y, B().prefill_workspace_bytes(M, N, K))),
            ("prefill_linear_ex", lambda st: B().prefill_linear_ex(x, codes, ws, wz, out_dtype=BF, stream=st), (y // 2, B().prefill_workspace_bytes(M, N, K))),
            ("prepare_activations", lambda st: B().prepare_activations(x, stream=st), (B().prepared_activations_bytes(M, K),)),
            ("prepare_weights", lambda st: B().prepare_weights(codes, ws, wz, stream=st), (B().prepared_weights_bytes(N, K),)),
            ("linear_prepared", lambda st: B().linear_prepared(act, pw, M, N, K, stream=st), (y,)),
            ("linear_act", lambda st: B().linear_act(act, codes, ws, wz, M, N, K, stream=st), (y,)),
            ("rmsnorm_quant_fp8", lambda st: B().rmsnorm_quant_fp8(x, w, 1e-5, residual=x, stream=st), (M * K, M * 32, M * K * 4)),
            ("rmsnorm_prepare", lambda st: B().rmsnorm_prepare(x, w, 1e-5, stream=st), (B().prepared_activations_bytes(M, K),)),
            ("swiglu_quant", lambda st: B().swiglu_quant(x, x, stream=st), (M * K, M * 4, M * K // 16)),
            ("quant_fp8", lambda st: B().quant_fp8(x, stream=st), (M * K, M * 32)),
            ("fp8_linear", lambda st: B().fp8_linear(e, es, we, wes, stream=st), (y,))):
        want = call(None)
        got, kept = over_freed_blocks(call, *sizes)
        assert kept, name
        for g, t in zip(*((v,) if isinstance(v, torch.Tensor) else v for v in (got, want))):
            assert (g is None and t is None) or torch.equal(g.view(torch.uint8), t.view(torch.uint8)), name


FORMS = [(1, 2, [1], 0), (1, 2, [300, 2, 40], 0), (1, 16, [1, 700], 0), (2, 7, [900, 2, 130], 20000), (4, 8, [2500, 700, 4], 20000), (90, 2, [400, 90], 0),
         (70, 1, [6000], 0), (60, 2, [400, 60], 2 ** 30)]


def form(seed, n, G, lens, most, fmt, D=128):
    """A problem whose bound on the keys, `most`, picks one of the ways that the work is cut."""
    p = problem(seed, [(n, kv) for kv in lens], 2, G, D, 16, fmt)
    p["max_kv"] = max(p["max_kv"], most)
    if 0 < most < 2 ** 20:
        p["table"] = torch.nn.functional.pad(p["table"], (0, most // 16 - p["table"].shape[1]), value=-7)
    return p


@pytest.mark.parametrize("fmt", [I8, E8])
@pytest.mark.parametrize("code", [50, -50])
@pytest.mark.parametrize("n,G,lens,most", FORMS, ids=str)
def test_an_infinite_query_over_codes_of_one_sign(n, G, lens, most, code, fmt):
    """All logits are infinite, of one sign: NaN whichever it is, for one visible key and for many; the other rows as
    they were."""
    p = form(n, n, G, lens, most, fmt)
    p["cache"].k[..., 5] = torch.tensor(code, device="cuda").to(fmt)
    want, allowed = reference(p)
    hurt = [(0, 1), (p["q"].shape[0] - 1, 0), (n // 2, 2 * G - 1), (p["q"].shape[0] - n, G)]
    for i, (t, h) in enumerate(hurt):
        p["q"][t, h, 5] = math.inf if i % 2 else -math.inf
    out = attend(p)
    rest = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    for t, h in hurt:
        rest[t, h] = False
        assert out[t, h].isnan().all(), (t, h)
    near(out[rest], want.to(out.device)[rest], allowed.to(out.device)[rest])


@pytest.mark.parametrize("n,G,lens,most", FORMS, ids=str)
def test_logits_below_the_smallest_number(n, G, lens, most):
    """Scale, queries and keys whose product vanishes in fp32: plain means of what is seen, hidden keys stay hidden."""
    p = form(n + 2, n, G, lens, most, E8)
    for scale in (1e-45, 1e-38):
        want, allowed = reference(p, scale=scale)
        near(attend(p, scale=scale), want, allowed)
        want, allowed = reference(p, scale=scale, window=40, sinks=3)
        near(attend(p, scale=scale, window=40, sinks=3), want, allowed)
    p["q"] *= 2.0 ** -110
    p["cache"].k_scale.mul_(2.0 ** -60)
    want, allowed = reference(p)
    near(attend(p), want, allowed)


@pytest.mark.parametrize("q_dt", [BF, F32])
@pytest.mark.parametrize("n,G,lens,most", FORMS, ids=str)
def test_queries_at_the_ends_of_their_type(n, G, lens, most, q_dt):
    """Rows of every magnitude that the type has, down to its smallest normal numbers and up to its largest."""
    p = form(n + 1, n, G, lens, most, I8)
    q = p["q"] = p["q"].to(q_dt)
    for i, e in enumerate((-126, -124, -121, -120, -119, -100, 100, 126)):
        t, h = i * (q.shape[0] - 1) // 7, i % q.shape[1]
        q[t, h] = (q[t, h].float().clamp(-1.9, 1.9) * 2.0 ** e).to(q_dt)
    q[-1, -1] = torch.finfo(q_dt).max
    q[0, 0, ::2] = -torch.finfo(q_dt).max
    scale = 2.0 ** -126
    want, allowed = reference(p, scale=scale)
    near(attend(p, scale=scale), want, allowed)
    q[-1, -1], q[0, 0] = 2.0 ** -126, 2.0 ** -125
    p["q"] = torch.where(q.float().abs() > 2.0 ** 20, 0.0, q.float()).to(q_dt)
    want, allowed = reference(p)
    near(attend(p), want, allowed)


@pytest.mark.parametrize("fmt", [I8, E8])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("n,G,lens,most", FORMS, ids=str)
def test_a_key_or_value_that_is_no_number(n, G, lens, most, which, fmt):
    """A place whose scale is NaN: the rows that see it are NaN, no other is touched."""
    for window in (dict(), dict(window=50, sinks=3)):
        p = form(n + 3, n, G, lens, most, fmt)
        c = p["cache"]
        want, allowed = reference(p, **window)
        hurt = torch.zeros(p["q"].shape[:2], dtype=torch.bool, device="cuda")
        for b, kv in enumerate(lens):
            for j, h in ((max(0, kv - 1 - n // 2), 0), (max(0, kv - 60), 1)):
                page = int(p["table"][b, j // 16])
                (c.k_scale if which == "k" else c.v_scale)[page, h, j % 16] = math.nan
                (c.k if which == "k" else c.v).view(torch.uint8)[page, h, j % 16] = 0
                for i in range(n):
                    at = kv - n + i
                    if j <= at and (not window or j > at - 50 or j < 3):
                        hurt[b * n + i, h * G:(h + 1) * G] = True
        out = attend(p, **window)
        assert out[hurt].isnan().all()
        rest = ~hurt
        near(out[rest], want.to(out.device)[rest], allowed.to(out.device)[rest])


@pytest.mark.parametrize("fmt", [I8, E8])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf], ids=str)
@pytest.mark.parametrize("D,rot", [(128, 0), (64, 32)])
def test_rows_that_are_no_numbers_in_the_cache(D, rot, bad, dt, fmt):
    """A key's or value's row with an element that is no finite number is kept as such: scale NaN, codes 0, read back as
    NaN; the others are stored as ever."""
    T, KV = 37, 3
    cache = B().KVCache.empty(4, KV, 16, D, fmt)
    k, v = normal(1, T, KV, D).to(dt), normal(2, T, KV, D).to(dt)
    slots = torch.arange(T, device="cuda")
    turn = (slots.int(), B().rope_table(rot)) if rot else ()
    B().kv_write(cache, k, v, slots, *turn)
    good, held = B().kv_read(cache, slots), [t.clone() for t in (cache.k.view(torch.uint8), cache.v.view(torch.uint8))]
    broken = [torch.zeros((T, KV), dtype=torch.bool, device="cuda") for _ in "kv"]
    for i, (t, h, d) in enumerate(((0, 0, 0), (5, 2, D - 1), (T - 1, 1, 17), (20, 0, rot // 2))):
        (k, v)[i % 2][t, h, d] = bad
        broken[i % 2][t, h] = True
    v[9, 1], broken[1][9, 1] = bad, True
    B().kv_write(cache, k, v, slots, *turn)
    for got, was, mask, codes, before, scale in zip(B().kv_read(cache, slots), good, broken, (cache.k, cache.v), held, (cache.k_scale, cache.v_scale)):
        assert got[mask].isnan().all() and torch.equal(got[~mask], was[~mask])
        assert not R.rows(codes.view(torch.uint8), slots, 16)[mask].any() and R.rows(scale, slots, 16)[mask].isnan().all()
        assert torch.equal(R.rows(codes.view(torch.uint8), slots, 16)[~mask], R.rows(before, slots, 16)[~mask])


def test_one_workspace_for_every_smaller_call():
    """Sized once for the largest step, it serves the smaller ones, whichever way they are cut."""
    most = dict(batch=4, total=900, max_q=300, max_kv=20000)
    ws = None
    for lens, kv in (([(300, 700)] * 3, 700), ([(1, 300)] * 4, 512), ([(1, 3000)] * 3, 20000), ([(5, 900), (2, 40)], 20000), ([(130, 4000)], 4096)):
        p = problem(len(lens), lens, 2, 4, 128, 32, I8)
        p["max_kv"] = max(p["max_kv"], kv)
        p["table"] = torch.nn.functional.pad(p["table"], (0, 640 - p["table"].shape[1]), value=-7)
        if ws is None:
            ws = B().workspace(B().attention_workspace_bound(p["cache"], 8, **most), "cuda")
        ws.fill_(0xFF)
        assert B().attention_workspace_bytes(p["q"], p["cache"], len(lens), p["max_q"], p["max_kv"]) <= ws.numel()
        want, allowed = reference(p)
        near(attend(p, ws=ws), want, allowed)


def test_a_tape_holds_what_its_calls_allocated():
    """Outputs and workspaces that recorded calls made for themselves live as long as the tape: later allocations get other
    memory, and a replay writes none that is theirs."""
    p = problem(5, [(1, 3000)] * 3, 2, 4, 128, 32, I8)
    p["max_kv"] = 20000
    p["table"] = torch.nn.functional.pad(p["table"], (0, 20000 // 32 - p["table"].shape[1]), value=-7)
    need = B().attention_workspace_bytes(p["q"], p["cache"], 3, p["max_q"], p["max_kv"])
    assert need > 1 << 20
    want = attend(p)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        warm = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)] + [torch.empty_like(want) for _ in range(2)]
        del warm
        torch.cuda.synchronize()
        with B().Tape(s) as tape:
            out = attend(p)
        others = [torch.full((need,), 0x77, dtype=torch.uint8, device="cuda") for _ in range(3)]
        out.zero_()
        for _ in range(3):
            tape.replay(s)
        s.synchronize()
        assert torch.equal(out, want)
        assert all((t == 0x77).all() for t in others)
        tape.free()


@pytest.mark.parametrize("up", [90, -90])
@pytest.mark.parametrize("n,G,lens,most", FORMS, ids=str)
def test_value_scales_far_apart(n, G, lens, most, up):
    """Keys whose values are 2^90 of the others': the small ones add to the weights' sum all the same."""
    p = form(n + 4, n, G, lens, most, I8)
    c = p["cache"]
    for b, kv in enumerate(lens):
        for j in range(kv // 2, kv):
            c.v_scale[int(p["table"][b, j // 16]), :, j % 16] *= 2.0 ** up
    want, allowed = reference(p)
    near(attend(p), want, allowed)
