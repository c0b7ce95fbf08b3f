"""Cases of the operators around the quantized linears of a decoder layer.

Three operators:
  norm    root-mean-square norm with the residual's addition, output in 8 bits with scales: INT8 codes
          per row with their block-64 row sums (what the W4A8 linear takes), or e4m3 codes with one
          scale for 128 columns (what the 8-bit floating-point linear takes)
  linear  matrix product in 8-bit floating point (e4m3) with a scale for each block of 128
  swiglu  silu(gate) * up, output in e4m3 with one scale for 128 columns

Per row of the norm: h = x + residual, r = 1 / sqrt(mean(h^2) + eps), t = h * gamma.  The factor r
is common to a row, so it goes into the scales and the codes are those of t:
  INT8  s = max|t| / 127, code = round half away from zero of t / s, scale = s * r
  e4m3  per 128 columns: code = t * (448 / max|t|) rounded to e4m3, scale = max|t| / 448 * r
Scales of e4m3 activations are laid out [columns / 128][rows].

A case: op, M (tokens), K (columns; of one half for swiglu), N (linear), dtype of the inputs (norm,
swiglu) or of the output (linear), and form ("int8" or "fp8", norm).
"""
import math

import torch

own = False

EPS = 1e-6
BLK = 128


def listed():
    return [
        # one generated token's hidden state before a W4A8 projection: latency alone
        {"name": "norm int8 1x4096", "op": "norm", "form": "int8", "M": 1, "K": 4096, "dtype": "bf16"},
        # a 512-token prompt at hidden size 2048 before the W4A8 projections of a layer
        {"name": "norm int8 512x2048", "op": "norm", "form": "int8", "M": 512, "K": 2048, "dtype": "bf16"},
        # a ragged prompt, fp32 stream, a last scale block of 16 columns
        {"name": "norm fp8 777x6160 f32", "op": "norm", "form": "fp8", "M": 777, "K": 6160, "dtype": "f32"},
        # a long prompt at hidden size 4096 before an 8-bit projection
        {"name": "norm fp8 16384x4096", "op": "norm", "form": "fp8", "M": 16384, "K": 4096, "dtype": "bf16"},
        # one token through an up-projection: latency and the weights' read
        {"name": "linear 1x1024->3072", "op": "linear", "M": 1, "K": 1024, "N": 3072, "dtype": "f32"},
        # eight sequences' tokens through a 7B-class up-projection: the weights' read
        {"name": "linear 8x4096->14336", "op": "linear", "M": 8, "K": 4096, "N": 14336, "dtype": "bf16"},
        # a 512-token prompt, 1.7B-class up-projection
        {"name": "linear 512x2048->6144", "op": "linear", "M": 512, "K": 2048, "N": 6144, "dtype": "bf16"},
        # nothing a multiple of a tile: odd rows and columns, a last block of 16
        {"name": "linear 777x1040->1001", "op": "linear", "M": 777, "K": 1040, "N": 1001, "dtype": "f32"},
        # a long prompt, 7B-class up-projection
        {"name": "linear 8192x4096->14336", "op": "linear", "M": 8192, "K": 4096, "N": 14336, "dtype": "bf16"},
        # one token between the up- and down-projection
        {"name": "swiglu 1x6144", "op": "swiglu", "M": 1, "K": 6144, "dtype": "bf16"},
        # a 512-token prompt, fp32 outputs of the W4A8 linears
        {"name": "swiglu 512x6144 f32", "op": "swiglu", "M": 512, "K": 6144, "dtype": "f32"},
        # a long prompt, 7B-class
        {"name": "swiglu 8192x14336", "op": "swiglu", "M": 8192, "K": 14336, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "swiglu"])
    while True:
        if op == "norm":
            form = rng.choice(["int8", "fp8"])
            unit = 64 if form == "int8" else 16
            c = {"op": op, "form": form, "M": _log(rng, 1, 16384), "K": unit * _log(rng, 256 // unit, 16384 // unit),
                 "dtype": rng.choice(["bf16", "f32"])}
            if c["M"] * c["K"] <= 16384 * 4096:
                return c
        elif op == "linear":
            c = {"op": op, "M": _log(rng, 1, 8192), "K": 16 * _log(rng, 8, 896), "N": _log(rng, 64, 14336),
                 "dtype": rng.choice(["bf16", "f32"])}
            if c["M"] * c["K"] * c["N"] <= 8192 * 4096 * 14336:
                return c
        else:
            c = {"op": op, "M": _log(rng, 1, 8192), "K": 16 * _log(rng, 16, 896), "dtype": rng.choice(["bf16", "f32"])}
            if c["M"] * c["K"] <= 8192 * 14336:
                return c


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _blocks(n):
    return (n + BLK - 1) // BLK


def _grouped(t):
    """t [rows][columns] as [rows][blocks][128], zeros past the last column."""
    rows, cols = t.shape
    return torch.nn.functional.pad(t, (0, _blocks(cols) * BLK - cols)).view(rows, _blocks(cols), BLK)


def _e4m3_groups(t):
    """e4m3 codes of t [rows][columns] fp32 and the scales max / 448 [rows][blocks]."""
    g = _grouped(t)
    amax = g.abs().amax(-1)
    live = amax >= 2.0 ** -100
    inv = torch.where(live, amax.new_full((), 448.0) / amax, torch.zeros_like(amax))
    q = (g * inv[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    q = q.view(t.shape[0], -1)[:, : t.shape[1]].contiguous()
    return q, torch.where(live, amax / amax.new_full((), 448.0), torch.zeros_like(amax))


def _inputs(case, seed):
    """The operator's input tensors, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    M, K, dt = case["M"], case["K"], _dt(case["dtype"])
    out = torch.randperm(K, generator=g, device="cuda")[:4]  # channels with large activations
    if case["op"] == "norm":
        x = normal(M, K)
        x[:, out] *= 20.0
        res = normal(M, K).mul_(2.0)
        gamma = 1.0 + 0.1 * normal(K)
        return {"x": x.to(dt), "res": res.to(dt), "gamma": gamma}
    if case["op"] == "swiglu":
        gu = torch.empty((M, 2 * K), dtype=dt, device="cuda")  # one projection's output: gate | up
        gate = normal(M, K).mul_(1.5)
        gate[:, out] *= 4.0
        gu[:, :K] = gate
        gu[:, K:] = normal(M, K)
        return {"gu": gu}
    N = case["N"]
    x = normal(M, K)
    x[:, out] *= 20.0
    a, sa = _e4m3_groups(x)
    w = normal(N, K).mul_(0.02)
    wb = torch.nn.functional.pad(w, (0, _blocks(K) * BLK - K, 0, _blocks(N) * BLK - N)).view(_blocks(N), BLK, _blocks(K), BLK)
    sw = wb.abs().amax((1, 3)) / 448.0
    w = (wb / sw[:, None, :, None]).clamp(-448.0, 448.0).view(_blocks(N) * BLK, -1)[:N, :K].to(torch.float8_e4m3fn)
    return {"a": a, "sa": sa.t().contiguous(), "w": w.contiguous(), "sw": sw, "bias": 0.1 * normal(N)}


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    M, K, dev = case["M"], case["K"], "cuda"
    # output buffers, as a serving loop keeps them
    if case["op"] == "linear":
        s["y"] = torch.empty((M, case["N"]), dtype=_dt(case["dtype"]), device=dev)
        return s
    if case["op"] == "norm":
        s["res_out"] = torch.empty((M, K), dtype=_dt(case["dtype"]), device=dev)
    if case.get("form") == "int8":
        s["q"] = torch.empty((M, K), dtype=torch.int8, device=dev)
        s["scale"] = torch.empty((M,), dtype=torch.float32, device=dev)
        s["rowsum"] = torch.empty((M, K // 64), dtype=torch.int32, device=dev)
    else:
        s["q"] = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=dev)
        s["scale"] = torch.empty((_blocks(K), M), dtype=torch.float32, device=dev)
    return s


def _run_own(s):
    from w4a8_block_quantized_gb300 import binding as b
    case = s["case"]
    if case["op"] == "linear":
        return {"y": b.fp8_linear(s["a"], s["sa"], s["w"], s["sw"], s["bias"], y=s["y"])}
    if case["op"] == "swiglu":
        K = case["K"]
        q, scale = b.swiglu_quant_fp8(s["gu"][:, :K], s["gu"][:, K:], a_q=s["q"], a_scale=s["scale"])
        return {"codes": q, "scale": scale}
    if case["form"] == "int8":
        q, scale, rowsum, res = b.rmsnorm_quant(s["x"], s["gamma"], EPS, residual=s["res"], residual_out=s["res_out"],
                                                a_q=s["q"], a_scale=s["scale"], rowsum=s["rowsum"])
        return {"codes": q, "scale": scale, "rowsum": rowsum, "residual": res}
    q, scale, res = b.rmsnorm_quant_fp8(s["x"], s["gamma"], EPS, residual=s["res"], residual_out=s["res_out"],
                                        a_q=s["q"], a_scale=s["scale"])
    return {"codes": q, "scale": scale, "residual": res}


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        a = (_grouped(s["a"].float()) * s["sa"].t()[..., None]).flatten(1)[:, :K]
        w = (_grouped(s["w"].float()) * s["sw"].repeat_interleave(BLK, 0)[:N, :, None]).flatten(1)[:, :K]
        return {"y": (torch.matmul(a, w.t()) + s["bias"]).to(_dt(case["dtype"]))}
    if case["op"] == "swiglu":
        g, u = s["gu"][:, : case["K"]].float(), s["gu"][:, case["K"]:].float()
        q, scale = _e4m3_groups(g / (1.0 + torch.exp(-g)) * u)
        return {"codes": q, "scale": scale.t().contiguous()}
    h = s["x"].float() + s["res"].float()
    r = torch.rsqrt((h * h).mean(-1) + EPS)
    t = h * s["gamma"]
    if case["form"] == "fp8":
        q, scale = _e4m3_groups(t)
        return {"codes": q, "scale": (scale * r[:, None]).t().contiguous(), "residual": h.to(s["x"].dtype)}
    sc = t.abs().amax(-1) / t.new_full((), 127.0)
    v = torch.where(sc[:, None] > 0, t / sc[:, None], torch.zeros_like(t))
    low = v.abs().floor()
    q = (torch.sign(v) * (low + (v.abs() - low >= 0.5))).clamp(-127.0, 127.0)
    rowsum = q.view(case["M"], -1, 64).sum(-1).to(torch.int32)
    return {"codes": q.to(torch.int8), "scale": sc * r, "rowsum": rowsum, "residual": h.to(s["x"].dtype)}


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "linear":
        N, nb = case["N"], _blocks(K)
        out = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": M * K + N * K + 4 * nb * (M + _blocks(N)) + 4 * N + out * M * N, "flops": 2 * M * N * K}
    el = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "swiglu":  # gate, up in; codes and scales out
        return {"bytes": M * K * (2 * el + 1) + 4 * M * _blocks(K), "flops": 8 * M * K}
    scales = 4 * M + 4 * M * (K // 64) if case["form"] == "int8" else 4 * M * _blocks(K)
    return {"bytes": M * K * (3 * el + 1) + 4 * K + scales, "flops": 8 * M * K}


def exact(case, seed):
    """The definition in 64 bits.  In the place of e4m3 codes: the values that were rounded to them."""
    i = _inputs(case, seed)
    if case["op"] == "linear":
        a, w = i["a"].double(), i["w"].double()
        y = torch.zeros((case["M"], case["N"]), dtype=torch.float64, device="cuda")
        for b in range(_blocks(case["K"])):
            cut = slice(b * BLK, (b + 1) * BLK)
            rows = i["sw"][:, b].double()[torch.arange(case["N"], device="cuda") // BLK]
            y += (a[:, cut] @ w[:, cut].T) * i["sa"][b].double()[:, None] * rows
        return {"y": y + i["bias"].double()}

    def e4m3(t):
        v, s = torch.empty_like(t), []
        for b in range(_blocks(t.shape[1])):
            cut = slice(b * BLK, (b + 1) * BLK)
            s.append(t[:, cut].abs().max(1).values / 448.0)
            v[:, cut] = t[:, cut] / s[-1][:, None]
        return v, torch.stack(s)

    if case["op"] == "swiglu":
        g, u = i["gu"].double().chunk(2, 1)
        v, s = e4m3(g * torch.sigmoid(g) * u)
        return {"codes": v, "scale": s}
    h = i["x"].double() + i["res"].double()
    rms = (h.square().sum(1) / case["K"] + EPS).sqrt()
    t = h * i["gamma"].double()
    if case["form"] == "fp8":
        v, s = e4m3(t)
        return {"codes": v, "scale": s / rms, "residual": h}
    return {"codes": None, "scale": t.abs().max(1).values / 127.0 / rms, "rowsum": None, "residual": h}
