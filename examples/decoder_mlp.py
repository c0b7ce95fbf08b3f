"""A decoder layer's MLP from the library's operators, in both weight formats:

    h = x + residual;  a = rms_norm(h) * gamma;  y = W_down (silu(W_gate a) * (W_up a))

  4 bits   rmsnorm_prepare -> linear_prepared_ex (gate and up rows in one matrix, bf16 out)
           -> swiglu_prepare -> linear_prepared_ex; one token takes the streaming kernel:
           rmsnorm_quant -> linear_ex -> swiglu_quant -> linear_ex
  8 bits   rmsnorm_quant_fp8 -> fp8_linear -> swiglu_quant_fp8 -> fp8_linear

Each form is four launches, with no activation written in more than 16 bits.  Run it:
python examples/decoder_mlp.py [tokens hidden inner].  It prints, for each form, the error against the
same MLP in fp32 on the dequantized weights, and the time of a replay of the calls captured into a graph.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from w4a8_block_quantized_gb300 import binding as b  # noqa: E402

EPS = 1e-6


def weights_4bit(rows, cols, gen):
    """Random u4 codes with fp16 scales and zeros for blocks of 64; the values they stand for."""
    q = torch.randint(0, 16, (rows, cols), generator=gen, device="cuda", dtype=torch.uint8)
    scale = (torch.rand((rows, cols // 64), generator=gen, device="cuda") * 0.004 + 0.002).half()
    zero = (torch.rand((rows, cols // 64), generator=gen, device="cuda") * 3 + 6).half()
    packed = q[:, 0::2] | (q[:, 1::2] << 4)
    w = (q.view(rows, -1, 64).float() - zero.float()[..., None]) * scale.float()[..., None]
    return (packed.contiguous(), scale, zero), w.view(rows, cols)


def weights_8bit(rows, cols, gen):
    """Random weights in e4m3 with a scale for each 128 x 128 block; the values they stand for."""
    w = torch.randn((rows, cols), generator=gen, device="cuda") * 0.02
    nr, nc = -(-rows // 128), -(-cols // 128)
    full = torch.nn.functional.pad(w, (0, nc * 128 - cols, 0, nr * 128 - rows)).view(nr, 128, nc, 128)
    scale = full.abs().amax((1, 3)) / 448
    q = (full / scale[:, None, :, None]).view(nr * 128, nc * 128)[:rows, :cols].contiguous().to(torch.float8_e4m3fn)
    each = scale.repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return (q, scale), q.float() * each


class Mlp4:
    """W4A8: weights prepared once for the tensor cores, and kept packed for the few-token kernel."""

    def __init__(self, hidden, inner, gamma, gen):
        self.hidden, self.inner, self.gamma = hidden, inner, gamma
        self.gate_up, self.w_gate_up = weights_4bit(2 * inner, hidden, gen)
        self.down, self.w_down = weights_4bit(hidden, inner, gen)
        self.p_gate_up, self.p_down = b.prepare_weights(*self.gate_up), b.prepare_weights(*self.down)

    def __call__(self, x, residual, stream=None):
        M, bf = x.shape[0], torch.bfloat16
        if M <= 8:
            q, s, rs, h = b.rmsnorm_quant(x, self.gamma, EPS, residual=residual, stream=stream)
            gu = b.linear_ex(q, s, rs, *self.gate_up, out_dtype=bf, stream=stream)
            q, s, rs = b.swiglu_quant(gu[:, :self.inner], gu[:, self.inner:], stream=stream)
            return b.linear_ex(q, s, rs, *self.down, out_dtype=bf, stream=stream), h
        act, h = b.rmsnorm_prepare(x, self.gamma, EPS, residual=residual, stream=stream)
        gu = b.linear_prepared_ex(act, self.p_gate_up, M, 2 * self.inner, self.hidden, out_dtype=bf, stream=stream)
        act = b.swiglu_prepare(gu[:, :self.inner], gu[:, self.inner:], stream=stream)
        return b.linear_prepared_ex(act, self.p_down, M, self.hidden, self.inner, out_dtype=bf, stream=stream), h


class Mlp8:
    """e4m3 weights and activations, a scale for each block of 128."""

    def __init__(self, hidden, inner, gamma, gen):
        self.hidden, self.inner, self.gamma = hidden, inner, gamma
        self.gate_up, self.w_gate_up = weights_8bit(2 * inner, hidden, gen)
        self.down, self.w_down = weights_8bit(hidden, inner, gen)

    def __call__(self, x, residual, stream=None):
        bf = torch.bfloat16
        a, s, h = b.rmsnorm_quant_fp8(x, self.gamma, EPS, residual=residual, stream=stream)
        gu = b.fp8_linear(a, s, *self.gate_up, out_dtype=bf, stream=stream)
        a, s = b.swiglu_quant_fp8(gu[:, :self.inner], gu[:, self.inner:], stream=stream)
        return b.fp8_linear(a, s, *self.down, out_dtype=bf, stream=stream), h


def plain(mlp, x, residual):
    """The same MLP in fp32 on the dequantized weights, activations not quantized."""
    h = x.float() + residual.float()
    a = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * mlp.gamma
    gu = a @ mlp.w_gate_up.t()
    t = torch.nn.functional.silu(gu[:, :mlp.inner]) * gu[:, mlp.inner:]
    return t @ mlp.w_down.t(), h


def run(tokens, hidden, inner, seed=0, replays=20):
    """For each form: (name, relative error of the output, whether the residual is exact, whether a
    captured run gives the same bits, us a replay)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    gamma = 1 + 0.1 * torch.randn(hidden, generator=gen, device="cuda")
    x = torch.randn((tokens, hidden), generator=gen, device="cuda").bfloat16()
    residual = torch.randn((tokens, hidden), generator=gen, device="cuda").bfloat16()
    found = []
    for name, make in (("4 bits", Mlp4), ("8 bits", Mlp8)):
        mlp = make(hidden, inner, gamma, gen)
        y, h = mlp(x, residual)
        want, want_h = plain(mlp, x, residual)
        err = float((y.float() - want).norm() / want.norm())
        # the same calls captured once and replayed
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            pool = [mlp(x, residual, stream)]  # sizes the stream's part of the allocator
            stream.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                pool.append(mlp(x, residual, stream))
            graph.replay()
            a, z = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record(stream)
            for _ in range(replays):
                graph.replay()
            z.record(stream)
        stream.synchronize()
        same = torch.equal(pool[1][0], y) and torch.equal(pool[1][1], h)
        assert b.sync_status() == 0
        found.append((name, err, torch.equal(h, want_h.bfloat16()), same, a.elapsed_time(z) / replays * 1e3))
    return found


if __name__ == "__main__":
    sizes = [int(v) for v in sys.argv[1:4]] or [512, 2048, 6144]
    for tokens in (sizes[0], 1):
        for name, err, exact, same, us in run(tokens, *sizes[1:]):
            print(f"{name}, {tokens} tokens, {sizes[1]} -> 2 x {sizes[2]} -> {sizes[1]}: relative error {err:.4f} "
                  f"against fp32, residual {'exact' if exact else 'DIFFERS'}, replay "
                  f"{'equal' if same else 'DIFFERS'}, {us:.1f} us")
