"""The operators around the linears, restated for the tests: fp64 definitions, and the parts that
are defined as single IEEE fp32 steps (codes of rmsnorm and quant) in numpy fp32."""
import numpy as np
import torch

U = 2.0 ** -24  # half an ulp of fp32, relative


def e4m3(v):
    """Nearest e4m3 value (ties to even, saturating at 448) of an fp64 or fp32 array, as fp64."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    e = np.clip(np.floor(np.log2(np.maximum(a, 2.0 ** -20))), -6, 8)
    step = 2.0 ** (e - 3)
    r = np.minimum(np.round(a / step) * step, 448.0)  # np.round is half-to-even; step is a power of two
    return np.where(np.isnan(v), np.nan, np.copysign(r, v))


def half_away(v):
    low = np.floor(np.abs(v))
    return np.copysign(low + (np.abs(v) - low >= 0.5), v)


def int8_rows(t):
    """t fp32 [M][K] -> codes, row scale (fp32, before the common factor), block-64 sums."""
    s = (np.abs(t).max(1) / np.float32(127)).astype(np.float32)
    q = np.zeros_like(t)
    live = s > 0
    q[live] = half_away((t[live] / s[live, None]).astype(np.float32))
    q = np.clip(q, -127, 127).astype(np.int8)
    return q, s, q.reshape(t.shape[0], -1, 64).astype(np.int32).sum(2)


def e4m3_rows(t):
    """t fp32 [M][K] -> code values (fp64), group scales fp32 [ceil(K/128)][M]."""
    M, K = t.shape
    nb = (K + 127) // 128
    q = np.zeros((M, K))
    s = np.zeros((nb, M), np.float32)
    for b in range(nb):
        g = t[:, b * 128:(b + 1) * 128]
        m = np.abs(g).max(1).astype(np.float32)
        live = m >= np.float32(2.0 ** -100)
        inv = np.zeros_like(m)
        inv[live] = np.float32(448) / m[live]
        q[:, b * 128:(b + 1) * 128] = e4m3((g * inv[:, None]).astype(np.float32))
        s[b, live] = m[live] / np.float32(448)
    return q, s


def norm_sum(x, residual):
    return x if residual is None else (x + residual).astype(np.float32)


def norm_factor(h, eps):
    """1 / sqrt(mean h^2 + eps) in fp64, and the relative error allowed to an fp32 evaluation: a
    sum of squares of at most `adds` rounded additions (32 values a thread, or 8 in 8192 of a
    longer row, then 5 + 32 partial sums), halved by the root, and four more roundings."""
    K = h.shape[1]
    r = 1.0 / np.sqrt((h.astype(np.float64) ** 2).sum(1) / K + float(np.float32(eps)))
    adds = max(32, 8 * -(-K // 8192)) + 5 + 32
    return r, (adds / 2 + 4) * U


def swiglu(g, u):
    """fp64 silu(g) * u and the relative error allowed to the fp32 evaluation: the documented bounds
    of __expf (2 + 1.173 |g| ulp), an addition, __fdividef (2 ulp) and a product."""
    g, u = g.astype(np.float64), u.astype(np.float64)
    t = g / (1.0 + np.exp(-g)) * u
    return t, (2 + 1.173 * np.abs(g) + 2 + 2) * 2 * U


def fp8_linear(a, sa, w, sw, bias):
    """fp64 result [M][N] and the sum of the magnitudes of its terms (without the bias), on the
    tensors' device."""
    M, K = a.shape
    N = w.shape[0]
    y = torch.zeros((M, N), dtype=torch.float64, device=a.device)
    mag = torch.zeros_like(y)
    for b in range((K + 127) // 128):
        cut = slice(128 * b, 128 * b + 128)
        A, W = a[:, cut].double(), w[:, cut].double()
        f = sa[b].double()[:, None] * sw[:, b].double().repeat_interleave(128)[:N][None, :]
        y += f * (A @ W.T)
        mag += f.abs() * (A.abs() @ W.abs().T)
    return (y if bias is None else y + bias.double()), mag


def fp8_linear_allowed(ref, mag, K, bf16):
    """Error allowed to a kernel that sums a block's 128 products on the tensor cores (4 steps of
    32 products, each aligned to its largest and cut at no fewer than 24 bits: at most 4 * 33 units
    of 2^-23 of the largest partial sum, bounded by 2^-16 of the magnitudes) and the blocks in fp32
    (one product, one fma a block, the halves of a split and the bias), plus the output's rounding."""
    nb = (K + 127) // 128
    tol = mag * (2.0 ** -16 + (nb + 12) * U) + ref.abs() * 2 * U + 1e-30
    return tol + ref.abs() * 2.0 ** -8 if bf16 else tol
