"""The e4m3 linear's forms called by name (tests/fp8_forms.cu), built on first use."""
import ctypes
import functools
import os
import subprocess

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "fp8_forms.cu")
LIB = os.path.join(HERE, "_build", "libfp8_forms.so")
TILES, SPLITS = (16, 32, 64, 128), (1, 2, 4, 8)
FORMS = [(0, 1)] + [(t, s) for t in TILES for s in SPLITS]  # 0: pairs of CTAs


@functools.lru_cache(None)
def lib():
    from w4a8_block_quantized_gb300 import build
    if not os.path.exists(LIB) or any(os.path.getmtime(f) > os.path.getmtime(LIB) for f in [SRC, *build._deps()]):
        os.makedirs(os.path.dirname(LIB), exist_ok=True)
        tmp = f"{LIB}.{os.getpid()}"
        r = subprocess.run([build.nvcc(), *build.ARCH, "-O3", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
                            "-Xptxas", "-v", "-I", os.path.join(build.ROOT, "include"), "-shared", "-o", tmp, SRC],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        build.check_register_split(r.stdout + r.stderr)
        os.replace(tmp, LIB)
    so = ctypes.CDLL(LIB)
    P, I, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    so.forms_run.argtypes = [I, I, P, P, P, P, P, P, I, L, L, L, P, L, L, I, P]
    so.forms_clusters.argtypes = [I, I]
    so.forms_pick.argtypes = [L, L, L, I, P, ctypes.POINTER(I), ctypes.POINTER(I)]
    so.forms_pick.restype = None
    return so


def pick(M, N, K, num_sms, fit):
    """The (tile, split) of a problem; fit(tile, split): the clusters that run at once."""
    table = (ctypes.c_int * 16)(*(fit(t, s) for t in TILES for s in SPLITS))
    tn, split = ctypes.c_int(), ctypes.c_int()
    lib().forms_pick(M, N, K, num_sms, table, ctypes.byref(tn), ctypes.byref(split))
    return tn.value, split.value


def fits(tn, split, M, N, K, num_sms):
    """Whether a split form takes the problem: at least a block of 128 for most CTAs, and every tile's cluster
    resident at once."""
    tiles = -(-M // tn) * -(-N // 128) if tn else 0
    return split == 1 or (split <= -(-K // 128) and tiles * split <= num_sms and tiles <= lib().forms_clusters(tn, split))


def run(form, a, sa, w, sw, bias=None, y=None, out_dtype=torch.float32, limit_us=1_000_000, copy_blocks=-1, num_sms=None,
        status=None):
    """(y, status word) of one launch, on the current stream."""
    (M, K), N = a.shape, w.shape[0]
    num_sms = torch.cuda.get_device_properties(0).multi_processor_count if num_sms is None else num_sms
    y = torch.empty((M, N), dtype=out_dtype, device="cuda") if y is None else y
    status = torch.zeros(1, dtype=torch.int32, device="cuda") if status is None else status
    rc = lib().forms_run(*form, a.data_ptr(), sa.data_ptr(), w.data_ptr(), sw.data_ptr(),
                         None if bias is None else bias.data_ptr(), y.data_ptr(), int(y.dtype == torch.bfloat16), M, N, K,
                         status.data_ptr(), limit_us, copy_blocks, num_sms, torch.cuda.current_stream().cuda_stream)
    assert rc == 0, f"form {form}: launch returned {rc}"
    return y, status
