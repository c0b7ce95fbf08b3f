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
