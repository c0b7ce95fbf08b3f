"""Workspace sizes of attention: one default bound on the keys, and a size that suffices for every smaller call."""
import ctypes
import random
import types

import pytest


def b():
    from w4a8_block_quantized_gb300 import binding
    return binding


@pytest.fixture(scope="module")
def lib():
    from w4a8_block_quantized_gb300 import build
    build.build()
    return b().load()


def cache(heads, D, page=16, pages=64):
    c = b()._KvCache(pages=pages, heads=heads, page=page, head_dim=D, format=0)
    return types.SimpleNamespace(c=c, ref=ctypes.addressof(c), pages=pages, page=page)


def size(lib, c, what="bytes", **kw):
    a = b()._AttentionArgs(**kw)
    return getattr(lib, "w4a8_attention_workspace_" + what)(c.ref, ctypes.addressof(a))


def test_a_bound_for_every_smaller_call(lib):
    rng = random.Random(3)
    log = lambda hi: int(2 ** rng.uniform(0, hi.bit_length() - 1))  # noqa: E731
    met = 0
    for _ in range(400):
        heads, D = rng.choice([1, 2, 4, 8, 32]), rng.choice([64, 128])
        c = cache(heads, D)
        same = dict(q_heads=heads * rng.choice([1, 2, 3, 4, 8, 12, 40]), window=rng.choice([0, 0, log(8192)]), sinks=rng.choice([0, 4, 130]))
        top = dict(batch=log(256), total=log(1 << 14), max_q=log(8192), max_kv=log(1 << 18))
        bound = size(lib, c, "bound", **same, **top)
        assert bound < 9 << 30
        for i in range(40):
            low = top if i == 0 else {k: rng.randint(max(1, v // rng.choice([1, 2, 50])), v) for k, v in top.items()}
            need = size(lib, c, **same, **low)
            assert need <= bound, (same, top, low)
            met += need > size(lib, c, **same, **top)
    assert met > 100  # smaller calls do need more at times
    c = cache(8, 128)
    assert size(lib, c, "bound", q_heads=6, batch=1, total=1, max_q=1, max_kv=5) == (1 << 64) - 1
    assert size(lib, c, "bound", q_heads=8, batch=0, total=1, max_q=1, max_kv=5) == 0


@pytest.mark.parametrize("batch,max_q,pages,width", [(16, 512, 1 << 16, 256), (1, 1, 32, 2048), (64, 8, 4096, 64)])
def test_the_call_and_the_size_query_take_one_default(lib, batch, max_q, pages, width):
    """Without max_kv both go by the page table's width, whatever the cache holds in all."""
    c = cache(8, 128, pages=pages)
    q, table = types.SimpleNamespace(shape=(batch * max_q, 32, 128)), types.SimpleNamespace(shape=(batch, width))
    got = b().attention_workspace_bytes(q, c, batch, max_q=max_q, page_table=table)
    want = size(lib, c, q_heads=32, batch=batch, total=batch * max_q, max_q=max_q, max_kv=width * 16)
    assert got == want  # (0 for the third: clusters join their own sums)
    assert b().attention_workspace_bound(c, 32, batch, batch * max_q, max_q, max_kv=width * 16) >= got
    with pytest.raises(ValueError, match="max_kv or the call's page_table"):
        b().attention_workspace_bytes(q, c, batch, max_q=max_q)
