"""Attention past 32-bit offsets: pages far into a cache, and more elements in a
row of queries than 32 bits count."""

import numpy as np
import pytest
import torch

from block_testlib import ROUND, TINY, TYPES, blank, close, f64
from cache_testlib import Cache, attend64, held
from test_gpu_attention import FOLDED, KINDS, ROUND_P

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("new", [2, 100])
def test_pages_past_32_bits(q4lib, name, cache, new):
    heads, kv_heads, d, page, length = 4, 2, 128, 64, 300
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn(length, kv_heads, d, generator=g, device="cuda").to(TYPES[name])
    q = torch.randn(new, heads * d, generator=g, device="cuda").to(TYPES[name])
    c = Cache(q4lib, [length], kv_heads, d, page, cache, spare=0)
    used = c.n_pages
    c.n_pages = (1 << 32) // c.nbytes + 2 * used
    c.pages = torch.empty(c.n_pages * c.nbytes, dtype=torch.uint8, device="cuda")
    c.table += c.n_pages - used
    c.table[0, 0] = 1                                       # and one near the front
    assert (c.n_pages - used) * c.nbytes > 1 << 32
    c.write(k.reshape(length, -1), k.reshape(length, -1), name, [length], [length])
    o = blank(new, heads * d, name)
    c.attend(o, q, name, heads, 0.1, 0, [length], [new])
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
    kk = held(k, cache)
    ref, tol = attend64(q, kk, kk, heads, kv_heads, d, 0.1, 0, [length], [new], ROUND_P[name, cache], 2 if name == "f32" else 1,
                        (name, cache) == FOLDED)
    close(o, f64(ref), f64(tol) + ROUND[name] * np.abs(f64(ref)) * 1.01 + TINY[name])


@pytest.mark.parametrize("name,cache", [("f16", "f16"), ("bf16", "i8"), ("f32", "f16")])
def test_heads_past_32_bits(q4lib, name, cache):
    """One token of 2^31 + 2048 elements: its last heads, and its first, are those of a
    token that has no others."""
    d, few = 256 if name == "f32" else 128, 64
    heads = (1 << 31) // d + 16
    free, _ = torch.cuda.mem_get_info()
    if free < 3 * heads * d * TYPES[name].itemsize:
        pytest.skip("not enough device memory")
    g = torch.Generator(device="cuda").manual_seed(2)
    k = torch.randn(40, d, generator=g, device="cuda").to(TYPES[name])
    c = Cache(q4lib, [40], 1, d, 16, cache)
    c.write(k, k, name, [40], [40])
    ends = torch.randn(2, few * d, generator=g, device="cuda").to(TYPES[name])
    q = torch.zeros(1, heads * d, dtype=TYPES[name], device="cuda")
    q[0, :few * d], q[0, -few * d:] = ends[0], ends[1]
    c.attend(q, q, name, heads, 0.1, 0, [40], [1])
    small = [blank(1, few * d, name) for _ in range(2)]
    for o, e in zip(small, ends):
        c.attend(o, e.reshape(1, -1), name, few, 0.1, 0, [40], [1])
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
    got = (q[:, :few * d], q[:, -few * d:])
    kk = held(k.reshape(40, 1, d), cache)
    for o, e, y in zip(small, ends, got):
        ref, tol = attend64(e.reshape(1, -1), kk, kk, few, 1, d, 0.1, 0, [40], [1], ROUND_P[name, cache], 2 if name == "f32" else 1,
                            (name, cache) == FOLDED)
        for x in (o, y):
            close(x, f64(ref), f64(tol) + ROUND[name] * np.abs(f64(ref)) * 1.01 + TINY[name])
