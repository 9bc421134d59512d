"""A len past what the table can hold: the write and the attention put the new
tokens at the same places; those past the table are not there, and the rows see
what is."""

import numpy as np
import pytest
import torch

from block_testlib import ROUND, TINY, TYPES, blank, close, f64
from cache_testlib import Cache, attend64, held
from test_gpu_attention import FOLDED, KINDS, ROUND_P

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("window", [0, 9, 40])
@pytest.mark.parametrize("new,over", [(20, 6), (1, 1), (3, 3), (4, 30), (150, 70), (150, 150)])
def test_places_past_the_table(q4lib, name, cache, window, new, over):
    heads, kv_heads, d, page = 4, 2, 64, 16
    room = 192                                              # tokens that the table holds
    length, old = room + over, max(0, room + over - new)
    g = torch.Generator(device="cuda").manual_seed(new + over)
    k = torch.randn(length, kv_heads, d, generator=g, device="cuda").to(TYPES[name])
    v = torch.randn(length, kv_heads, d, generator=g, device="cuda").to(TYPES[name])
    q = torch.randn(new, heads * d, generator=g, device="cuda").to(TYPES[name])
    flat_k, flat_v = k.reshape(length, -1), v.reshape(length, -1)
    c = Cache(q4lib, [room], kv_heads, d, page, cache)
    assert c.table.shape[1] * page == room
    before = min(old, room)
    c.write(flat_k[:before], flat_v[:before], name, [before], [before])
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
    c.write(flat_k[old:], flat_v[old:], name, [length], [new])
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == q4lib.Q4_ERR_DEVICE_CHECK
    o = blank(new, heads * d, name)
    c.attend(o, q, name, heads, 0.125, window, [length], [new])
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
    hk, hv = held(k, cache), held(v, cache)
    for i in range(new):
        pos = old + i
        lo, hi = max(0, pos + 1 - window) if window else 0, min(pos + 1, room)
        if lo >= hi:
            assert not bool(o[i].any())
            continue
        ref, tol = attend64(q[i:i + 1], hk[lo:hi], hv[lo:hi], heads, kv_heads, d, 0.125, 0, [hi - lo], [1], ROUND_P[name, cache],
                            2 if name == "f32" else 1, (name, cache) == FOLDED)
        close(o[i:i + 1], f64(ref), f64(tol) + ROUND[name] * np.abs(f64(ref)) * 1.01 + TINY[name], f"row {i}")


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("new", [2, 100])
def test_the_largest_len(q4lib, name, cache, new):
    """2^31 - 1 tokens by the batch's word: every row sees all that the table holds."""
    heads, kv_heads, d, room = 2, 1, 64, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn(room, kv_heads * d, generator=g, device="cuda").to(TYPES[name])
    q = torch.randn(new, heads * d, generator=g, device="cuda").to(TYPES[name])
    c = Cache(q4lib, [room], kv_heads, d, 16, cache)
    c.write(k, k, name, [room], [room])
    o, last = blank(new, heads * d, name), blank(new, heads * d, name)
    c.attend(o, q, name, heads, 0.125, 0, [(1 << 31) - 1], [new])
    kk = held(k.reshape(room, 1, d), cache)
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
    for i in range(0, new, 7):
        ref, tol = attend64(q[i:i + 1], kk, kk, heads, kv_heads, d, 0.125, 0, [room], [1], ROUND_P[name, cache], 2 if name == "f32" else 1,
                            (name, cache) == FOLDED)
        close(o[i:i + 1], f64(ref), f64(tol) + ROUND[name] * np.abs(f64(ref)) * 1.01 + TINY[name], f"row {i}")
    # and a window ends before any token that is there
    c.attend(last, q, name, heads, 0.125, 1 << 29, [(1 << 31) - 1], [new])
    torch.cuda.synchronize()
    assert not bool(last.any())
