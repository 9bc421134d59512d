"""Queries that are not finite, or next to nothing, in blocks whose rows see nothing
or not all of a tile."""

import numpy as np
import pytest
import torch

from block_testlib import ROUND, TINY, TYPES, blank, close, f64
from cache_testlib import Cache, attend64, held
from test_gpu_attention import FOLDED, KINDS, ROUND_P

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("new", [8, 200])
def test_rows_that_see_nothing_whatever_their_queries(q4lib, name, cache, new):
    """Zeros for a row that sees nothing, if its query is not finite, too; NaN for
    such a row that sees something; the others as ever."""
    heads, kv_heads, d, length = 4, 2, 64, new // 2
    g = torch.Generator(device="cuda").manual_seed(2)
    k = torch.randn(length, kv_heads * d, generator=g, device="cuda").to(TYPES[name])
    c = Cache(q4lib, [length], kv_heads, d, 16, cache)
    c.write(k, k, name, [length], [length])
    q = torch.randn(new, heads * d, generator=g, device="cuda").to(TYPES[name])
    good, bad = blank(new, heads * d, name), blank(new, heads * d, name)
    c.attend(good, q, name, heads, 0.125, 0, [length], [new])
    assert not bool(good[:new - length].any())
    q[0, 3], q[1, d + 5], q[2, 2 * d] = float("nan"), float("inf"), -float("inf")
    q[new - 2, 1] = float("nan")
    c.attend(bad, q, name, heads, 0.125, 0, [length], [new])
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
    hit = torch.zeros_like(bad, dtype=torch.bool)
    hit[new - 2, :d] = True
    assert torch.equal(torch.isnan(bad), hit) and torch.equal(bad[~hit], good[~hit])


@pytest.mark.parametrize("name,cache", [("bf16", "i8"), ("f32", "i8"), ("f16", "i8")])
@pytest.mark.parametrize("new", [3, 150])
def test_queries_next_to_nothing(q4lib, name, cache, new):
    """Scores that vanish whatever the keys: the mean of the values seen."""
    heads, kv_heads, d, length = 2, 1, 64, new + 20
    g = torch.Generator(device="cuda").manual_seed(6)
    k = torch.randn(length, kv_heads, d, generator=g, device="cuda").to(TYPES[name])
    q = (torch.randn(new, heads * d, generator=g, device="cuda") * 2.0 ** -112).to(TYPES[name])
    c = Cache(q4lib, [length], kv_heads, d, 16, cache)
    c.write(k.reshape(length, -1), k.reshape(length, -1), name, [length], [length])
    o = blank(new, heads * d, name)
    kk = held(k, cache)
    for scale in (1.0, 1e-7, 1e-30):
        c.attend(o, q, name, heads, scale, 0, [length], [new])
        ref, tol = attend64(q, kk, kk, heads, kv_heads, d, scale, 0, [length], [new], ROUND_P[name, cache], 2 if name == "f32" else 1,
                            (name, cache) == FOLDED)
        close(o, f64(ref), f64(tol) + ROUND[name] * np.abs(f64(ref)) * 1.01 + TINY[name], f"scale {scale}")
