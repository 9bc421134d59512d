"""What a page holds that was never written, or that the cache does not have,
stays with the rows that see it: other sequences of the call, and rows of the same
sequence that do not see it, get what they get without it."""

import numpy as np
import pytest
import torch

from block_testlib import ROUND, TINY, TYPES, blank, close, f64
from cache_testlib import Cache, attend64, held
from test_gpu_attention import FOLDED, KINDS, ROUND_P

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 70])
def test_sequences_over_pages_never_written(q4lib, name, cache, d, new):
    """Every other sequence reads pages of NaN, more tiles of them than a ring
    holds; the short ones between them end inside a tile."""
    heads, kv_heads, pairs, page = 4, 2, 200, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    short = new + 4
    lens, counts = [1280 + new, short] * pairs, [new, new] * pairs
    c = Cache(q4lib, [short] * pairs, kv_heads, d, page, cache, seed=2)
    k = torch.randn(pairs * short, kv_heads * d, generator=g, device="cuda").to(TYPES[name])
    c.write(k, k, name, [short] * pairs, [short] * pairs)
    q = torch.randn(2 * pairs * new, heads * d, generator=g, device="cuda").to(TYPES[name])
    fresh = (set(range(c.n_pages)) - set(int(x) for x in c.table.flatten() if x >= 0)).pop()
    per = -(-lens[0] // page)
    table = torch.full((2 * pairs, per), fresh, dtype=torch.int32, device="cuda")
    table[1::2, :c.table.shape[1]] = c.table
    c.table = table
    o = blank(2 * pairs * new, heads * d, name)
    c.attend(o, q, name, heads, 0.125, 0, lens, counts)
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
    got, mine = (x.reshape(2 * pairs, new, heads * d)[1::2].reshape(pairs * new, heads * d) for x in (o, q))
    kk = held(k.reshape(pairs * short, kv_heads, d), cache)
    ref, tol = attend64(mine, kk, kk, heads, kv_heads, d, 0.125, 0, [short] * pairs, [new] * pairs, ROUND_P[name, cache],
                        2 if name == "f32" else 1, (name, cache) == FOLDED)
    close(got, f64(ref), f64(tol) + ROUND[name] * np.abs(f64(ref)) * 1.01 + TINY[name], f"{name} {cache}")


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("new", [60, 250])
def test_rows_before_a_page_that_is_not_there(q4lib, name, cache, page, new):
    """An entry that the cache does not have: recorded; the rows before its tokens,
    and the sequence next to it, are untouched by it."""
    heads, kv_heads, d, length = 4, 2, 64, new + 300
    g = torch.Generator(device="cuda").manual_seed(5)
    lens, counts = [length, 40], [new, 9]
    total = sum(lens)
    k = torch.randn(total, kv_heads * d, generator=g, device="cuda").to(TYPES[name])
    q = torch.randn(sum(counts), heads * d, generator=g, device="cuda").to(TYPES[name])
    c = Cache(q4lib, lens, kv_heads, d, page, cache, seed=2)
    c.table += (c.table >= 0).to(torch.int32) * 2           # pages 0 and n_pages - 1 are never written
    c.n_pages += 4
    c.pages = torch.full((c.n_pages * c.nbytes,), 255, dtype=torch.uint8, device="cuda")
    c.write(k, k, name, lens, lens)
    good = blank(sum(counts), heads * d, name)
    c.attend(good, q, name, heads, 0.125, 0, lens, counts)
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
    entry = (length - new // 2) // page                     # in the middle of the new tokens
    for bad in (-1, c.n_pages, 1 << 30):
        c.table[0, entry] = bad
        o = blank(sum(counts), heads * d, name)
        c.attend(o, q, name, heads, 0.125, 0, lens, counts)
        torch.cuda.synchronize()
        assert q4lib.q4_last_device_status(clear=True) == q4lib.Q4_ERR_DEVICE_CHECK
        clean = max(0, entry * page - (length - new))       # rows before the page's first token
        assert clean > 0 or page == 128
        assert torch.equal(o[:clean], good[:clean]) and torch.equal(o[new:], good[new:])
