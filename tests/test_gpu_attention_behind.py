"""Attention with a window over sequences whose beginning is gone: table entries
behind the window are not looked at, pages and places behind it were never
written, and the results are those of the whole sequence, to the bit."""

import numpy as np
import pytest
import torch

from block_testlib import ROUND, TINY, TYPES, blank, close, f64
from cache_testlib import Cache, attend64, held
from test_gpu_attention import FOLDED, KINDS, ROUND_P

pytestmark = pytest.mark.gpu

# What a page that was never written holds: NaN in every type, or -infinity in the
# scales of codes and in bf16 values.
FILLS = {"nan": 0xFFFFFFFF, "-inf": 0xFF800000}


def behind(q4, name, cache, heads, kv_heads, d, page, lens, counts, window, entry, fill):
    """Two caches with the same places: one written from the start, one from the
    first visible token of each sequence on, with `entry` ("none": -1, "fresh": a page
    that was never written) behind it."""
    g = torch.Generator(device="cuda").manual_seed(page + window)
    total = sum(lens)
    k = torch.randn(total, kv_heads, d, generator=g, device="cuda").to(TYPES[name])
    v = torch.randn(total, kv_heads, d, generator=g, device="cuda").to(TYPES[name])
    q = torch.randn(sum(counts), heads * d, generator=g, device="cuda").to(TYPES[name])
    whole, cut = (Cache(q4, lens, kv_heads, d, page, cache, seed=1) for _ in range(2))
    cut.pages.view(torch.int32).fill_(int(np.uint32(FILLS[fill]).astype(np.int32)))
    flat_k, flat_v = k.reshape(total, -1), v.reshape(total, -1)
    whole.write(flat_k, flat_v, name, lens, lens)
    first = [max(0, n - m + 1 - window) for n, m in zip(lens, counts)]
    left = [n - f for n, f in zip(lens, first)]
    at = [sum(lens[:i]) for i in range(len(lens))]
    rows_ = torch.cat([torch.arange(at[i] + first[i], at[i] + lens[i], device="cuda") for i in range(len(lens))])
    spare = (set(range(cut.n_pages)) - set(int(x) for x in cut.table.flatten() if x >= 0)).pop()
    for i, f in enumerate(first):
        cut.table[i, :f // page] = -1 if entry == "none" else spare
    cut.write(flat_k[rows_], flat_v[rows_], name, lens, left)
    torch.cuda.synchronize()
    assert q4.q4_last_device_status(clear=True) == 0
    outs = []
    for c in (whole, cut):
        o = blank(sum(counts), heads * d, name)
        c.attend(o, q, name, heads, d ** -0.5, window, lens, counts)
        torch.cuda.synchronize()
        assert q4.q4_last_device_status(clear=True) == 0
        outs.append(o)
    ref, tol = attend64(q, held(k, cache), held(v, cache), heads, kv_heads, d, d ** -0.5, window, lens, counts, ROUND_P[name, cache],
                        2 if name == "f32" else 1, (name, cache) == FOLDED)
    close(outs[1], f64(ref), f64(tol) + ROUND[name] * np.abs(f64(ref)) * 1.01 + TINY[name], f"{name} {cache}")
    assert torch.equal(*outs)


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("entry,fill", [("none", "nan"), ("fresh", "nan"), ("none", "-inf"), ("fresh", "-inf")])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("window", [1, 15, 100])
@pytest.mark.parametrize("new", [1, 20, 140])
def test_nothing_behind_the_window(q4lib, name, cache, entry, fill, page, window, new):
    """Windows that start inside a tile and inside a page: one new token, blocks of
    some, and of many query rows."""
    lens = [100 + new, 1000 + new, 271 + new, new]
    behind(q4lib, name, cache, 4, 2, 64, page, lens, [new] * 4, window, entry, fill)


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("d", [40, 128, 200])
@pytest.mark.parametrize("new", [2, 300])
def test_head_sizes(q4lib, name, cache, d, new):
    behind(q4lib, name, cache, 4, 1, d, 16, [700 + new, 90 + new], [new, new], 77, "fresh", "nan")


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("step", range(0, 128, 9))
def test_every_place_in_a_tile(q4lib, name, cache, step):
    for new in (1, 90):
        behind(q4lib, name, cache, 2, 1, 64, 16, [200 + step + new], [new], 33, "none", "nan")
