"""Attention of new tokens over the paged cache against the formula in 64 bits:
types, head layouts, lengths around tiles and pages, windows, rows that see
nothing, what stands in masked places, and many shares of one sequence."""

import math

import numpy as np
import pytest
import torch

from block_testlib import ROUND, TINY, TYPES, blank, close, f64, gaps_kept, rows
from cache_testlib import Cache, attend64, held, ints, starts_of

pytestmark = pytest.mark.gpu

KINDS = [("f16", "f16"), ("f32", "f16"), ("bf16", "bf16"), ("bf16", "i8"), ("f16", "i8"), ("f32", "i8")]
# The terms' rounding: the operands' type, or two fp16 numbers.
ROUND_P = {("f16", "f16"): 2.0 ** -11, ("f32", "f16"): 2.0 ** -21, ("bf16", "bf16"): 2.0 ** -8, ("bf16", "i8"): 2.0 ** -11,
           ("f16", "i8"): 2.0 ** -11, ("f32", "i8"): 2.0 ** -21}
FOLDED = ("bf16", "i8")   # operands may carry their scales, rounded to fp16


def run(q4, name, cache, heads, kv_heads, d, page, lens, counts, window=0, pad=0, shift=0, max_new=None, more_rows=0, sharp=1.0,
        seed=3, scale=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    total, scale = sum(max(n, 0) for n in lens), scale or d ** -0.5
    k = torch.randn(total, kv_heads, d, generator=g, device="cuda").to(TYPES[name])
    v = (torch.randn(total, kv_heads, d, generator=g, device="cuda") * (0.1 + 3 * torch.rand(total, kv_heads, 1, generator=g, device="cuda"))).to(TYPES[name])
    c = Cache(q4, lens, kv_heads, d, page, cache, seed)
    c.write(k.reshape(total, -1), v.reshape(total, -1), name, lens, lens)
    n = sum(counts)
    q = torch.randn(n + more_rows, heads * d, generator=g, device="cuda") * sharp
    q = rows(q, name, pad, shift)
    o = blank(n + more_rows, heads * d, name, pad, shift)
    if more_rows:
        o[n:] = 5.0
    c.attend(o, q, name, heads, scale, window, lens, counts, max_new)
    torch.cuda.synchronize()
    assert q4.q4_last_device_status(clear=True) == 0
    ref, tol = attend64(q[:n], held(k, cache), held(v, cache), heads, kv_heads, d, scale, window, lens, counts, ROUND_P[name, cache],
                        2 if name == "f32" else 1, (name, cache) == FOLDED)
    close(o[:n], f64(ref), f64(tol) + ROUND[name] * np.abs(f64(ref)) * 1.01 + TINY[name], f"{name} {cache}")
    assert gaps_kept(o)
    if more_rows:
        assert bool((o[n:] == 5.0).all())
    return o, c, q


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 300])
def test_one_token(q4lib, name, cache, length):
    run(q4lib, name, cache, 4, 2, 128, 16, [length], [1])


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("d", [8, 40, 64, 72, 128, 136, 192, 200, 256])
@pytest.mark.parametrize("new", [1, 9, 40])
def test_head_sizes(q4lib, name, cache, d, new):
    run(q4lib, name, cache, 6, 2, d, 32, [new + 50, 90], [new, min(new, 4)])


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (5, 5), (3, 1), (8, 1), (10, 2), (12, 4), (32, 2)])
@pytest.mark.parametrize("new", [1, 3, 7, 33])
def test_head_layouts(q4lib, name, cache, heads, kv_heads, new):
    """Groups of query heads that share a cached head, blocks of rows that end
    inside a group."""
    run(q4lib, name, cache, heads, kv_heads, 64, 64, [new, new + 1, new + 200], [new, new, new])


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 1024])
@pytest.mark.parametrize("new", [1, 6, 30, 100])
def test_ragged(q4lib, name, cache, page, new):
    """Sequences of all sizes in one call, some without new tokens, rows and
    queries past the last one."""
    rng = np.random.default_rng(page + new)
    lens = [int(x) for x in rng.integers(0, 400, 9)] + [700, 1, 0]
    counts = [min(int(rng.integers(0, new + 1)), n) for n in lens]
    counts[9] = new
    run(q4lib, name, cache, 4, 2, 128, page, lens, counts, more_rows=3)


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 200])
@pytest.mark.parametrize("new", [1, 5, 80])
def test_window(q4lib, name, cache, window, new):
    run(q4lib, name, cache, 4, 2, 64, 32, [new, new + 130, 500], [new, new, new], window=window)


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("pad,shift", [(1, 0), (8, 0), (0, 1), (3, 5), (64, 0)])
def test_rows_anywhere(q4lib, name, cache, pad, shift):
    run(q4lib, name, cache, 4, 2, 80, 16, [100, 7], [20, 2], pad=pad, shift=shift)


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("new", [1, 4, 20])
def test_long(q4lib, name, cache, new):
    """Long sequences next to short ones: a sequence is dealt to many CTAs."""
    run(q4lib, name, cache, 8, 2, 128, 64, [9001, 3, 2500], [new, 1, new], max_new=0)


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("d", [64, 128])
def test_blocks_of_all_sizes_in_a_row(q4lib, name, cache, d):
    """Blocks of few and of many rows in turn, over more tiles than any ring has."""
    counts = [20, 70, 33, 300, 17, 130, 64, 65]
    run(q4lib, name, cache, 8, 2, d, 32, [n + 1500 for n in counts], counts)


@pytest.mark.parametrize("name,cache", KINDS)
def test_prompt(q4lib, name, cache):
    run(q4lib, name, cache, 4, 2, 128, 64, [515, 700], [515, 300])


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("sharp", [1e-3, 8.0])
def test_flat_and_sharp(q4lib, name, cache, sharp):
    """All terms alike, and scores of +-100."""
    run(q4lib, name, cache, 4, 1, 128, 16, [700, 20], [5, 5], sharp=sharp)


@pytest.mark.parametrize("name,cache", KINDS)
def test_max_new_is_only_a_hint(q4lib, name, cache):
    for max_new in (0, 1, 50, 1000):
        run(q4lib, name, cache, 4, 2, 128, 16, [300, 41], [50, 1], max_new=max_new)


@pytest.mark.parametrize("name,cache", KINDS)
def test_many_sequences(q4lib, name, cache):
    rng = np.random.default_rng(11)
    lens = [int(x) for x in rng.integers(0, 60, 1024)]
    run(q4lib, name, cache, 2, 1, 64, 16, lens, [min(1, n) for n in lens])


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("new", [4, 40])
def test_rows_that_see_nothing(q4lib, name, cache, new):
    """A len below the number of new tokens: the first rows have no place in the
    sequence, and give zeros. An empty sequence with new tokens, too."""
    g = torch.Generator(device="cuda").manual_seed(1)
    kv_heads, heads, d = 2, 4, 64
    k = torch.randn(new, kv_heads * d, generator=g, device="cuda").to(TYPES[name])
    c = Cache(q4lib, [new, 0], kv_heads, d, 16, cache)
    c.write(k, k, name, [new, 0], [new, 0])
    q = torch.randn(2 * new, heads * d, generator=g, device="cuda").to(TYPES[name])
    o = blank(2 * new, heads * d, name)
    c.attend(o, q, name, heads, 0.125, 0, [new - 3, 0], [new, new])
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
    kk = held(k.reshape(new, kv_heads, d), cache)[:new - 3]
    ref, tol = attend64(q[:new], kk, kk, heads, kv_heads, d, 0.125, 0, [new - 3], [new], ROUND_P[name, cache], 2 if name == "f32" else 1)
    assert not bool(ref[:3].any()) and not bool(o[:3].any()) and not bool(o[new:].any())
    close(o[:new], f64(ref), f64(tol) + ROUND[name] * np.abs(f64(ref)) * 1.01 + TINY[name])


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("new", [8, 60, 130])
def test_what_is_not_finite_stays_with_its_rows(q4lib, name, cache, new):
    """A token whose key or value is not finite: NaN in the rows that see it, in
    the query heads of its head alone; the rows before it as ever. Pages hold NaN
    wherever no token was written."""
    g = torch.Generator(device="cuda").manual_seed(2)
    kv_heads, heads, d, length = 2, 4, 64, new + 70
    k = torch.randn(length, kv_heads, d, generator=g, device="cuda").to(TYPES[name])
    v = torch.randn(length, kv_heads, d, generator=g, device="cuda").to(TYPES[name])
    q = torch.randn(new, heads * d, generator=g, device="cuda").to(TYPES[name])
    at = length - 3
    bad_k, bad_v = k.clone(), v.clone()
    bad_v[at, 1, 7] = float("inf")
    bad_k[at + 1, 0, 0] = float("nan")
    outs = []
    for kk, vv in ((k, v), (bad_k, bad_v)):
        c = Cache(q4lib, [length], kv_heads, d, 32, cache)
        c.write(kk.reshape(length, -1), vv.reshape(length, -1), name, [length], [length])
        o = blank(new, heads * d, name)
        c.attend(o, q, name, heads, 0.125, 0, [length], [new])
        outs.append(o)
    good, bad = outs
    assert bool(torch.isfinite(good).all())
    hit = torch.zeros_like(bad, dtype=torch.bool)
    hit[new - 3:, 2 * d:] = True
    hit[new - 2:, :2 * d] = True
    assert torch.equal(torch.isnan(bad), hit)
    assert torch.equal(bad[~hit], good[~hit])


@pytest.mark.parametrize("name,cache", KINDS)
def test_queries_that_are_not_finite(q4lib, name, cache):
    g = torch.Generator(device="cuda").manual_seed(2)
    kv_heads, heads, d, length = 1, 2, 64, 90
    k = torch.randn(length, kv_heads * d, generator=g, device="cuda").to(TYPES[name])
    c = Cache(q4lib, [length], kv_heads, d, 32, cache)
    c.write(k, k, name, [length], [length])
    q = torch.randn(3, heads * d, generator=g, device="cuda").to(TYPES[name])
    good, bad = blank(3, heads * d, name), blank(3, heads * d, name)
    c.attend(good, q, name, heads, 0.125, 0, [length], [3])
    q[1, 3] = float("nan")
    q[2, d + 1] = float("nan")
    c.attend(bad, q, name, heads, 0.125, 0, [length], [3])
    hit = torch.zeros_like(bad, dtype=torch.bool)
    hit[1, :d] = True
    hit[2, d:] = True
    assert torch.equal(torch.isnan(bad), hit) and torch.equal(bad[~hit], good[~hit])


@pytest.mark.parametrize("name,cache", [("bf16", "i8"), ("f32", "i8")])
def test_scales_of_all_sizes(q4lib, name, cache):
    """Codes whose scales span many powers of two: values from 1e-30 to 1e30, and
    rows of zeros."""
    kv_heads, heads, d, length = 1, 2, 64, 200
    g = torch.Generator(device="cuda").manual_seed(4)
    k = torch.randn(length, 1, d, generator=g, device="cuda").to(TYPES[name])
    v = torch.randn(length, 1, d, generator=g, device="cuda").to(TYPES[name])
    for order in (1, -1):
        size = torch.logspace(-30, 30, length, device="cuda")
        vv = (v * (size if order == 1 else size.flip(0))[:, None, None]).to(TYPES[name])
        vv[::7] = 0.0
        c = Cache(q4lib, [length], kv_heads, d, 16, cache)
        c.write(k.reshape(length, -1), vv.reshape(length, -1), name, [length], [length])
        q = torch.randn(length, heads * d, generator=g, device="cuda").to(TYPES[name])
        o = blank(length, heads * d, name)
        c.attend(o, q, name, heads, 0.125, 0, [length], [length])
        ref, tol = attend64(q, held(k, cache), held(vv, cache), heads, kv_heads, d, 0.125, 0, [length], [length], ROUND_P[name, cache],
                            2 if name == "f32" else 1, (name, cache) == FOLDED)
        close(o, f64(ref), f64(tol) + ROUND[name] * np.abs(f64(ref)) * 1.01 + TINY[name])


def test_query_is_the_output(q4lib):
    """O may be Q."""
    _, c, q = run(q4lib, "bf16", "bf16", 4, 2, 128, 16, [300, 40], [7, 2])
    o = blank(9, 512, "bf16")
    c.attend(o, q, "bf16", 4, 0.1, 0, [300, 40], [7, 2])
    c.attend(q, q, "bf16", 4, 0.1, 0, [300, 40], [7, 2])
    assert torch.equal(o, q)


@pytest.mark.parametrize("name,cache", KINDS)
def test_same_bits_again(q4lib, name, cache):
    o, c, q = run(q4lib, name, cache, 8, 2, 128, 64, [5000, 700], [9, 3])
    again = blank(*o.shape, name)
    for _ in range(3):
        c.attend(again, q, name, 8, 128 ** -0.5, 0, [5000, 700], [9, 3])
        assert torch.equal(o, again)


def test_rewound(q4lib):
    """A smaller len is the sequence before its last tokens were written."""
    g = torch.Generator(device="cuda").manual_seed(8)
    k = torch.randn(90, 128, generator=g, device="cuda").bfloat16()
    c = Cache(q4lib, [90], 1, 128, 16, "i8")
    c.write(k, k, "bf16", [90], [90])
    q = torch.randn(2, 256, generator=g, device="cuda").bfloat16()
    a, b = blank(2, 256, "bf16"), blank(2, 256, "bf16")
    c.attend(a, q, "bf16", 2, 0.1, 0, [70], [2])
    d = Cache(q4lib, [70], 1, 128, 16, "i8")
    d.write(k[:70], k[:70], "bf16", [70], [70])
    d.attend(b, q, "bf16", 2, 0.1, 0, [70], [2])
    assert torch.equal(a, b)


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("new", [1, 80])
def test_bad_page_is_recorded(q4lib, name, cache, new):
    c = Cache(q4lib, [100], 1, 64, 16, cache, fill=0)
    q, o = rows(torch.ones(new, 64), name), blank(new, 64, name)
    good = int(c.table[0, 3])
    for bad in (-1, c.n_pages, 1 << 30):
        c.table[0, 3] = bad
        c.attend(o, q, name, 1, 0.1, 0, [100], [new])
        torch.cuda.synchronize()
        assert q4lib.q4_last_device_status(clear=True) == q4lib.Q4_ERR_DEVICE_CHECK
    # not needed: not looked at
    c.attend(o, q, name, 1, 0.1, 0, [48], [min(new, 48)])
    c.attend(o, q, name, 1, 0.1, 36, [100], [1])
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
    c.table[0, 3] = good
    c.attend(o, q, name, 1, 0.1, 0, [100], [new])
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
