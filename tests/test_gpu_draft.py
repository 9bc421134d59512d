"""Probabilities from logits, and the verification of drafted tokens, against 64
bits: rows of all lengths and alignments, temperatures, banned tokens, greedy
rows; and the accepted and drawn tokens, exactly."""

import numpy as np
import pytest
import torch

from block_testlib import TYPES, blank, close, f64, gaps_kept, rows, type_of

pytestmark = pytest.mark.gpu


def probs(q4, x, name, temperature, pad=0, shift=0):
    p = blank(x.shape[0], x.shape[1], "f32", pad, shift)
    q4.q4_token_probs(p, p.stride(0), x, x.stride(0), type_of(q4, name), temperature, x.shape[0], x.shape[1])
    return p


def softmax64(x, t):
    z = f64(x) / t[:, None]
    top = z.max(axis=1, keepdims=True)
    e = np.exp(z - np.where(np.isinf(top), 0.0, top))
    s = e.sum(axis=1, keepdims=True)
    p = e / np.where(s == 0, 1.0, s)
    # the argument (x - max) log2(e) / T: three roundings; 2^x: 2^-22; the sum: 2^-24 for
    # each of 40 values a thread and 42 more steps at most for its tree; two products
    away = np.abs(np.where(np.isinf(z), 0.0, z - np.where(np.isinf(top), 0.0, top))) * 1.4427
    return p, p * (4 * away * 2.0 ** -24 + 2.0 ** -21 + (x.shape[1] / 8192 + 90) * 2.0 ** -24) + 2.0 ** -126


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 7, 64, 1000, 4097, 32768, 50257, 151936, 300001])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (1, 3)])
def test_probabilities(q4lib, name, n, pad, shift):
    g = torch.Generator(device="cuda").manual_seed(n)
    m = 3
    x = torch.randn(m, n, generator=g, device="cuda") * 3
    x[torch.rand(m, n, generator=g, device="cuda") < 0.1] = float("-inf")
    x[1, n // 2] = 40.0
    x = rows(x, name, pad, shift)
    t = torch.tensor([1.0, 0.7, 2.5], device="cuda")
    p = probs(q4lib, x, name, t, pad, shift)
    ref, tol = softmax64(x, f64(t))
    close(p, ref, tol)
    assert gaps_kept(p)
    ref, tol = softmax64(x, np.ones(m))
    close(probs(q4lib, x, name, None), ref, tol)


@pytest.mark.parametrize("rows_", [1, 5, 64, 333])
def test_many_rows(q4lib, rows_):
    g = torch.Generator(device="cuda").manual_seed(rows_)
    x = torch.randn(rows_, 10000, generator=g, device="cuda") * 2
    ref, tol = softmax64(x, np.ones(rows_))
    close(probs(q4lib, x, "f32", None), ref, tol)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("n", [5, 1000, 151936])
def test_greedy(q4lib, name, n):
    """Temperature 0: the lowest of the largest logits."""
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.round(torch.randn(4, n, generator=g, device="cuda") * 2).to(TYPES[name])   # many ties
    x[1, -1] = 50.0
    x[2] = float("-inf")
    x[3, 0] = float("nan")
    t = torch.tensor([0.0, 0.0, 0.0, 0.0], device="cuda")
    p = probs(q4lib, x, name, t)
    want = torch.zeros_like(p)
    want[0, int(f64(x[0]).argmax())] = 1.0
    want[1, n - 1] = 1.0
    want[3, int(np.nanargmax(f64(x[3])))] = 1.0
    assert torch.equal(p, want)


@pytest.mark.parametrize("n", [9, 70000])
def test_rows_without_probabilities(q4lib, n):
    x = torch.zeros(5, n, device="cuda")
    x[0] = float("-inf")
    x[1, 3] = float("nan")
    x[2, n - 1] = float("inf")
    t = torch.tensor([1.0, 1.0, 1.0, -1.0, 1.0], device="cuda")
    p = probs(q4lib, x, "f32", t)
    assert not bool(p[0].any())
    assert bool(torch.isnan(p[1]).all()) and bool(torch.isnan(p[2]).any()) and bool(torch.isnan(p[3]).all())
    close(p[4], np.full(n, 1.0 / n), np.full(n, 2.0 ** -20 / n))


def verify(q4, p, q, drafted, counts, accept, sample, n, pad=0):
    s, t = drafted.shape
    tokens = torch.full((s, t + 1 + pad), 99, dtype=torch.int32, device="cuda")
    kept = torch.full((s,), -5, dtype=torch.int32, device="cuda")
    q4.q4_draft_verify(tokens, tokens.stride(0), kept, p, p.stride(0), q, q.stride(0) if q is not None else 0, drafted,
                       max(1, drafted.stride(0)), counts, accept, max(1, accept.stride(0)), sample, s, t, n)
    torch.cuda.synchronize()
    assert bool((tokens[:, t + 1:] == 99).all())
    return tokens[:, :t + 1].cpu().numpy(), kept.cpu().numpy()


def verify64(p, q, drafted, counts, accept, sample, n):
    """The definition, a slot at a time, with sums in 64 bits."""
    p, a, u = f64(p), f64(accept), f64(sample)
    q = None if q is None else f64(q)
    drafted = drafted.cpu().numpy()
    s, t = drafted.shape
    tokens, kepts = np.full((s, t + 1), -1, dtype=np.int32), np.zeros(s, dtype=np.int32)
    for i in range(s):
        count = t if counts is None else int(counts[i])
        kept = 0
        while kept < count:
            x = drafted[i, kept]
            if not 0 <= x < n:
                break
            qx = 1.0 if q is None else q[i * t + kept, x]
            if not a[i, kept] * qx < p[i * (t + 1) + kept, x]:
                break
            kept += 1
        left = p[i * (t + 1) + kept].copy()
        rest = left
        if kept < count:
            if q is None:
                rest = left.copy()
                if 0 <= drafted[i, kept] < n:
                    rest[drafted[i, kept]] = 0.0
            else:
                rest = np.maximum(left - q[i * t + kept], 0.0)
        if rest.sum() == 0:
            rest = left
        run = np.cumsum(rest)
        past = np.nonzero(run > u[i] * run[-1])[0]
        tokens[i, :kept] = drafted[i, :kept]
        tokens[i, kept] = past[0] if len(past) else 0
        kepts[i] = kept
    return tokens, kepts


@pytest.mark.parametrize("n", [1, 2, 5, 31, 257, 2048, 20000, 151936, 100003])
@pytest.mark.parametrize("draft", [1, 4, 40])
@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("pad", [0, 1])
def test_verification(q4lib, n, draft, given, pad):
    g = torch.Generator(device="cuda").manual_seed(n + draft)
    s = 6 if n > 50000 and draft > 8 else 17
    target = 2 * torch.randn(s, draft + 1, n, generator=g, device="cuda")
    other = 2 * torch.randn(s, draft, n, generator=g, device="cuda")
    p = rows(torch.softmax(target, dim=2).reshape(-1, n), "f32", pad)
    q = torch.softmax(0.8 * target[:, :draft] + 0.2 * other, dim=2).reshape(-1, n)
    drafted = torch.multinomial(q, 1, generator=g).reshape(s, draft).to(torch.int32)
    q = rows(q, "f32", pad) if given else None
    drafted[2, 0] = -1                              # padding
    drafted[3, draft - 1] = n
    counts = torch.randint(0, draft + 1, (s,), generator=g, device="cuda").to(torch.int32)
    counts[2:4] = draft
    accept = torch.rand(s, draft, generator=g, device="cuda") * (0.2 if not given else 1.0)
    sample = torch.rand(s, generator=g, device="cuda")
    for c in (counts, None):
        got, want = verify(q4lib, p, q, drafted, c, accept, sample, n, pad), verify64(p, q, drafted, c, accept, sample, n)
        assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])


@pytest.mark.parametrize("n", [4, 3000, 60000])
def test_edges_of_the_draw(q4lib, n):
    """u = 0 takes the first index with some probability, u just below 1 the last;
    places between equal steps go up; probabilities in a few steps are exact."""
    p = torch.zeros(6, n, device="cuda")
    for i, at in enumerate(([1, n - 1], [0, 2], [n // 2, n - 2])):
        p[2 * i + 1, at[0]] = 0.25
        p[2 * i + 1, at[1]] = 0.75 if at[1] != at[0] else 1.0
    p = p[1::2].contiguous()                        # max_draft = 0: one row a slot
    none = torch.zeros((3, 0), dtype=torch.int32, device="cuda")
    acc = torch.zeros((3, 0), device="cuda")
    for u in (0.0, 0.24999999, 0.25, 0.5, 0.99999994, 2.0 ** -149, 1e-30):
        sample = torch.full((3,), u, device="cuda")
        got = verify(q4lib, p, None, none, None, acc, sample, n)
        want = verify64(p, None, none, None, acc, sample, n)
        assert np.array_equal(got[0], want[0]) and not got[1].any()


@pytest.mark.parametrize("slots", [1, 40])
@pytest.mark.parametrize("pad", [0, 1])
def test_largest_vocabulary(q4lib, slots, pad):
    """Equal probabilities of 2^-20 each: the token is the whole part of u 2^20, exactly."""
    n = 1 << 20
    p = torch.full((slots, n + pad), 2.0 ** -20, device="cuda")[:, :n]
    sample = (torch.arange(slots, device="cuda", dtype=torch.float32) + 1 + 2.0 ** -10) / (slots + 1)
    sample[-1] = 0.99999994
    none, acc = torch.zeros((slots, 0), dtype=torch.int32, device="cuda"), torch.zeros((slots, 0), device="cuda")
    got, _ = verify(q4lib, p, None, none, None, acc, sample, n)
    assert np.array_equal(got[:, 0], np.floor(f64(sample) * n).astype(np.int32))


def test_nothing_left(q4lib):
    """p = q with a token refused all the same, and rows of zeros."""
    n = 5000
    g = torch.Generator(device="cuda").manual_seed(1)
    p = torch.softmax(torch.randn(6, n, generator=g, device="cuda"), dim=1)
    p[4:] = 0.0
    q = p[0::2].contiguous()
    drafted = torch.tensor([[3], [4], [5]], dtype=torch.int32, device="cuda")
    q[0, 3] *= 2.0                                  # refused, and what is left is nothing but rounding
    p[0], q[0] = q[0].clone(), q[0]
    p[0, 3] /= 2.0
    accept, sample = torch.full((3, 1), 0.9, device="cuda"), torch.tensor([0.3, 0.6, 0.9], device="cuda")
    got, want = verify(q4lib, p, q, drafted, None, accept, sample, n), verify64(p, q, drafted, None, accept, sample, n)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_probabilities_that_are_none(q4lib):
    """NaN and negative ones count as 0; tokens stay inside the vocabulary."""
    n = 3000
    p = torch.full((2, n), float("nan"), device="cuda")
    p[0, 7], p[0, 9], p[0, 8] = 0.5, 0.5, -3.0
    none, acc = torch.zeros((2, 0), dtype=torch.int32, device="cuda"), torch.zeros((2, 0), device="cuda")
    for u, x in ((0.1, 7), (0.6, 9)):
        got, _ = verify(q4lib, p, None, none, None, acc, torch.full((2,), u, device="cuda"), n)
        assert got[0, 0] == x and got[1, 0] == 0
