"""Tokens sorted by expert and back, and the gradient, through the C ABI: the
sort and its copies exactly, sums against 64 bits.

Tolerances, e = 2^-24: a token's row is a sum of at most top_k + 1 terms in
fp32, so (top_k + 2) e of the sum of the terms' sizes and half a unit of the
stored type; a weight's gradient is a sum over d values in chains of d / 32 and
a tree, held to (d / 32 + 8) e of the sum of the terms' sizes."""

import numpy as np
import pytest

from block_testlib import ROUND, TINY, TYPES, blank, close, f64, gaps_kept, rows, type_of

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def choices(t, k, e, seed, drop=0.1, one=False):
    rng = np.random.default_rng(seed)
    ids = np.full((t, k), e - 1) if one else np.minimum(rng.geometric(min(0.9, 3.0 / e), (t, k)) - 1, e - 1)
    ids[rng.random((t, k)) < drop] = -1
    if drop and t > 2:
        ids[1] = -1                     # a token without any expert
        ids[2, 0] = e                   # ids past the last expert are none either
        ids[2, -1] = -2 ** 31
    return ids


def reference(ids, e):
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < e), flat, e)
    pair_of = np.argsort(key, kind="stable")
    row = np.empty_like(pair_of)
    row[pair_of] = np.arange(flat.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=e + 1)[:e])])
    return offsets, np.where(key < e, row, -1 - row).reshape(ids.shape), pair_of


def workspace(q4lib, t, k, e):
    n = q4lib.q4_moe_workspace_size(t, k, e)
    return torch.full((max(n, 1),), 0xAB, dtype=torch.uint8, device="cuda"), n


def dispatch(q4lib, ids, e, X, name, int64=True, pad=0, shift=0, pairs=True, stream=None):
    t, k = ids.shape
    idd = torch.as_tensor(ids, dtype=torch.int64 if int64 else torch.int32).cuda()
    offsets = torch.full((e + 1,), -9, dtype=torch.int64, device="cuda")
    row_of = torch.full((t, k), -9, dtype=torch.int32, device="cuda")
    pair_of = torch.full((t * k,), -9, dtype=torch.int32, device="cuda") if pairs else None
    ws, wsb = workspace(q4lib, t, k, e)
    Xs = blank(t * k, X.shape[1], name, pad, shift) if X is not None else None
    torch.cuda.synchronize()
    q4lib.q4_moe_dispatch(Xs, Xs.stride(0) if X is not None else 0, offsets, row_of, pair_of, idd, 8 if int64 else 4, X,
                          X.stride(0) if X is not None else 0, type_of(q4lib, name), t, k, e,
                          X.shape[1] if X is not None else 0, ws, wsb, stream=stream)
    torch.cuda.synchronize()
    return offsets.cpu().numpy(), row_of.cpu().numpy(), pair_of.cpu().numpy() if pairs else None, Xs


CASES = [(1, 1, 1), (1, 8, 128), (2, 2, 3), (31, 3, 7), (128, 8, 64), (129, 8, 64), (1000, 2, 512), (3000, 1, 513),
         (700, 6, 4096), (5000, 8, 100), (40000, 4, 33)]


@pytest.mark.parametrize("t,k,e", CASES)
@pytest.mark.parametrize("int64", [True, False])
@pytest.mark.parametrize("drop", [0.0, 0.2])
def test_sort(q4lib, t, k, e, int64, drop):
    ids = choices(t, k, e, t + e, drop)
    got = dispatch(q4lib, ids, e, None, "f32", int64)
    for a, b in zip(got[:3], reference(ids, e)):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("t,k,e", [(1, 4, 8), (300, 2, 5), (9000, 2, 5)])
@pytest.mark.parametrize("what", ["one expert", "none"])
def test_sort_of_one_expert_and_of_none(q4lib, t, k, e, what):
    ids = choices(t, k, e, 1, 0.0, one=True) if what == "one expert" else np.full((t, k), -1)
    got = dispatch(q4lib, ids, e, None, "f32")
    for a, b in zip(got[:3], reference(ids, e)):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("t,k,e", [(1, 8, 16), (130, 3, 9), (2000, 8, 64)])
@pytest.mark.parametrize("d", [1, 3, 8, 33, 256, 1000])
@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (2, 2), (1, 1)])
def test_rows_in_order(q4lib, t, k, e, d, name, pad, shift):
    ids = choices(t, k, e, d)
    X = rows(torch.as_tensor(np.random.default_rng(2).standard_normal((t, d))), name, pad, shift)
    X[0, 0] = float("nan")
    offsets, row_of, pair_of, Xs = dispatch(q4lib, ids, e, X, name, pad=pad, shift=shift)
    ref = reference(ids, e)
    assert np.array_equal(row_of, ref[1])
    kept = ref[1].reshape(-1)[ref[2]] >= 0
    want = X[torch.as_tensor(ref[2] // k).cuda()].clone()
    want[torch.as_tensor(~kept).cuda()] = 0.0
    assert torch.equal(Xs.contiguous().view(torch.uint8), want.contiguous().view(torch.uint8))
    assert gaps_kept(Xs)


@pytest.mark.parametrize("t", [100, 5000])
def test_pairs_are_optional_and_streams_do_not_matter(q4lib, t):
    ids = choices(t, 4, 12, 3)
    X = torch.randn(t, 64, device="cuda")
    a = dispatch(q4lib, ids, 12, X, "f32", pairs=False)
    b = dispatch(q4lib, ids, 12, X, "f32", stream=torch.cuda.Stream())
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1]) and torch.equal(a[3], b[3])


def sorted_rows(ids, e, d, name, seed, pad=0, shift=0):
    """Rows as experts would write them; those of pairs without one hold NaN
    and infinities."""
    row_of = reference(ids, e)[1]
    y = torch.as_tensor(np.random.default_rng(seed).standard_normal((ids.size, d)))
    n = int((row_of >= 0).sum())
    y[n:] = float("nan")
    y[n + 1::2] = float("inf")
    return torch.as_tensor(row_of, dtype=torch.int32).cuda(), rows(y, name, pad, shift)


SHAPES = [(1, 8, 16, 2560), (1, 1, 1, 1), (33, 3, 5, 257), (500, 8, 64, 96), (2000, 2, 16, 130), (77, 5, 8, 1000), (20, 12, 30, 4096)]


@pytest.mark.parametrize("t,k,e,d", SHAPES)
@pytest.mark.parametrize("name,pad,shift", [("f32", 0, 0), ("f32", 1, 1), ("f16", 0, 0), ("bf16", 8, 0), ("bf16", 2, 2), ("bf16", 1, 1)])
@pytest.mark.parametrize("base,weighted", [(False, True), (True, True), (False, False)])
def test_combine(q4lib, t, k, e, d, name, pad, shift, base, weighted):
    ids = choices(t, k, e, d)
    row_of, Ys = sorted_rows(ids, e, d, name, 4, pad, shift)
    w = torch.as_tensor(np.random.default_rng(5).standard_normal((t, k)), dtype=torch.float32).cuda()
    w[row_of < 0] = float("nan")
    bs = rows(torch.as_tensor(np.random.default_rng(6).standard_normal((t, d))), name, pad, shift) if base else None
    Y = blank(t, d, name, pad, shift)
    q4lib.q4_moe_combine(Y, Y.stride(0), bs, bs.stride(0) if base else 0, Ys, Ys.stride(0), type_of(q4lib, name), row_of,
                         w if weighted else None, t, k, d)
    r, has = row_of.cpu().numpy(), (row_of >= 0).cpu().numpy()
    y, size = (f64(bs), np.abs(f64(bs))) if base else (np.zeros((t, d)), np.zeros((t, d)))
    ys, wv = f64(Ys), f64(w) if weighted else np.ones((t, k))
    for j in range(k):
        i = np.nonzero(has[:, j])[0]
        term = wv[i, j, None] * ys[r[i, j]]
        y[i] += term
        size[i] += np.abs(term)
    close(Y, y, (k + 2) * E * size + ROUND[name] * np.abs(y) + TINY[name])
    assert gaps_kept(Y)


@pytest.mark.parametrize("t,k,e,d", SHAPES)
@pytest.mark.parametrize("name,pad,shift", [("f32", 0, 0), ("f32", 1, 1), ("f16", 0, 0), ("bf16", 8, 0), ("bf16", 2, 2), ("bf16", 1, 1)])
def test_combine_backward(q4lib, t, k, e, d, name, pad, shift):
    ids = choices(t, k, e, d)
    row_of, Ys = sorted_rows(ids, e, d, name, 7, pad, shift)
    w = torch.as_tensor(np.random.default_rng(8).standard_normal((t, k)), dtype=torch.float32).cuda()
    dY = rows(torch.as_tensor(np.random.default_rng(9).standard_normal((t, d))), name, pad, shift)
    dYs, dw = blank(t * k, d, name, pad, shift), torch.full((t, k), float("nan"), device="cuda")
    q4lib.q4_moe_combine_backward(dYs, dYs.stride(0), dw, dY, dY.stride(0), Ys, Ys.stride(0), type_of(q4lib, name), row_of, w, t,
                                  k, d)
    r, has = row_of.cpu().numpy(), (row_of >= 0).cpu().numpy()
    g, ys, wv = f64(dY), f64(Ys), f64(w)
    dys, dwr, size = np.zeros((t * k, d)), np.zeros((t, k)), np.zeros((t, k))
    for j in range(k):
        i = np.nonzero(has[:, j])[0]
        dys[r[i, j]] = wv[i, j, None] * g[i]
        term = g[i] * ys[r[i, j]]
        dwr[i, j], size[i, j] = term.sum(axis=1), np.abs(term).sum(axis=1)
    close(dYs, dys, (E + ROUND[name]) * np.abs(dys) + TINY[name], "dys")
    close(dw, dwr, (d / 32 + 8) * E * size + 1e-37, "dweights")
    assert gaps_kept(dYs)
    again = blank(t * k, d, name, pad, shift)
    q4lib.q4_moe_combine_backward(again, again.stride(0), None, dY, dY.stride(0), Ys, Ys.stride(0), type_of(q4lib, name), row_of,
                                  w, t, k, d)
    assert torch.equal(again, dYs)


def test_in_place(q4lib):
    ids = choices(50, 3, 6, 10)
    row_of, Ys = sorted_rows(ids, 6, 64, "f32", 11)
    base, w = torch.randn(50, 64, device="cuda"), torch.rand(50, 3, device="cuda")
    Y = torch.empty_like(base)
    q4lib.q4_moe_combine(Y, 64, base, 64, Ys, 64, 0, row_of, w, 50, 3, 64)
    q4lib.q4_moe_combine(base, 64, base, 64, Ys, 64, 0, row_of, w, 50, 3, 64)
    assert torch.equal(Y, base)
    a, b, dw = torch.empty_like(Ys), Ys.clone(), torch.empty_like(w)
    q4lib.q4_moe_combine_backward(a, 64, dw, Y, 64, Ys, 64, 0, row_of, w, 50, 3, 64)
    q4lib.q4_moe_combine_backward(b, 64, dw, Y, 64, b, 64, 0, row_of, w, 50, 3, 64)
    assert torch.equal(a, b)


def test_gradients_against_differences(q4lib):
    # L = sum of c * Y through dispatch, a fixed linear map per row, and combine:
    # L is linear in X and in the weights, so differences of any step are exact
    # up to rounding
    t, k, e, d = 40, 4, 6, 48
    rng = np.random.default_rng(12)
    ids = choices(t, k, e, 13)
    X, c = (np.float64(np.float32(rng.standard_normal((t, d)))) for _ in range(2))
    w = np.float64(np.float32(rng.standard_normal((t, k))))
    a = np.float64(np.float32(rng.standard_normal(e + 1)))     # expert's factor
    offsets, row_of, pair_of = reference(ids, e)
    factor = a[np.minimum(np.searchsorted(offsets, np.arange(t * k), side="right") - 1, e)]

    def loss(X, w):
        ys = X[pair_of // k] * factor[:, None]
        y = np.where((row_of >= 0)[:, :, None], w[:, :, None] * ys[np.maximum(row_of, 0)], 0.0).sum(axis=1)
        return (c * y).sum()

    dev = lambda v: torch.as_tensor(v, dtype=torch.float32).cuda()   # noqa: E731
    _, rd, _, Xs = dispatch(q4lib, ids, e, dev(X), "f32")
    rd = torch.as_tensor(rd).cuda()
    f = dev(factor)[:, None]
    Ys, dYs, dw, dX = (Xs * f).contiguous(), torch.empty((t * k, d), device="cuda"), torch.empty((t, k), device="cuda"), torch.empty((t, d), device="cuda")
    q4lib.q4_moe_combine_backward(dYs, d, dw, dev(c), d, Ys, d, 0, rd, dev(w), t, k, d)
    q4lib.q4_moe_combine(dX, d, None, 0, (dYs * f).contiguous(), d, 0, rd, None, t, k, d)
    for grad, args in ((f64(dX), lambda v, h: (X + h * v, w)), (f64(dw), lambda v, h: (X, w + h * v))):
        v = rng.standard_normal(grad.shape)
        diff = (loss(*args(v, 1.0)) - loss(*args(v, -1.0))) / 2
        assert abs((grad * v).sum() - diff) <= 1e-5 * np.abs(grad * v).sum()


def test_no_tokens(q4lib):
    offsets, r = torch.full((5,), 3, dtype=torch.int64, device="cuda"), torch.full((1,), 3, dtype=torch.int32, device="cuda")
    x = torch.full((1, 8), 3.0, device="cuda")
    q4lib.q4_moe_dispatch(x, 8, offsets, r, r, offsets, 8, x, 8, 0, 0, 2, 4, 8, None, 0)
    q4lib.q4_moe_combine(x, 8, None, 0, x, 8, 0, r, None, 0, 2, 8)
    q4lib.q4_moe_combine_backward(x, 8, x, x, 8, x, 8, 0, r, None, 0, 2, 8)
    torch.cuda.synchronize()
    assert bool((offsets == 0).all()) and bool((x == 3.0).all()) and int(r) == 3
