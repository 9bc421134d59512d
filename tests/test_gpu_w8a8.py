"""The int8 product with token and channel scales, through the C ABI: the token
coding bit for bit against the rule in numpy, the product against the 64-bit
product of the codes.

Tolerance: with B = sum_c |xq code| below 2^24 every sum is exact, and an output
has the roundings of sx * s_j, of the product and of its type: 3 halves of a
unit in the last place, taken as 2 units. Where B is larger the tensor cores
round (or cut) the running sum at each of k / 16 steps, at most 2^-23 of B."""

import numpy as np
import pytest

from block_testlib import ROUND, TINY, TYPES, blank, close, gaps_kept, rows, type_of

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def code_rows(x):
    """The rule, each step one fp32 operation."""
    x = np.asarray(x, np.float32)
    amax = np.abs(x).max(axis=1)
    codes = np.zeros(x.shape, np.int8)
    scale = np.zeros(x.shape[0], np.float32)
    for t in range(x.shape[0]):
        if not np.isfinite(x[t]).all():
            scale[t] = np.nan
        elif amax[t] >= np.float32(2.0 ** -110):
            scale[t] = amax[t] / np.float32(127)
            codes[t] = np.rint(x[t] * (np.float32(127) / amax[t])).astype(np.int8)
    return codes, scale


def tokens(m, k, name, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, k)) * np.exp(rng.uniform(-3, 3, (m, 1)))
    return torch.as_tensor(x).to(TYPES[name]).float().numpy()


def packed(q4lib, n, k, seed):
    rng = np.random.default_rng(seed)
    W = (rng.standard_normal((n, k)) * 0.05).astype(np.float32)
    W[::5] *= 0.01
    if n > 3:
        W[3] = 0.0
    P = torch.empty(q4lib.q4_w8_packed_size(n, k), dtype=torch.uint8, device="cuda")
    q4lib.q4_w8_quantize(P, torch.as_tensor(W).cuda(), n, k)
    return P, *code_rows(W)


def workspace(q4lib, m, k, n):
    need = q4lib.q4_w8a8_workspace_size(m, k, n)
    return torch.full((max(need, 1),), 0xAB, dtype=torch.uint8, device="cuda"), need


def reference(codes, scale, wc, ws, name):
    c, w = codes.astype(np.float64), wc.astype(np.float64)
    s = scale.astype(np.float64)[:, None] * ws.astype(np.float64)[None, :]
    y, B = (c @ w.T) * s, np.abs(c) @ np.abs(w).T
    tol = 2.0 * (ROUND["f32"] + ROUND[name]) * np.abs(y) + TINY[name]
    return y, tol + np.where(B >= 2.0 ** 24, codes.shape[1] / 16 * 2.0 ** -23 * B * np.abs(s), 0.0)


def run(q4lib, P, X, xname, yname, m, k, n, pad=0, shift=0):
    ws, wsb = workspace(q4lib, m, k, n)
    Xd, Y = rows(X, xname, pad, shift), blank(m, n, yname, pad, shift)
    q4lib.q4_w8a8_matmul(P, Xd, Xd.stride(0), type_of(q4lib, xname), Y, Y.stride(0), type_of(q4lib, yname), m, k, n, ws, wsb)
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
    assert gaps_kept(Y)
    return Y


@pytest.mark.parametrize("m,k", [(1, 1), (1, 32), (3, 2560), (17, 1000), (5, 4099), (700, 96), (2, 40000)])
@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (1, 1)])
def test_token_codes_bit_for_bit(q4lib, m, k, name, pad, shift):
    X = tokens(m, k, name, seed=m + k)
    if m > 2:
        X[1] = 0.0
        X[2, k // 2] = np.inf
    Xd = rows(X, name, pad, shift)
    codes = torch.full((m, k), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((m,), -1.0, device="cuda")
    q4lib.q4_a8_quantize(codes, scale, Xd, Xd.stride(0), type_of(q4lib, name), m, k)
    c, s = code_rows(X)
    assert np.array_equal(codes.cpu().numpy(), c)
    assert np.array_equal(np.nan_to_num(scale.cpu().numpy(), nan=-7.0),
                          np.nan_to_num(s, nan=-7.0))


def test_token_codes_of_tiny_and_large_rows(q4lib):
    X = np.zeros((6, 64), np.float32)
    X[0, 3], X[1, 3], X[2, 3], X[3, 3] = 2.0 ** -111, 2.0 ** -110, 2.0 ** -149, 3.4e38
    X[4, :] = -1e-30
    X[5, 5] = np.nan
    codes = torch.empty((6, 64), dtype=torch.int8, device="cuda")
    scale = torch.empty(6, device="cuda")
    q4lib.q4_a8_quantize(codes, scale, torch.as_tensor(X).cuda(), 64, q4lib.Q4_TYPE_F32, 6, 64)
    c, s = code_rows(X)
    assert np.array_equal(codes.cpu().numpy(), c)
    assert np.array_equal(np.nan_to_num(scale.cpu().numpy(), nan=-7.0), np.nan_to_num(s, nan=-7.0))


@pytest.mark.parametrize("m", [1, 2, 3, 7, 8, 9, 16, 17, 32, 33, 47, 64, 65, 100, 129, 257, 300])
@pytest.mark.parametrize("n,k", [(1, 32), (130, 96), (200, 1056), (513, 2080), (1000, 4096)])
def test_product(q4lib, m, n, k):
    P, wc, ws = packed(q4lib, n, k, seed=n)
    X = tokens(m, k, "f32", seed=m)
    Y = run(q4lib, P, X, "f32", "f32", m, k, n)
    y, tol = reference(*code_rows(X), wc, ws, "f32")
    close(Y, y, tol, f"m={m} n={n} k={k}")


@pytest.mark.parametrize("m,n,k", [(1, 9728, 2560), (4, 2560, 9728), (16, 14336, 4096), (31, 2560, 9728),
                                   (540, 9728, 2560), (540, 2560, 9728), (1100, 4096, 14336)])
def test_product_at_working_sizes(q4lib, m, n, k):
    P, wc, ws = packed(q4lib, n, k, seed=1)
    X = tokens(m, k, "bf16", seed=2)
    Y = run(q4lib, P, X, "bf16", "f32", m, k, n)
    y, tol = reference(*code_rows(X), wc, ws, "f32")
    close(Y, y, tol, f"m={m} n={n} k={k}")


@pytest.mark.parametrize("xname,yname", [("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("m", [1, 6, 13, 40, 290])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (3, 1)])
def test_types_and_strides(q4lib, xname, yname, m, pad, shift):
    n, k = 333, 544
    P, wc, ws = packed(q4lib, n, k, seed=3)
    X = tokens(m, k, xname, seed=4)
    Y = run(q4lib, P, X, xname, yname, m, k, n, pad, shift)
    y, tol = reference(*code_rows(X), wc, ws, yname)
    close(Y, y, tol, f"{xname} to {yname}")


@pytest.mark.parametrize("m", [1, 5, 12, 30, 70])
def test_sums_at_the_largest_codes(q4lib, m):
    # every product 127 * 127: the sums leave 2^24, up to 2^31
    n, k = 140, 131072
    W = torch.ones((n, k), device="cuda")
    W[1::2] = -1.0
    P = torch.empty(q4lib.q4_w8_packed_size(n, k), dtype=torch.uint8, device="cuda")
    q4lib.q4_w8_quantize(P, W, n, k)
    X = np.full((m, k), 0.5, np.float32)
    Y = run(q4lib, P, X, "f32", "f32", m, k, n)
    wc = np.where(np.arange(n) % 2, -127, 127).astype(np.int8)[:, None] * np.ones((1, k), np.int8)
    y, tol = reference(*code_rows(X), wc, np.full(n, np.float32(1) / np.float32(127)), "f32")
    close(Y, y, tol)


@pytest.mark.parametrize("m", [3, 20, 90])
def test_codes_form_is_the_same_product(q4lib, m):
    n, k = 270, 640
    P, wc, ws = packed(q4lib, n, k, seed=5)
    X = tokens(m, k, "f32", seed=6)
    Y = run(q4lib, P, X, "f32", "f32", m, k, n)
    c, s = code_rows(X)
    wsp, wsb = workspace(q4lib, m, k, n)
    Z = blank(m, n, "f32")
    q4lib.q4_w8a8_matmul_codes(P, torch.as_tensor(c).cuda(), torch.as_tensor(s).cuda(), Z, n, q4lib.Q4_TYPE_F32, m, k, n, wsp, wsb)
    assert torch.equal(Y, Z)


@pytest.mark.parametrize("m", [4, 24, 80])
def test_rows_without_a_finite_value_and_of_zeros(q4lib, m):
    n, k = 200, 256
    P, wc, ws = packed(q4lib, n, k, seed=7)
    X = tokens(m, k, "f32", seed=8)
    X[0, 9], X[1, 250], X[2] = np.nan, -np.inf, 0.0
    Y = run(q4lib, P, X, "f32", "f32", m, k, n)
    y, tol = reference(*code_rows(X), wc, ws, "f32")
    assert torch.isnan(Y[:2]).all()
    assert bool((Y[2] == 0).all())
    close(Y[2:], y[2:], tol[2:])


@pytest.mark.parametrize("m", [5, 33, 300])
def test_same_bits_each_run_and_on_another_stream(q4lib, m):
    n, k = 700, 1120
    P, _, _ = packed(q4lib, n, k, seed=9)
    X = tokens(m, k, "f32", seed=10)
    Y = run(q4lib, P, X, "f32", "f32", m, k, n)
    s = torch.cuda.Stream()
    Xd, Z = rows(X, "f32"), blank(m, n, "f32")
    ws, wsb = workspace(q4lib, m, k, n)
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        q4lib.q4_w8a8_matmul(P, Xd, k, 0, Z, n, 0, m, k, n, ws, wsb, stream=s)
    s.synchronize()
    assert torch.equal(Y, Z)


def test_calls_back_to_back_share_a_workspace(q4lib):
    # shapes in turn through one workspace in one stream
    shapes = [(300, 700, 1120), (1, 130, 96), (64, 513, 2080), (17, 200, 32), (9, 1000, 4096)]
    need = max(q4lib.q4_w8a8_workspace_size(m, k, n) for m, n, k in shapes)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    made = []
    for i, (m, n, k) in enumerate(shapes):
        P, wc, wsc = packed(q4lib, n, k, seed=20 + i)
        X = tokens(m, k, "f32", seed=30 + i)
        made.append((P, wc, wsc, X, rows(X, "f32"), blank(m, n, "f32")))
    torch.cuda.synchronize()
    for _ in range(3):
        for (m, n, k), (P, wc, wsc, X, Xd, Y) in zip(shapes, made):
            q4lib.q4_w8a8_matmul(P, Xd, k, 0, Y, n, 0, m, k, n, ws, need)
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
    for (m, n, k), (P, wc, wsc, X, Xd, Y) in zip(shapes, made):
        y, tol = reference(*code_rows(X), wc, wsc, "f32")
        close(Y, y, tol, f"m={m} n={n} k={k}")


def test_no_rows_write_nothing(q4lib):
    P, _, _ = packed(q4lib, 64, 64, seed=11)
    Y = torch.full((1, 64), 3.0, device="cuda")
    q4lib.q4_w8a8_matmul(P, Y, 64, 0, Y, 64, 0, 0, 64, 64, None, 0)
    q4lib.q4_w8a8_matmul_codes(P, P, Y, Y, 64, 0, 0, 64, 64, None, 0)
    q4lib.q4_a8_quantize(P, Y, Y, 64, 0, 0, 64)
    torch.cuda.synchronize()
    assert bool((Y == 3.0).all())


def test_a_workspace_too_small_is_refused(q4lib):
    for m in (4, 40):
        need = q4lib.q4_w8a8_workspace_size(m, 64, 64)
        P, _, _ = packed(q4lib, 64, 64, seed=12)
        X, Y = torch.ones((m, 64), device="cuda"), torch.full((m, 64), 3.0, device="cuda")
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        assert q4lib.q4_w8a8_matmul(P, X, 64, 0, Y, 64, 0, m, 64, 64, ws, need - 1, check=False) == q4lib.Q4_ERR_WORKSPACE
        assert q4lib.q4_w8a8_matmul(P, X, 64, 0, Y, 64, 0, m, 64, 64, None, 0, check=False) == q4lib.Q4_ERR_WORKSPACE
        torch.cuda.synchronize()
        assert bool((Y == 3.0).all())
