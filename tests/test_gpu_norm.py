"""The norms before and after a block and their gradients, through the C ABI,
against the formulas in 64 bits and (the gradients) against differences.

Tolerances, e = 2^-24: a mean of squares is a sum of positive terms over chains
of at most 128 additions and a tree, so within 160 e; its root halves that, and
a result adds a few products: 128 e of the normed part, one e of a sum, and half
a unit of the stored type. Sums with signs are held to e times the sum of their
terms' sizes."""

import numpy as np
import pytest

from block_testlib import ROUND, TINY, TYPES, blank, close, f64, gaps_kept, rows, type_of

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

E = 2.0 ** -24
EPS = 1e-6
GATES = ["none", "channel", "token", "full"]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def values(m, d, name, seed, spread=2.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, d)) * np.exp(rng.uniform(-spread, spread, (m, 1)))
    return torch.as_tensor(x).to(TYPES[name])


def weights(d, seed):
    return torch.as_tensor(1.0 + 0.3 * np.random.default_rng(seed).standard_normal(d), dtype=torch.float32).cuda()


def gate_of(q4lib, kind, m, d, name, seed, pad=0, shift=0):
    rng = np.random.default_rng(seed)
    if kind == "none":
        return None, 0, q4lib.Q4_GATE_NONE
    if kind == "full":
        g = rows(torch.as_tensor(rng.standard_normal((m, d))), name, pad, shift)
        return g, g.stride(0), q4lib.Q4_GATE_FULL
    n, k = (d, q4lib.Q4_GATE_CHANNEL) if kind == "channel" else (m, q4lib.Q4_GATE_TOKEN)
    return torch.as_tensor(rng.standard_normal(n), dtype=torch.float32).cuda(), 0, k


def wide(gate, kind):
    """The gate as it applies to [m x d] in 64 bits."""
    if kind == "none":
        return 1.0
    g = f64(gate)
    return g[None, :] if kind == "channel" else g[:, None] if kind == "token" else g


def unit(x, eps=EPS):
    r = 1.0 / np.sqrt((x * x).mean(axis=1, keepdims=True) + eps)
    return x * r, r


SIZES = [(1, 1), (1, 2560), (3, 5), (5, 32), (2, 33), (7, 257), (70, 160), (400, 130), (33, 1000), (310, 2048), (9, 4097),
         (320, 4096), (3, 9000), (2, 20000), (310, 8200)]


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (2, 2), (1, 1)])
def test_norm_before(q4lib, m, d, name, pad, shift):
    X, w = rows(values(m, d, name, m + d), name, pad, shift), weights(d, 1)
    H = blank(m, d, name, pad, shift)
    ty = type_of(q4lib, name)
    q4lib.q4_norm_before(H, H.stride(0), ty, None, X, X.stride(0), ty, w, 0.25, EPS, m, d)
    h = unit(f64(X))[0] * (f64(w) + 0.25)
    close(H, h, (128 * E + ROUND[name]) * np.abs(h) + TINY[name])
    assert gaps_kept(H)


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (1, 1)])
def test_norm_before_as_codes(q4lib, m, d, name, pad, shift):
    X, w = rows(values(m, d, name, m + d), name, pad, shift), weights(d, 2)
    if m > 1:
        X[1] = 0.0
    H = torch.full((m * (d + pad) + shift,), 99, dtype=torch.int8, device="cuda")[shift:].view(m, d + pad)[:, :d]
    s = torch.full((m,), -1.0, device="cuda")
    q4lib.q4_norm_before(H, d + pad, q4lib.Q4_TYPE_I8, s, X, X.stride(0), type_of(q4lib, name), w, 0.0, EPS, m, d)
    h = unit(f64(X))[0] * f64(w)
    # a code is the rule's of a value within 128 e: a tie may fall to either side
    amax = np.abs(h).max(axis=1, keepdims=True)
    close(s, amax[:, 0] / 127.0, 130 * E * amax[:, 0] / 127 + 1e-45)
    c = np.divide(h * 127.0, amax, out=np.zeros_like(h), where=amax > 0)
    assert np.abs(f64(H) - c).max() <= 0.5 + 127 * 260 * E


def join_reference(R, B, w, off, g, scale):
    f = scale * g * unit(f64(B))[0] * (f64(w) + off)
    return f64(R) + f, np.abs(f)


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("name,pad,shift", [("f32", 0, 0), ("f32", 1, 1), ("f16", 0, 0), ("bf16", 8, 0), ("bf16", 2, 2), ("bf16", 1, 1)])
@pytest.mark.parametrize("kind", GATES)
def test_norm_after_and_before(q4lib, m, d, name, pad, shift, kind):
    R, B = rows(values(m, d, name, 3), name, pad, shift), rows(values(m, d, name, 4), name, pad, shift)
    w, wn, ty = weights(d, 5), weights(d, 6), type_of(q4lib, name)
    gate, ldg, gk = gate_of(q4lib, kind, m, d, name, 7, pad, shift)
    Y, H, Z = (blank(m, d, name, pad, shift) for _ in range(3))
    ld = Y.stride(0)
    q4lib.q4_norm_after_before(Y, ld, H, ld, ty, None, R, ld, B, ld, ty, w, 0.5, gate, ldg, gk, -0.7, wn, 0.0, EPS, m, d)
    q4lib.q4_norm_after(Z, ld, R, ld, B, ld, ty, w, 0.5, gate, ldg, gk, -0.7, EPS, m, d)
    y, f = join_reference(R, B, w, 0.5, wide(gate, kind), -0.7)
    close(Y, y, 128 * E * f + 2 * E * np.abs(y) + ROUND[name] * np.abs(y) + TINY[name], "y")
    h = unit(f64(Y))[0] * f64(wn)
    close(H, h, (128 * E + ROUND[name]) * np.abs(h) + TINY[name], "h")
    assert torch.equal(Y, Z)
    assert gaps_kept(Y) and gaps_kept(H)


@pytest.mark.parametrize("m,d", [(1, 2560), (40, 640), (300, 1024), (3, 20000)])
def test_join_as_codes_and_in_place(q4lib, m, d):
    R, B, w, wn = values(m, d, "bf16", 8).cuda(), values(m, d, "bf16", 9).cuda(), weights(d, 10), weights(d, 11)
    ty = q4lib.Q4_TYPE_BF16
    Y, H, S = torch.empty_like(R), torch.empty((m, d), dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    H2, S2 = torch.empty_like(H), torch.empty_like(S)
    q4lib.q4_norm_after_before(Y, d, H, d, q4lib.Q4_TYPE_I8, S, R, d, B, d, ty, w, 0.0, None, 0, 0, 1.0, wn, 0.0, EPS, m, d)
    q4lib.q4_norm_before(H2, d, q4lib.Q4_TYPE_I8, S2, Y, d, ty, wn, 0.0, EPS, m, d)
    assert torch.equal(H, H2) and torch.equal(S, S2)          # the two calls' results
    q4lib.q4_norm_after(R, d, R, d, B, d, ty, w, 0.0, None, 0, 0, 1.0, EPS, m, d)
    assert torch.equal(R, Y)
    q4lib.q4_norm_before(Y, d, ty, None, Y, d, ty, None, 0.0, EPS, m, d)
    h = unit(f64(R))[0]
    close(Y, h, (128 * E + ROUND["bf16"]) * np.abs(h) + TINY["bf16"])


def test_zero_and_nonfinite_rows(q4lib):
    m, d = 6, 640
    X = values(m, d, "f32", 12).cuda()
    X[0], X[1, 3], X[2, 5] = 0.0, float("nan"), float("inf")
    H, C, S = torch.empty_like(X), torch.empty((m, d), dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    q4lib.q4_norm_before(H, d, 0, None, X, d, 0, None, 0.0, 1e-30, m, d)
    q4lib.q4_norm_before(C, d, q4lib.Q4_TYPE_I8, S, X, d, 0, None, 0.0, 1e-30, m, d)
    assert bool((H[0] == 0).all()) and bool((C[0] == 0).all()) and float(S[0]) == 0.0
    assert bool(torch.isnan(H[1]).all()) and bool(torch.isnan(S[1])) and bool((C[1] == 0).all())
    assert bool(torch.isnan(H[2, 5])) and bool(torch.isnan(S[2]))
    h = unit(f64(X[3:]), 1e-30)[0]
    close(H[3:], h, 129 * E * np.abs(h) + TINY["f32"])


# ------------------------------------------------------------- gradients --

def workspace(q4lib, m, d):
    n = q4lib.q4_norm_workspace_size(m, d)
    return torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda"), n   # NaN: read nowhere unwritten


def unit_grad(x, dn, eps=EPS):
    u, r = unit(x, eps)
    mean = (dn * u).mean(axis=1, keepdims=True)
    return r * (dn - u * mean), r * (np.abs(dn) + np.abs(u) * np.abs(dn * u).mean(axis=1, keepdims=True)), u


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("name,pad,shift", [("f32", 0, 0), ("f32", 1, 1), ("f16", 0, 0), ("bf16", 8, 0), ("bf16", 2, 2), ("bf16", 1, 1)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_before_backward(q4lib, m, d, name, pad, shift, residual):
    X, dH = rows(values(m, d, name, 13, 1.0), name, pad, shift), rows(values(m, d, name, 14, 0.5), name, pad, shift)
    dR = rows(values(m, d, name, 15, 0.5), name, pad, shift) if residual else None
    w, dw, dX, ty = weights(d, 16), torch.empty(d, device="cuda"), blank(m, d, name, pad, shift), type_of(q4lib, name)
    ws, wsb = workspace(q4lib, m, d)
    ld = X.stride(0)
    q4lib.q4_norm_before_backward(dX, ld, dw, dH, ld, dR, ld if residual else 0, X, ld, ty, w, -0.5, EPS, m, d, ws, wsb)
    dn = f64(dH) * (f64(w) - 0.5)
    dx, size, u = unit_grad(f64(X), dn)
    dr = f64(dR) if residual else 0.0
    close(dX, dx + dr, 256 * E * size + 2 * E * np.abs(dr) + ROUND[name] * np.abs(dx + dr) + TINY[name], "dx")
    t = f64(dH) * u
    close(dw, t.sum(axis=0), (192 + m / 16) * E * np.abs(t).sum(axis=0) + 1e-30, "dw")
    assert gaps_kept(dX)


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("name,pad,shift", [("f32", 0, 0), ("f32", 1, 1), ("f16", 0, 0), ("bf16", 8, 0), ("bf16", 1, 1)])
@pytest.mark.parametrize("kind", GATES)
def test_norm_after_backward(q4lib, m, d, name, pad, shift, kind):
    B, dY = rows(values(m, d, name, 17, 1.0), name, pad, shift), rows(values(m, d, name, 18, 0.5), name, pad, shift)
    w, dw, dB, ty = weights(d, 19), torch.empty(d, device="cuda"), blank(m, d, name, pad, shift), type_of(q4lib, name)
    gate, ldg, gk = gate_of(q4lib, kind, m, d, name, 20, pad, shift)
    dg = None if kind == "none" else blank(m, d, name, pad, shift) if kind == "full" else torch.full_like(gate, float("nan"))
    ws, wsb = workspace(q4lib, m, d)
    ld, s = B.stride(0), 1.3
    q4lib.q4_norm_after_backward(dB, ld, dw, dg, ld if kind == "full" else 0, dY, ld, B, ld, ty, w, 0.25, gate, ldg, gk, s,
                                 EPS, m, d, ws, wsb)
    s = float(np.float32(s))
    g, dy, wo = wide(gate, kind), f64(dY), f64(w) + 0.25
    db, size, u = unit_grad(f64(B), s * g * dy * wo)
    close(dB, db, 256 * E * size + ROUND[name] * np.abs(db) + TINY[name], "db")
    t = s * g * dy * u
    chain = 192 + m / 16
    close(dw, t.sum(axis=0), chain * E * np.abs(t).sum(axis=0) + 1e-30, "dw")
    t = s * dy * u * wo
    if kind == "channel":
        close(dg, t.sum(axis=0), chain * E * np.abs(t).sum(axis=0) + 1e-30, "dgate")
    elif kind == "token":
        close(dg, t.sum(axis=1), 384 * E * np.abs(t).sum(axis=1) + 1e-30, "dgate")
    elif kind == "full":
        close(dg, t, (160 * E + ROUND[name]) * np.abs(t) + TINY[name], "dgate")
    assert gaps_kept(dB)


@pytest.mark.parametrize("kind", GATES)
def test_gradients_against_differences(q4lib, kind):
    # L = sum of c * H + e * Y over one join; central differences in 64 bits
    # along a random direction of every input, h = 1e-5: relative error of the
    # differences below 1e-7, of the fp32 gradients below 1e-4 of the terms
    m, d, s = 5, 96, 0.8
    rng = np.random.default_rng(21)
    R, B, c, e = (rng.standard_normal((m, d)) for _ in range(4))
    w, wn = 1 + 0.2 * rng.standard_normal(d), 1 + 0.2 * rng.standard_normal(d)
    gshape = {"none": (1, 1), "channel": (1, d), "token": (m, 1), "full": (m, d)}[kind]
    g = np.ones(gshape) if kind == "none" else rng.standard_normal(gshape)
    R, B, c, e, w, wn, g = (np.asarray(np.float32(v), np.float64) for v in (R, B, c, e, w, wn, g))

    def loss(R, B, w, wn, g):
        y = R + s * g * unit(B)[0] * w
        return (c * unit(y)[0] * wn).sum() + (e * y).sum()

    dev = lambda v: torch.as_tensor(np.ascontiguousarray(v), dtype=torch.float32).cuda()   # noqa: E731
    Rd, Bd, wd, wnd, cd, ed = map(dev, (R, B, w, wn, c, e))
    gk = {"none": 0, "channel": 1, "token": 2, "full": 3}[kind]
    gd = None if kind == "none" else dev(g)
    Y, H, dYt, dB = (torch.empty((m, d), device="cuda") for _ in range(4))
    dwn, dw = (torch.empty(d, device="cuda") for _ in range(2))
    dg = None if kind == "none" else torch.empty_like(gd)
    ws, wsb = workspace(q4lib, m, d)
    q4lib.q4_norm_after_before(Y, d, H, d, 0, None, Rd, d, Bd, d, 0, wd, 0.0, gd, d, gk, s, wnd, 0.0, EPS, m, d)
    q4lib.q4_norm_before_backward(dYt, d, dwn, cd, d, ed, d, Y, d, 0, wnd, 0.0, EPS, m, d, ws, wsb)
    q4lib.q4_norm_after_backward(dB, d, dw, dg, d, dYt, d, Bd, d, 0, wd, 0.0, gd, d, gk, s, EPS, m, d, ws, wsb)
    args = [R, B, w, wn, g]
    grads = [f64(dYt), f64(dB), f64(dw), f64(dwn), None if kind == "none" else f64(dg).reshape(gshape)]
    for i, grad in enumerate(grads):
        if grad is None:
            continue
        v = rng.standard_normal(args[i].shape)
        step = 1e-5
        up, down = ([a + k * step * v if j == i else a for j, a in enumerate(args)] for k in (1, -1))
        diff = (loss(*up) - loss(*down)) / (2 * step)
        assert abs((grad * v).sum() - diff) <= 1e-4 * np.abs(grad * v).sum()


def test_gradients_in_place_and_unwanted(q4lib):
    m, d = 37, 512
    X, dH, dR, w = values(m, d, "f32", 22).cuda(), values(m, d, "f32", 23).cuda(), values(m, d, "f32", 24).cuda(), weights(d, 25)
    ws, wsb = workspace(q4lib, m, d)
    dX, dw = torch.empty_like(X), torch.empty(d, device="cuda")
    q4lib.q4_norm_before_backward(dX, d, dw, dH, d, dR, d, X, d, 0, w, 0.0, EPS, m, d, ws, wsb)
    for over in (dH, dR):
        o = over.clone()
        a = [o if over is dH else dH, o if over is dR else dR]
        q4lib.q4_norm_before_backward(o, d, None, a[0], d, a[1], d, X, d, 0, w, 0.0, EPS, m, d, None, 0)
        assert torch.equal(o, dX)
    dB = torch.empty_like(X)
    q4lib.q4_norm_after_backward(dB, d, None, None, 0, dH, d, X, d, 0, w, 0.0, None, 0, 0, 1.0, EPS, m, d, None, 0)
    o = dH.clone()
    q4lib.q4_norm_after_backward(o, d, dw, None, 0, o, d, X, d, 0, w, 0.0, None, 0, 0, 1.0, EPS, m, d, ws, wsb)
    assert torch.equal(o, dB)


@pytest.mark.parametrize("m,d", [(700, 640), (1, 4096), (5000, 96)])
def test_same_bits_each_run_and_on_another_stream(q4lib, m, d):
    B, dY, w, g = values(m, d, "bf16", 26).cuda(), values(m, d, "bf16", 27).cuda(), weights(d, 28), weights(d, 29)
    ws, wsb = workspace(q4lib, m, d)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for stream in (None, s, s):
        dB, dw, dg = torch.empty_like(B), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
        torch.cuda.synchronize()
        q4lib.q4_norm_after_backward(dB, d, dw, dg, 0, dY, d, B, d, 2, w, 0.0, g, 0, 1, 1.0, EPS, m, d, ws, wsb, stream=stream)
        torch.cuda.synchronize()
        got.append((dB, dw, dg))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


def test_no_rows(q4lib):
    d = 64
    x = torch.full((1, d), 3.0, device="cuda")
    dw, dg, w = torch.full((d,), 3.0, device="cuda"), torch.full((d,), 3.0, device="cuda"), weights(d, 30)
    q4lib.q4_norm_before(x, d, 0, None, x, d, 0, w, 0.0, EPS, 0, d)
    q4lib.q4_norm_after_before(x, d, x, d, 0, None, x, d, x, d, 0, w, 0.0, None, 0, 0, 1.0, w, 0.0, EPS, 0, d)
    q4lib.q4_norm_before_backward(x, d, dw, x, d, None, 0, x, d, 0, w, 0.0, EPS, 0, d, None, 0)
    assert bool((x == 3.0).all()) and bool((dw == 0).all())
    dw.fill_(3.0)
    q4lib.q4_norm_after_backward(x, d, dw, dg, 0, x, d, x, d, 0, w, 0.0, w, 0, 1, 1.0, EPS, 0, d, None, 0)
    assert bool((dw == 0).all()) and bool((dg == 0).all())
