"""The norms and their gradients over so many rows that each CTA goes round its
ring of rows several times: values, codes, weights of 1, and results written over
an input. The formulas and tolerances are test_gpu_norm.py's, in 64 bits on the
device."""

import pytest

from block_testlib import ROUND, TINY, blank, close, gaps_kept, rows, type_of
from test_gpu_norm import E, EPS, workspace

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


# one, two and four vectors a thread, rows of 512 threads; then odd boundaries.
# At least six rows a CTA, of which three to six are in the ring.
CASES = [(9001, 1024, "bf16", 0, 0), (7000, 520, "f32", 0, 0), (4300, 4096, "bf16", 0, 0), (3000, 2560, "f32", 8, 0),
         (1000, 16384, "bf16", 0, 0), (2100, 6000, "f16", 0, 0), (6000, 1031, "bf16", 1, 3), (3000, 2561, "f32", 0, 1),
         (3001, 4097, "f16", 0, 1)]


def values(m, d, seed, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(m, d, generator=g, device="cuda") * torch.exp(spread * (2 * torch.rand(m, 1, generator=g, device="cuda") - 1))


def weights(d, seed):
    return 1.0 + 0.3 * torch.randn(d, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def unit(x):
    r = 1.0 / (x.pow(2).mean(dim=1, keepdim=True) + EPS).sqrt()
    return x * r, r


def held(y, ref, tol, what):
    """close() of a reference on the device."""
    return close(y, ref.cpu().numpy(), tol.cpu().numpy(), what)


def gate_of(q4lib, kind, m, d, name, pad, shift):
    if kind == "none":
        return None, 0, q4lib.Q4_GATE_NONE, 1.0
    if kind == "channel":
        g = weights(d, 40)
        return g, 0, q4lib.Q4_GATE_CHANNEL, g.double()
    if kind == "token":
        g = weights(m, 41)
        return g, 0, q4lib.Q4_GATE_TOKEN, g.double()[:, None]
    g = rows(values(m, d, 42), name, pad, shift)
    return g, g.stride(0), q4lib.Q4_GATE_FULL, g.double()


@pytest.mark.parametrize("m,d,name,pad,shift", CASES)
@pytest.mark.parametrize("kind", ["none", "token", "full"])
@pytest.mark.parametrize("weighted", [True, False])
def test_join(q4lib, m, d, name, pad, shift, kind, weighted):
    ty = type_of(q4lib, name)
    R, B = rows(values(m, d, 1), name, pad, shift), rows(values(m, d, 2), name, pad, shift)
    gate, ldg, gk, g64 = gate_of(q4lib, kind, m, d, name, pad, shift)
    w, wn = (weights(d, 3), weights(d, 4)) if weighted else (None, None)
    w64, wn64 = (w.double() + 0.5, wn.double()) if weighted else (1.0, 1.0)
    Y, H = blank(m, d, name, pad, shift), blank(m, d, name, pad, shift)
    ld = Y.stride(0)
    q4lib.q4_norm_after_before(Y, ld, H, ld, ty, None, R, ld, B, ld, ty, w, 0.5, gate, ldg, gk, -0.7, wn, 0.0, EPS, m, d)
    f = -0.7 * g64 * unit(B.double())[0] * w64
    y = R.double() + f
    held(Y, y, 128 * E * f.abs() + (2 * E + ROUND[name]) * y.abs() + TINY[name], "y")
    h = unit(Y.double())[0] * wn64
    held(H, h, (128 * E + ROUND[name]) * h.abs() + TINY[name], "h")
    assert gaps_kept(Y) and gaps_kept(H)
    # the stream's results over the stream
    Z = blank(m, d, name, pad, shift)
    q4lib.q4_norm_after_before(R, ld, Z, ld, ty, None, R, ld, B, ld, ty, w, 0.5, gate, ldg, gk, -0.7, wn, 0.0, EPS, m, d)
    assert torch.equal(R, Y) and torch.equal(Z, H)


@pytest.mark.parametrize("m,d,name,pad,shift", CASES)
@pytest.mark.parametrize("kind", ["channel", "full"])
@pytest.mark.parametrize("gap,byte", [(0, 0), (3, 1)])
def test_join_as_codes(q4lib, m, d, name, pad, shift, kind, gap, byte):
    ty = type_of(q4lib, name)
    R, B = rows(values(m, d, 5), name, pad, shift), rows(values(m, d, 6), name, pad, shift)
    gate, ldg, gk, g64 = gate_of(q4lib, kind, m, d, name, pad, shift)
    w, wn = weights(d, 7), weights(d, 8)
    R[1] = 0.0
    B[1] = 0.0
    Y, S = blank(m, d, name, pad, shift), torch.full((m,), -1.0, device="cuda")
    codes = torch.full((m * (d + gap) + byte,), 99, dtype=torch.int8, device="cuda")
    H = codes[byte:].view(m, d + gap)
    ld = Y.stride(0)
    q4lib.q4_norm_after_before(Y, ld, H, d + gap, q4lib.Q4_TYPE_I8, S, R, ld, B, ld, ty, w, 0.0, gate, ldg, gk, 0.9, wn, 0.0, EPS, m, d)
    f = 0.9 * g64 * unit(B.double())[0] * w.double()
    y = R.double() + f
    held(Y, y, 128 * E * f.abs() + (2 * E + ROUND[name]) * y.abs() + TINY[name], "y")
    h = unit(Y.double())[0] * wn.double()
    amax = h.abs().amax(dim=1, keepdim=True)
    held(S, amax[:, 0] / 127, 130 * E * amax[:, 0] / 127 + 1e-45, "scales")
    c = torch.where(amax > 0, h * 127 / amax, torch.zeros_like(h))
    assert float((H[:, :d].double() - c).abs().max()) <= 0.5 + 127 * 260 * E
    assert bool((H[:, d:] == 99).all()) and bool((codes[:byte] == 99).all())
    # what q4_norm_before makes of the same Y: a row's squares may add in another order
    H2, S2 = torch.empty((m, d), dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    q4lib.q4_norm_before(H2, d, q4lib.Q4_TYPE_I8, S2, Y, ld, ty, wn, 0.0, EPS, m, d)
    held(S2, S.double(), 260 * E * S.double() + 1e-45, "scales of both calls")
    assert float((H2.double() - H[:, :d].double()).abs().max()) <= 1.0


@pytest.mark.parametrize("m,d,name,pad,shift", CASES)
@pytest.mark.parametrize("residual,weighted", [(False, True), (True, True), (True, False)])
def test_before_backward(q4lib, m, d, name, pad, shift, residual, weighted):
    ty = type_of(q4lib, name)
    X, dH, dR = (rows(values(m, d, s, 0.5), name, pad, shift) for s in (9, 10, 11))
    w, w64 = (weights(d, 12), weights(d, 12).double() - 0.5) if weighted else (None, 1.0)
    ws, wsb = workspace(q4lib, m, d)
    ld = X.stride(0)

    def call(out, dH, dR, X, dw):
        q4lib.q4_norm_before_backward(out, ld, dw, dH, ld, dR if residual else None, ld if residual else 0, X, ld, ty, w, -0.5,
                                      EPS, m, d, ws, wsb)

    dX, dw = blank(m, d, name, pad, shift), torch.empty(d, device="cuda")
    call(dX, dH, dR, X, dw)
    x, dn = X.double(), dH.double() * w64
    u, r = unit(x)
    mean = (dn * u).mean(dim=1, keepdim=True)
    size = r * (dn.abs() + u.abs() * (dn * u).abs().mean(dim=1, keepdim=True))
    dr = dR.double() if residual else torch.zeros_like(x)
    dx = r * (dn - u * mean) + dr
    held(dX, dx, 256 * E * size + 2 * E * dr.abs() + ROUND[name] * dx.abs() + TINY[name], "dx")
    t = dH.double() * u
    held(dw, t.sum(dim=0), (192 + m / 16) * E * t.abs().sum(dim=0) + 1e-30, "dw")
    assert gaps_kept(dX)
    for over in ([0, 1, 2] if residual else [0, 2]):
        a, dw2 = [rows(v, name, pad, shift) for v in (dH, dR, X)], torch.empty_like(dw)
        call(a[over], *a, dw2)
        assert torch.equal(a[over], dX) and torch.equal(dw2, dw)


@pytest.mark.parametrize("m,d,name,pad,shift", CASES)
@pytest.mark.parametrize("kind", ["none", "channel", "token", "full"])
def test_after_backward(q4lib, m, d, name, pad, shift, kind):
    ty, s = type_of(q4lib, name), 1.5
    B, dY = (rows(values(m, d, v, 0.5), name, pad, shift) for v in (13, 14))
    gate, ldg, gk, g64 = gate_of(q4lib, kind, m, d, name, pad, shift)
    w = weights(d, 15) if kind != "token" else None
    w64 = w.double() + 0.25 if w is not None else 1.0
    ws, wsb = workspace(q4lib, m, d)
    ld = B.stride(0)

    def call(out, dY, B, dw, dg):
        q4lib.q4_norm_after_backward(out, ld, dw, dg, ld if kind == "full" else 0, dY, ld, B, ld, ty, w, 0.25, gate, ldg, gk, s, EPS,
                                     m, d, ws, wsb)

    dB, dw = blank(m, d, name, pad, shift), torch.empty(d, device="cuda")
    dg = None if kind == "none" else blank(m, d, name, pad, shift) if kind == "full" else torch.full_like(gate, float("nan"))
    call(dB, dY, B, dw, dg)
    dn = s * g64 * dY.double() * w64
    u, r = unit(B.double())
    size = r * (dn.abs() + u.abs() * (dn * u).abs().mean(dim=1, keepdim=True))
    db = r * (dn - u * (dn * u).mean(dim=1, keepdim=True))
    held(dB, db, 256 * E * size + ROUND[name] * db.abs() + TINY[name], "db")
    chain, t = 192 + m / 16, s * g64 * dY.double() * u
    held(dw, t.sum(dim=0), chain * E * t.abs().sum(dim=0) + 1e-30, "dw")
    t = s * dY.double() * u * w64
    if kind == "channel":
        held(dg, t.sum(dim=0), chain * E * t.abs().sum(dim=0) + 1e-30, "dgate")
    elif kind == "token":
        held(dg, t.sum(dim=1), 384 * E * t.abs().sum(dim=1) + 1e-30, "dgate")
    elif kind == "full":
        held(dg, t, (160 * E + ROUND[name]) * t.abs() + TINY[name], "dgate")
    assert gaps_kept(dB)
    for over in (0, 1):
        a, dw2 = [rows(v, name, pad, shift) for v in (dY, B)], torch.empty_like(dw)
        dg2 = None if dg is None else blank(m, d, name, pad, shift) if kind == "full" else torch.empty_like(dg)
        call(a[over], *a, dw2, dg2)
        assert torch.equal(a[over], dB) and torch.equal(dw2, dw)
        assert dg is None or torch.equal(dg2, dg)
