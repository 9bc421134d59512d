"""The norms and their gradients over rows that start at no 16-byte boundary:
many rows a CTA, NaN between the rows and in neighbouring ones, matrices whose
rows start unlike one another, parameters and codes aligned to their elements
alone. The formulas and tolerances are test_gpu_norm.py's."""

import numpy as np
import pytest

from block_testlib import ROUND, TINY, blank, close, f64, rows, type_of
from test_gpu_norm import E, EPS, GATES, gate_of, join_reference, unit, unit_grad, values, weights, wide, workspace

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def nan_between(v):
    """NaN in the gaps between the rows of an input."""
    m, d = v.shape
    if m > 1 and v.stride(0) > d:
        torch.as_strided(v, (m - 1, v.stride(0) - d), (v.stride(0), 1), v.storage_offset() + d).fill_(float("nan"))
    return v


def odd_params(w):
    """The same parameters, 4 bytes into a buffer, NaN around them."""
    buf = torch.full((w.numel() + 2,), float("nan"), device="cuda")
    buf[1:-1].copy_(w)
    return buf[1:-1]


# rows a warp, a CTA and a ring each, several a CTA; in the types' largest
# vectors, short of one and past one
SIZES = [(5000, 131), (700, 1031), (2500, 1030), (613, 4097), (40, 4099), (330, 8209), (2, 17001)]
LAYOUTS = [("f32", 0, 0), ("f32", 1, 3), ("f16", 3, 1), ("bf16", 0, 5), ("bf16", 1, 0)]


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("name,pad,shift", LAYOUTS)
@pytest.mark.parametrize("kind", ["channel", "full"])
def test_join(q4lib, m, d, name, pad, shift, kind):
    R, B = (nan_between(rows(values(m, d, name, s), name, pad, shift)) for s in (3, 4))
    B[m // 2], R[1 if m > 1 else 0, 0] = float("nan"), float("inf")
    w, wn, ty = odd_params(weights(d, 5)), odd_params(weights(d, 6)), type_of(q4lib, name)
    gate, ldg, gk = gate_of(q4lib, kind, m, d, name, 7, pad, shift)
    if kind == "channel":
        gate = odd_params(gate)
    Y, H = blank(m, d, name, pad, shift), blank(m, d, name, pad, shift)
    ld = Y.stride(0)
    q4lib.q4_norm_after_before(Y, ld, H, ld, ty, None, R, ld, B, ld, ty, w, 0.5, gate, ldg, gk, -0.7, wn, 0.0, EPS, m, d)
    y, f = join_reference(R, B, w, 0.5, wide(gate, kind), -0.7)
    close(Y, y, 128 * E * f + 2 * E * np.abs(y) + ROUND[name] * np.abs(y) + TINY[name], "y")
    ok = np.isfinite(f64(Y)).all(axis=1)
    h = unit(f64(Y)[ok])[0] * f64(wn)
    close(f64(H)[ok], h, (128 * E + ROUND[name]) * np.abs(h) + TINY[name], "h")
    assert np.isnan(f64(H)[m // 2]).all()


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("gap", [0, 3])
def test_codes_at_any_byte(q4lib, m, d, name, gap):
    # aligned values where d is a multiple of 16 bytes' worth, codes never
    for width in (d, (d + 7) // 8 * 8):
        X, w = rows(values(m, width, name, m), name), weights(width, 2)
        ld = width + gap
        H = torch.full((m * ld + 1,), 99, dtype=torch.int8, device="cuda")
        h8 = H[1:].view(m, ld)
        s, v = torch.empty(m, device="cuda"), blank(m, width, name)
        q4lib.q4_norm_before(h8, ld, q4lib.Q4_TYPE_I8, s, X, width, type_of(q4lib, name), w, 0.0, EPS, m, width)
        h = unit(f64(X))[0] * f64(w)
        amax = np.abs(h).max(axis=1, keepdims=True)
        close(s, amax[:, 0] / 127.0, 130 * E * amax[:, 0] / 127 + 1e-45)
        assert np.abs(f64(h8[:, :width]) - h * 127.0 / amax).max() <= 0.5 + 127 * 260 * E
        assert int(H[0]) == 99 and bool((h8[:, width:] == 99).all())
        q4lib.q4_norm_before(v, width, type_of(q4lib, name), None, X, width, type_of(q4lib, name), w, 0.0, EPS, m, width)
        close(v, h, (128 * E + ROUND[name]) * np.abs(h) + TINY[name])


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("name,pad,shift", LAYOUTS)
@pytest.mark.parametrize("residual", [False, True])
def test_before_backward(q4lib, m, d, name, pad, shift, residual):
    X, dH, dR = (nan_between(rows(values(m, d, name, s, 0.5), name, pad, shift)) for s in (13, 14, 15))
    w, dw, dX, ty = odd_params(weights(d, 16)), torch.empty(d, device="cuda"), blank(m, d, name, pad, shift), type_of(q4lib, name)
    ws, wsb = workspace(q4lib, m, d)
    ld = X.stride(0)
    q4lib.q4_norm_before_backward(dX, ld, dw, dH, ld, dR if residual else None, ld if residual else 0, X, ld, ty, w, -0.5, EPS,
                                  m, d, ws, wsb)
    dx, size, u = unit_grad(f64(X), f64(dH) * (f64(w) - 0.5))
    dr = f64(dR) if residual else 0.0
    close(dX, dx + dr, 256 * E * size + 2 * E * np.abs(dr) + ROUND[name] * np.abs(dx + dr) + TINY[name], "dx")
    t = f64(dH) * u
    close(dw, t.sum(axis=0), (192 + m / 16) * E * np.abs(t).sum(axis=0) + 1e-30, "dw")


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("name,pad,shift", LAYOUTS)
@pytest.mark.parametrize("kind", GATES)
def test_after_backward(q4lib, m, d, name, pad, shift, kind):
    B, dY = (nan_between(rows(values(m, d, name, s, 0.5), name, pad, shift)) for s in (17, 18))
    w, dw, dB, ty = odd_params(weights(d, 19)), torch.empty(d, device="cuda"), blank(m, d, name, pad, shift), type_of(q4lib, name)
    gate, ldg, gk = gate_of(q4lib, kind, m, d, name, 20, pad, shift)
    dg = None if kind == "none" else blank(m, d, name, pad, shift) if kind == "full" else torch.full_like(gate, float("nan"))
    ws, wsb = workspace(q4lib, m, d)
    ld = B.stride(0)
    q4lib.q4_norm_after_backward(dB, ld, dw, dg, ld if kind == "full" else 0, dY, ld, B, ld, ty, w, 0.25, gate, ldg, gk, 1.5,
                                 EPS, m, d, ws, wsb)
    g, dy, wo = wide(gate, kind), f64(dY), f64(w) + 0.25
    db, size, u = unit_grad(f64(B), 1.5 * g * dy * wo)
    close(dB, db, 256 * E * size + ROUND[name] * np.abs(db) + TINY[name], "db")
    chain, t = 192 + m / 16, 1.5 * g * dy * u
    close(dw, t.sum(axis=0), chain * E * np.abs(t).sum(axis=0) + 1e-30, "dw")
    t = 1.5 * dy * u * wo
    if kind == "channel":
        close(dg, t.sum(axis=0), chain * E * np.abs(t).sum(axis=0) + 1e-30, "dgate")
    elif kind == "token":
        close(dg, t.sum(axis=1), 384 * E * np.abs(t).sum(axis=1) + 1e-30, "dgate")
    elif kind == "full":
        close(dg, t, (160 * E + ROUND[name]) * np.abs(t) + TINY[name], "dgate")


@pytest.mark.parametrize("m,d", [(700, 1031), (3, 257), (400, 96), (2, 9000)])
@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
def test_rows_that_start_unlike(q4lib, m, d, name):
    ty, w = type_of(q4lib, name), weights(d, 30)
    X, dH, dX = rows(values(m, d, name, 31, 0.5), name, 1, 0), rows(values(m, d, name, 32, 0.5), name, 0, 1), blank(m, d, name, 3, 2)
    H, dw = blank(m, d, name, 2, 1), torch.empty(d, device="cuda")
    q4lib.q4_norm_before(H, H.stride(0), ty, None, X, X.stride(0), ty, w, 0.0, EPS, m, d)
    h = unit(f64(X))[0] * f64(w)
    close(H, h, (128 * E + ROUND[name]) * np.abs(h) + TINY[name])
    ws, wsb = workspace(q4lib, m, d)
    q4lib.q4_norm_before_backward(dX, dX.stride(0), dw, dH, dH.stride(0), None, 0, X, X.stride(0), ty, w, 0.0, EPS, m, d, ws, wsb)
    dx, size, u = unit_grad(f64(X), f64(dH) * f64(w))
    close(dX, dx, 256 * E * size + ROUND[name] * np.abs(dx) + TINY[name])
    t = f64(dH) * u
    close(dw, t.sum(axis=0), (192 + m / 16) * E * np.abs(t).sum(axis=0) + 1e-30)
