"""What the calls around the linear layers refuse, and their size functions: all
on the host, before any device work (no GPU is needed; addresses are made up)."""

import pytest

A = 0x100000          # 256-byte aligned
F32, F16, BF16, I8 = 0, 1, 2, 3
INVALID, ALIGN, WORKSPACE = 1, 2, 6
BIG = 1 << 40


def refuse(q4lib, name, args, code):
    assert getattr(q4lib, name)(*args, stream=0, check=False) == code


def change(good, **at):
    args = list(good)
    for k, v in at.items():
        args[int(k[1:])] = v
    return args


QUANT = [A, A, A, 64, F32, 2, 64]   # Xq, sx, X, ldx, type, m, k


@pytest.mark.parametrize("at,code", [
    (dict(_0=0), INVALID), (dict(_1=0), INVALID), (dict(_2=0), INVALID), (dict(_3=63), INVALID), (dict(_4=I8), INVALID),
    (dict(_4=7), INVALID), (dict(_5=-1), INVALID), (dict(_6=0), INVALID), (dict(_6=(1 << 24) + 1, _3=BIG), INVALID),
    (dict(_1=A + 2), ALIGN), (dict(_2=A + 2), ALIGN), (dict(_2=A + 1, _4=BF16), ALIGN),
])
def test_token_coding(q4lib, at, code):
    refuse(q4lib, "q4_a8_quantize", change(QUANT, **at), code)


MATMUL = [A, A, 64, F32, A, 96, F32, 2, 64, 96, A, BIG]   # W, X, ldx, xtype, Y, ldy, ytype, m, k, n, ws, bytes


@pytest.mark.parametrize("at,code", [
    (dict(_0=0), INVALID), (dict(_1=0), INVALID), (dict(_4=0), INVALID), (dict(_2=63), INVALID), (dict(_5=95), INVALID),
    (dict(_3=I8), INVALID), (dict(_6=I8), INVALID), (dict(_6=-1), INVALID), (dict(_7=-1), INVALID),
    (dict(_8=48), INVALID), (dict(_8=0), INVALID), (dict(_8=131072 + 32, _2=BIG), INVALID), (dict(_9=0), INVALID),
    (dict(_0=A + 8), ALIGN), (dict(_1=A + 2), ALIGN), (dict(_4=A + 2), ALIGN), (dict(_4=A + 1, _6=F16), ALIGN),
    (dict(_10=A + 128), ALIGN), (dict(_10=0), WORKSPACE), (dict(_11=10), WORKSPACE),
])
def test_int8_product(q4lib, at, code):
    refuse(q4lib, "q4_w8a8_matmul", change(MATMUL, **at), code)


CODES = [A, A, A, A, 96, F32, 2, 64, 96, A, BIG]   # W, Xq, sx, Y, ldy, ytype, m, k, n, ws, bytes


@pytest.mark.parametrize("at,code", [
    (dict(_0=0), INVALID), (dict(_1=0), INVALID), (dict(_2=0), INVALID), (dict(_3=0), INVALID), (dict(_4=95), INVALID),
    (dict(_5=I8), INVALID), (dict(_6=-1), INVALID), (dict(_7=40), INVALID), (dict(_8=0), INVALID),
    (dict(_0=A + 4), ALIGN), (dict(_1=A + 4), ALIGN), (dict(_2=A + 2), ALIGN), (dict(_3=A + 2), ALIGN),
    (dict(_9=A + 16), ALIGN), (dict(_9=0), WORKSPACE), (dict(_10=0), WORKSPACE),
])
def test_int8_product_of_codes(q4lib, at, code):
    refuse(q4lib, "q4_w8a8_matmul_codes", change(CODES, **at), code)


BEFORE = [A, 64, F32, 0, A, 64, F32, A, 0.0, 1e-6, 2, 64]   # H, ldh, htype, h_scale, X, ldx, type, w, off, eps, m, d


@pytest.mark.parametrize("at,code", [
    (dict(_0=0), INVALID), (dict(_4=0), INVALID), (dict(_1=63), INVALID), (dict(_5=63), INVALID), (dict(_2=F16), INVALID),
    (dict(_6=I8, _2=I8), INVALID), (dict(_2=I8), INVALID), (dict(_9=0.0), INVALID), (dict(_9=-1.0), INVALID),
    (dict(_9=float("inf")), INVALID), (dict(_9=float("nan")), INVALID), (dict(_10=-1), INVALID), (dict(_11=0), INVALID),
    (dict(_0=A + 2), ALIGN), (dict(_4=A + 2), ALIGN), (dict(_7=A + 2), ALIGN), (dict(_2=I8, _3=A + 2), ALIGN),
])
def test_norm_before(q4lib, at, code):
    refuse(q4lib, "q4_norm_before", change(BEFORE, **at), code)


# Y, ldy, R, ldr, B, ldb, type, w, off, gate, ldg, kind, scale, eps, m, d
AFTER = [A, 64, A, 64, A, 64, F32, A, 0.0, 0, 0, 0, 1.0, 1e-6, 2, 64]


@pytest.mark.parametrize("at,code", [
    (dict(_0=0), INVALID), (dict(_2=0), INVALID), (dict(_4=0), INVALID), (dict(_1=63), INVALID), (dict(_3=63), INVALID),
    (dict(_5=63), INVALID), (dict(_6=I8), INVALID), (dict(_11=4), INVALID), (dict(_11=-1), INVALID), (dict(_11=1), INVALID),
    (dict(_11=3, _9=A, _10=63), INVALID), (dict(_13=0.0), INVALID), (dict(_14=-1), INVALID), (dict(_15=0), INVALID),
    (dict(_11=1, _9=A + 2), ALIGN), (dict(_11=2, _9=A + 2), ALIGN), (dict(_11=3, _9=A + 2, _10=64), ALIGN), (dict(_0=A + 1), ALIGN),
])
def test_norm_after(q4lib, at, code):
    refuse(q4lib, "q4_norm_after", change(AFTER, **at), code)


# Y, ldy, H, ldh, htype, h_scale, R, ldr, B, ldb, type, w, off, gate, ldg, kind, scale, w_next, off, eps, m, d
JOIN = [A, 64, A, 64, F32, 0, A, 64, A, 64, F32, A, 0.0, 0, 0, 0, 1.0, A, 0.0, 1e-6, 2, 64]


@pytest.mark.parametrize("at,code", [
    (dict(_2=0), INVALID), (dict(_3=63), INVALID), (dict(_4=BF16), INVALID), (dict(_4=I8), INVALID), (dict(_21=0), INVALID),
    (dict(_17=A + 2), ALIGN), (dict(_4=I8, _5=A + 1), ALIGN),
])
def test_norm_after_before(q4lib, at, code):
    refuse(q4lib, "q4_norm_after_before", change(JOIN, **at), code)


# dX, lddx, dw, dH, lddh, dR, lddr, X, ldx, type, w, off, eps, m, d, ws, bytes
BEFORE_BWD = [A, 64, A, A, 64, A, 64, A, 64, F32, A, 0.0, 1e-6, 2, 64, A, BIG]


@pytest.mark.parametrize("at,code", [
    (dict(_0=0), INVALID), (dict(_3=0), INVALID), (dict(_7=0), INVALID), (dict(_1=63), INVALID), (dict(_4=63), INVALID),
    (dict(_6=63), INVALID), (dict(_8=63), INVALID), (dict(_9=I8), INVALID), (dict(_12=0.0), INVALID), (dict(_13=-1), INVALID),
    (dict(_2=A + 2), ALIGN), (dict(_5=A + 2), ALIGN), (dict(_15=A + 4), ALIGN), (dict(_15=0), WORKSPACE),
    (dict(_16=2 * 64 * 4 - 1), WORKSPACE),
])
def test_norm_before_backward(q4lib, at, code):
    refuse(q4lib, "q4_norm_before_backward", change(BEFORE_BWD, **at), code)


# dB, lddb, dw, dgate, lddgate, dY, lddy, B, ldb, type, w, off, gate, ldg, kind, scale, eps, m, d, ws, bytes
AFTER_BWD = [A, 64, A, A, 0, A, 64, A, 64, F32, A, 0.0, A, 0, 1, 1.0, 1e-6, 2, 64, A, BIG]


@pytest.mark.parametrize("at,code", [
    (dict(_0=0), INVALID), (dict(_5=0), INVALID), (dict(_7=0), INVALID), (dict(_1=63), INVALID), (dict(_14=9), INVALID),
    (dict(_12=0), INVALID), (dict(_14=0), INVALID), (dict(_14=3, _13=64), INVALID), (dict(_3=A + 2), ALIGN),
    (dict(_12=A + 2), ALIGN), (dict(_19=0), WORKSPACE), (dict(_2=0, _20=1), WORKSPACE), (dict(_16=-1.0), INVALID),
])
def test_norm_after_backward(q4lib, at, code):
    refuse(q4lib, "q4_norm_after_backward", change(AFTER_BWD, **at), code)


# Xs, ldxs, offsets, row_of, pair_of, ids, id_bytes, X, ldx, type, tokens, top_k, experts, d, ws, bytes
DISPATCH = [A, 64, A, A, A, A, 8, A, 64, F32, 20000, 2, 8, 64, A, BIG]


@pytest.mark.parametrize("at,code", [
    (dict(_0=0), INVALID), (dict(_7=0), INVALID), (dict(_2=0), INVALID), (dict(_3=0), INVALID), (dict(_5=0), INVALID),
    (dict(_6=2), INVALID), (dict(_1=63), INVALID), (dict(_8=63), INVALID), (dict(_9=I8), INVALID), (dict(_10=-1), INVALID),
    (dict(_11=0), INVALID), (dict(_11=1025), INVALID), (dict(_10=1 << 24), INVALID), (dict(_12=0), INVALID),
    (dict(_12=4097), INVALID), (dict(_13=0), INVALID), (dict(_2=A + 4), ALIGN), (dict(_3=A + 2), ALIGN), (dict(_4=A + 2), ALIGN),
    (dict(_5=A + 4), ALIGN), (dict(_0=A + 2), ALIGN), (dict(_14=A + 8), ALIGN), (dict(_14=0), WORKSPACE), (dict(_15=4), WORKSPACE),
])
def test_dispatch(q4lib, at, code):
    refuse(q4lib, "q4_moe_dispatch", change(DISPATCH, **at), code)


COMBINE = [A, 64, A, 64, A, 64, F32, A, A, 4, 2, 64]   # Y, ldy, base, ldbase, Ys, ldys, type, row_of, weights, tokens, top_k, d


@pytest.mark.parametrize("at,code", [
    (dict(_0=0), INVALID), (dict(_4=0), INVALID), (dict(_7=0), INVALID), (dict(_1=63), INVALID), (dict(_3=63), INVALID),
    (dict(_5=63), INVALID), (dict(_6=I8), INVALID), (dict(_9=-1), INVALID), (dict(_10=0), INVALID), (dict(_11=0), INVALID),
    (dict(_2=A + 2), ALIGN), (dict(_7=A + 2), ALIGN), (dict(_8=A + 2), ALIGN),
])
def test_combine(q4lib, at, code):
    refuse(q4lib, "q4_moe_combine", change(COMBINE, **at), code)


# dYs, lddys, dweights, dY, lddy, Ys, ldys, type, row_of, weights, tokens, top_k, d
COMBINE_BWD = [A, 64, A, A, 64, A, 64, F32, A, A, 4, 2, 64]


@pytest.mark.parametrize("at,code", [
    (dict(_0=0), INVALID), (dict(_3=0), INVALID), (dict(_5=0), INVALID), (dict(_8=0), INVALID), (dict(_1=63), INVALID),
    (dict(_4=63), INVALID), (dict(_6=63), INVALID), (dict(_7=I8), INVALID), (dict(_10=-1), INVALID), (dict(_12=0), INVALID),
    (dict(_2=A + 2), ALIGN), (dict(_9=A + 2), ALIGN), (dict(_0=A + 1, _7=BF16), ALIGN),
])
def test_combine_backward(q4lib, at, code):
    refuse(q4lib, "q4_moe_combine_backward", change(COMBINE_BWD, **at), code)


def test_size_functions(q4lib):
    assert q4lib.q4_norm_workspace_size(3, 100) == 3 * 100 * 4
    assert q4lib.q4_norm_workspace_size(1 << 20, 100) == 608 * 100 * 4
    assert q4lib.q4_norm_workspace_size(-1, 100) == 0 and q4lib.q4_norm_workspace_size(3, 0) == 0
    assert q4lib.q4_moe_workspace_size(8, 8, 128) == 0                       # one CTA sorts few pairs
    assert q4lib.q4_moe_workspace_size(65536, 1, 100) == 32 * 101 * 4        # chunks of 2048 pairs
    assert q4lib.q4_moe_workspace_size(1 << 24, 2, 100) == 0 and q4lib.q4_moe_workspace_size(100, 0, 100) == 0
    assert q4lib.q4_w8a8_workspace_size(0, 64, 64) == 0 and q4lib.q4_w8a8_workspace_size(4, 48, 64) == 0
    assert q4lib.q4_w8a8_workspace_size(4, 64, 64) == 512                    # 256 bytes of codes, 16 of scales


def test_nothing_to_do_is_ok_without_a_device(q4lib):
    refuse(q4lib, "q4_a8_quantize", change(QUANT, _5=0), 0)
    refuse(q4lib, "q4_w8a8_matmul", change(MATMUL, _7=0, _10=0, _11=0), 0)
    refuse(q4lib, "q4_norm_before", change(BEFORE, _10=0), 0)
    refuse(q4lib, "q4_norm_after", change(AFTER, _14=0), 0)
    refuse(q4lib, "q4_norm_before_backward", change(BEFORE_BWD, _13=0, _2=0), 0)
    refuse(q4lib, "q4_moe_combine", change(COMBINE, _9=0), 0)
    refuse(q4lib, "q4_moe_combine_backward", change(COMBINE_BWD, _10=0), 0)
