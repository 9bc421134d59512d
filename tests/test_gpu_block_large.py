"""Rows so far apart that element offsets pass 32 bits: the calls around the linear
layers give the bits that they give on the same rows next to each other."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

M, D, LD = 2200, 192, 1 << 20      # (M - 1) * LD > 2^31 elements


@pytest.fixture(scope="module", autouse=True)
def _need_room():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < (40 << 30):
        pytest.skip("not enough device memory")


def far(x):
    v = torch.empty(M * LD, dtype=torch.bfloat16, device="cuda").view(M, LD)[:, :D]
    if x is not None:
        v.copy_(x)
    return v


def test_norms(q4lib):
    r, b = (torch.randn(M, D, device="cuda").bfloat16() for _ in range(2))
    w, ty = torch.randn(D, device="cuda"), q4lib.Q4_TYPE_BF16
    got = []
    for R, B, Y, H in ((r, b, torch.empty_like(r), torch.empty_like(r)), (far(r), far(b), far(None), far(None))):
        ld = R.stride(0)
        q4lib.q4_norm_after_before(Y, ld, H, ld, ty, None, R, ld, B, ld, ty, w, 0.0, None, 0, 0, 0.5, w, 0.0, 1e-6, M, D)
        need = q4lib.q4_norm_workspace_size(M, D)
        ws, dw = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty(D, device="cuda")
        q4lib.q4_norm_before_backward(R, ld, dw, H, ld, Y, ld, B, ld, ty, w, 0.0, 1e-6, M, D, ws, need)
        got.append((Y, H, R, dw))
    for a, c in zip(*got):
        assert torch.equal(a, c)


def test_experts(q4lib):
    t, k, e = M // 2, 2, 7
    x, ty = torch.randn(t, D, device="cuda").bfloat16(), q4lib.Q4_TYPE_BF16
    ids, w = torch.randint(-1, e, (t, k), device="cuda"), torch.randn(t, k, device="cuda")
    got = []
    for xs in (torch.empty((t * k, D), dtype=torch.bfloat16, device="cuda"), far(None)):
        offsets, row_of = torch.empty(e + 1, dtype=torch.int64, device="cuda"), torch.empty((t, k), dtype=torch.int32, device="cuda")
        y, dw = torch.empty_like(x), torch.empty_like(w)
        q4lib.q4_moe_dispatch(xs, xs.stride(0), offsets, row_of, None, ids, 8, x, D, ty, t, k, e, D, None, 0)
        q4lib.q4_moe_combine(y, D, None, 0, xs, xs.stride(0), ty, row_of, w, t, k, D)
        q4lib.q4_moe_combine_backward(xs, xs.stride(0), dw, x, D, xs, xs.stride(0), ty, row_of, w, t, k, D)
        got.append((offsets, row_of, y, dw, xs))
    for a, c in zip(*got):
        assert torch.equal(a, c)


@pytest.mark.parametrize("m", [M, 9])
def test_int8_product(q4lib, m):
    n = 130
    x, W = torch.randn(M, D, device="cuda").bfloat16(), torch.randn(n, D, device="cuda")
    P = torch.empty(q4lib.q4_w8_packed_size(n, D), dtype=torch.uint8, device="cuda")
    q4lib.q4_w8_quantize(P, W, n, D)
    need = q4lib.q4_w8a8_workspace_size(m, D, n)
    ws, got, ty = torch.empty(need, dtype=torch.uint8, device="cuda"), [], q4lib.Q4_TYPE_BF16
    for X, Y in ((x, torch.empty((M, n), dtype=torch.bfloat16, device="cuda")), (far(x), far(None)[:, :n])):
        q4lib.q4_w8a8_matmul(P, X[M - m:], X.stride(0), ty, Y[M - m:], Y.stride(0), ty, m, D, n, ws, need)
        got.append(Y[M - m:].clone())
    assert torch.equal(*got)
