"""The int8 product right behind the kernel that writes its weights: with weights
not declared read-only it reads what that kernel wrote, and declaring them so
changes no bit."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

N, K = 3000, 2080


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def setup(q4lib, m, coded):
    g = torch.Generator(device="cuda").manual_seed(m)
    Ws = [torch.randn(N, K, generator=g, device="cuda") for _ in range(3)]
    X = torch.randn(m, K, generator=g, device="cuda")
    P = torch.empty(q4lib.q4_w8_packed_size(N, K), dtype=torch.uint8, device="cuda")
    need = q4lib.q4_w8a8_workspace_size(m, K, N)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    codes, scales = torch.empty((m, K), dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    q4lib.q4_a8_quantize(codes, scales, X, K, q4lib.Q4_TYPE_F32, m, K)

    def product(Y):
        if coded:
            q4lib.q4_w8a8_matmul_codes(P, codes, scales, Y, N, q4lib.Q4_TYPE_F32, m, K, N, ws, need)
        else:
            q4lib.q4_w8a8_matmul(P, X, K, q4lib.Q4_TYPE_F32, Y, N, q4lib.Q4_TYPE_F32, m, K, N, ws, need)

    return Ws, P, product


@pytest.mark.parametrize("m", [1, 8, 16, 40, 300])
@pytest.mark.parametrize("coded", [False, True])
def test_product_behind_its_quantiser(q4lib, m, coded):
    Ws, P, product = setup(q4lib, m, coded)
    right = []
    for W in Ws:
        q4lib.q4_w8_quantize(P, W, N, K)
        torch.cuda.synchronize()
        right.append(torch.empty(m, N, device="cuda"))
        product(right[-1])
        torch.cuda.synchronize()
    Ys = [torch.empty(m, N, device="cuda") for _ in range(60)]
    torch.cuda.synchronize()
    for i, Y in enumerate(Ys):
        q4lib.q4_w8_quantize(P, Ws[i % 3], N, K)
        product(Y)
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
    for i, Y in enumerate(Ys):
        assert torch.equal(Y, right[i % 3]), f"call {i}"


@pytest.mark.parametrize("m", [1, 8, 40])
@pytest.mark.parametrize("coded", [False, True])
def test_weights_declared_read_only(q4lib, m, coded):
    Ws, P, product = setup(q4lib, m, coded)
    q4lib.q4_w8_quantize(P, Ws[0], N, K)
    Ys = [torch.empty(m, N, device="cuda") for _ in range(4)]
    product(Ys[0])
    torch.cuda.synchronize()
    try:
        q4lib.q4_set_weight_prefetch(True)
        for Y in Ys[1:]:
            product(Y)
        torch.cuda.synchronize()
    finally:
        q4lib.q4_set_weight_prefetch(False)
    assert q4lib.q4_last_device_status(clear=True) == 0
    assert all(torch.equal(Y, Ys[0]) for Y in Ys)
