"""One workspace of the int8 product, sized for the largest batch, serves every
smaller one."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("n,k,most", [(9728, 2560, 64), (4096, 4096, 320), (2560, 9728, 100)])
def test_a_workspace_for_the_largest_batch(q4lib, n, k, most):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator(device="cuda").manual_seed(n)
    W, X = torch.randn(n, k, generator=g, device="cuda"), torch.randn(most, k, generator=g, device="cuda")
    P = torch.empty(q4lib.q4_w8_packed_size(n, k), dtype=torch.uint8, device="cuda")
    q4lib.q4_w8_quantize(P, W, n, k)
    need = q4lib.q4_w8a8_workspace_size(most, k, n)
    # filled, and nothing written past its end
    ws = torch.full((need + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    Y = torch.empty((most, n), device="cuda")
    q4lib.q4_w8a8_matmul(P, X, k, 0, Y, n, 0, most, k, n, ws, need)
    for m in sorted({1, 9, 16, 17, 24, 31, 33, 52, 53, most // 2, most - 1}):
        Z = torch.full((m, n), float("nan"), device="cuda")
        q4lib.q4_w8a8_matmul(P, X, k, 0, Z, n, 0, m, k, n, ws, need)
        # sums of these codes stay below 2^24: exact in every plan
        assert torch.equal(Z, Y[:m]), f"{m} tokens"
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
    assert bool((ws[need:] == 0xAB).all())
