"""The bounded waits of the kernels around the linear layers: with a limit of 1 ns
the int8 product, whose first wait is for a copy just issued, reports
Q4_ERR_DEVICE_TIMEOUT through the status word, lets the copies in flight land and
returns. A norm's rows may have landed before they are first waited for: it
reports the same, or its results are right. The next call with the default limit
is right either way."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _with_limit(q4lib, ns, call):
    q4lib.q4_last_device_status(clear=True)
    q4lib.q4_set_wait_limit_ns(ns)
    try:
        call()
        return q4lib.q4_last_device_status(clear=True)
    finally:
        q4lib.q4_set_wait_limit_ns(2_000_000_000)


@pytest.mark.parametrize("m,n,k", [(40, 200, 96), (300, 1000, 4096), (2000, 4096, 1056)])
def test_int8_product(q4lib, m, n, k):
    W, X, Y = torch.randn(n, k, device="cuda"), torch.randn(m, k, device="cuda"), torch.empty(m, n, device="cuda")
    P = torch.empty(q4lib.q4_w8_packed_size(n, k), dtype=torch.uint8, device="cuda")
    q4lib.q4_w8_quantize(P, W, n, k)
    need = q4lib.q4_w8a8_workspace_size(m, k, n)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    call = lambda: q4lib.q4_w8a8_matmul(P, X, k, 0, Y, n, 0, m, k, n, ws, need)   # noqa: E731
    assert _with_limit(q4lib, 2_000_000_000, call) == 0
    right = Y.clone()
    assert _with_limit(q4lib, 1, call) == q4lib.Q4_ERR_DEVICE_TIMEOUT
    assert _with_limit(q4lib, 2_000_000_000, call) == 0
    assert torch.equal(Y, right)


@pytest.mark.parametrize("m,d,kind", [(400, 2560, 0), (3000, 4096, 3)])
def test_norms(q4lib, m, d, kind):
    R, B, dY, gate = (torch.randn(m, d, device="cuda") for _ in range(4))
    # zeros: each call writes some of these, and all are compared
    w, dw = torch.randn(d, device="cuda"), torch.zeros(d, device="cuda")
    Y, H, dB, dg = (torch.zeros(m, d, device="cuda") for _ in range(4))
    need = q4lib.q4_norm_workspace_size(m, d)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    g, dgate = (gate, dg) if kind else (None, None)
    calls = [
        lambda: q4lib.q4_norm_after_before(Y, d, H, d, 0, None, R, d, B, d, 0, w, 0.0, g, d, kind, 1.0, w, 0.0, 1e-6, m, d),
        lambda: q4lib.q4_norm_before_backward(dB, d, dw, dY, d, R, d, B, d, 0, w, 0.0, 1e-6, m, d, ws, need),
        lambda: q4lib.q4_norm_after_backward(dB, d, dw, dgate, d, dY, d, B, d, 0, w, 0.0, g, d, kind, 1.0, 1e-6, m, d, ws, need),
    ]
    for call in calls:
        assert _with_limit(q4lib, 2_000_000_000, call) == 0
        right = [t.clone() for t in (Y, H, dB, dw)]
        status = _with_limit(q4lib, 1, call)
        assert status in (0, q4lib.Q4_ERR_DEVICE_TIMEOUT)
        if status:
            assert _with_limit(q4lib, 2_000_000_000, call) == 0
        assert all(torch.equal(a, b) for a, b in zip((Y, H, dB, dw), right))
