"""The int8 product's sums, through tokens and weights that are whole numbers: below
2^24 the same bits whatever the batch, and past that to what the running sum loses.

A weight row that holds a 127 is its own codes with a scale of 1, so an output is
the sum itself. Past 2^24 the tensor cores add 16 columns a step to a running sum
in fp32 (up to 16 tokens: integers, one rounding at the end). A step loses less than
a unit in the last place of the sum, 2^-23 of the sizes added so far, and nothing
while those are below 2^24; slices' sums lose half a unit each when they are added."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def integers(rows, k, lo, hi, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randint(lo, hi + 1, (rows, k), generator=g, device="cuda")
    w[:, 0] = 127
    return w


def product(q4lib, codes, w, scales=None):
    m, k, n = codes.shape[0], codes.shape[1], w.shape[0]
    P = torch.empty(q4lib.q4_w8_packed_size(n, k), dtype=torch.uint8, device="cuda")
    q4lib.q4_w8_quantize(P, w.float().contiguous(), n, k)
    need = q4lib.q4_w8a8_workspace_size(m, k, n)
    ws, Y = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty((m, n), device="cuda")
    sx = torch.ones(m, device="cuda") if scales is None else scales
    q4lib.q4_w8a8_matmul_codes(P, codes.to(torch.int8).contiguous(), sx, Y, n, q4lib.Q4_TYPE_F32, m, k, n, ws, need)
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
    return Y


@pytest.mark.parametrize("n,k", [(700, 1024), (2560, 9728), (9728, 2560), (300, 65536)])
def test_below_two_to_24_a_token_has_its_bits_in_every_batch(q4lib, n, k):
    top = min(127, int((2 ** 24 / k) ** 0.5))
    codes, w = integers(300, k, -top, top, 1), integers(n, k, -top, top, 2)
    codes[:, 0] = top
    w[:, 0], scale = 127, torch.rand(300, device="cuda") + 0.5
    codes[:, 1:9] = 0      # room for column 0's larger weight
    s = codes.double() @ w.double().t()
    assert float((codes.double().abs() @ w.double().abs().t()).max()) < 2 ** 24
    want = s.float() * scale[:, None]                      # the sum is exact, sx times 1 is sx
    for m in (1, 7, 16, 17, 33, 130, 300):
        assert torch.equal(product(q4lib, codes[:m], w, scale[:m].contiguous()), want[:m]), f"{m} tokens"


@pytest.mark.parametrize("m", [1, 16, 17, 30, 70, 300])
@pytest.mark.parametrize("n,k", [(140, 8192), (140, 131072), (2560, 9728)])
@pytest.mark.parametrize("lo,hi", [(64, 127), (-127, 127)])
def test_past_two_to_24(q4lib, m, n, k, lo, hi):
    codes, w = integers(m, k, lo, hi, 3), integers(n, k, lo, hi, 4)
    Y = product(q4lib, codes, w)
    a, b = codes.double(), w.double()
    s = a @ b.t()
    if m <= 16:
        assert torch.equal(Y, s.float())
        return
    lost, size = torch.zeros_like(s), torch.zeros_like(s)
    a, b = a.abs(), b.abs()
    for c in range(0, k, 16):
        size += a[:, c:c + 16] @ b[:, c:c + 16].t()
        lost += torch.where(size >= 2.0 ** 24, size, torch.zeros_like(size))
    tol = 2.0 ** -23 * lost + 16 * 2.0 ** -24 * size + 2.0 ** -24 * s.abs()
    assert bool(((Y.double() - s).abs() <= tol).all())
