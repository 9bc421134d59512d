"""Calls of no rows take the addresses that empty tensors have, which is none."""

import pytest

A = 0x100000
F32, I8 = 0, 3


CALLS = [
    ("q4_a8_quantize", [0, 0, 0, 64, F32, 0, 64]),
    ("q4_w8a8_matmul", [A, 0, 64, F32, 0, 96, F32, 0, 64, 96, 0, 0]),
    ("q4_w8a8_matmul_codes", [A, 0, 0, 0, 96, F32, 0, 64, 96, 0, 0]),
    ("q4_norm_before", [0, 64, F32, 0, 0, 64, F32, A, 0.0, 1e-6, 0, 64]),
    ("q4_norm_before", [0, 64, I8, 0, 0, 64, F32, A, 0.0, 1e-6, 0, 64]),
    ("q4_norm_after", [0, 64, 0, 64, 0, 64, F32, A, 0.0, 0, 0, 2, 1.0, 1e-6, 0, 64]),
    ("q4_norm_after_before", [0, 64, 0, 64, I8, 0, 0, 64, 0, 64, F32, A, 0.0, 0, 64, 3, 1.0, A, 0.0, 1e-6, 0, 64]),
    ("q4_norm_before_backward", [0, 64, 0, 0, 64, 0, 64, 0, 64, F32, A, 0.0, 1e-6, 0, 64, 0, 0]),
    ("q4_norm_after_backward", [0, 64, 0, 0, 64, 0, 64, 0, 64, F32, A, 0.0, 0, 64, 3, 1.0, 1e-6, 0, 64, 0, 0]),
    ("q4_moe_combine", [0, 64, 0, 64, 0, 64, F32, 0, 0, 0, 2, 64]),
    ("q4_moe_combine_backward", [0, 64, 0, 0, 64, 0, 64, F32, 0, 0, 0, 2, 64]),
]


@pytest.mark.parametrize("name,args", CALLS)
def test_no_rows_no_addresses(q4lib, name, args):
    assert getattr(q4lib, name)(*args, stream=0, check=False) == 0


@pytest.mark.parametrize("name,args", CALLS)
def test_what_is_kept_is_still_asked_for(q4lib, name, args):
    # a row more and the same addresses are refused; so is a negative count
    at = {"q4_a8_quantize": 5, "q4_w8a8_matmul": 7, "q4_w8a8_matmul_codes": 6, "q4_norm_before": 10, "q4_norm_after": 14,
          "q4_norm_after_before": 20, "q4_norm_before_backward": 13, "q4_norm_after_backward": 17, "q4_moe_combine": 9,
          "q4_moe_combine_backward": 10}[name]
    for count in (1, -1):
        assert getattr(q4lib, name)(*(args[:at] + [count] + args[at + 1:]), stream=0, check=False) == 1


@pytest.mark.gpu
def test_empty_tensors(q4lib):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    d, e, k = 64, 4, 2
    x, ids = torch.empty((0, d), device="cuda"), torch.empty((0, k), dtype=torch.int64, device="cuda")
    row_of, weights = torch.empty((0, k), dtype=torch.int32, device="cuda"), torch.empty((0, k), device="cuda")
    offsets = torch.full((e + 1,), 3, dtype=torch.int64, device="cuda")
    q4lib.q4_moe_dispatch(x, d, offsets, row_of, row_of, ids, 8, x, d, F32, 0, k, e, d, None, 0)
    assert bool((offsets == 0).all())
    offsets.fill_(3)
    kept = torch.full((4, d), 3.0, device="cuda")            # a buffer kept for larger batches
    q4lib.q4_moe_dispatch(kept, d, offsets, row_of, None, ids, 8, x, d, F32, 0, k, e, d, None, 0)
    assert bool((offsets == 0).all()) and bool((kept == 3.0).all())
    q4lib.q4_moe_combine(x, d, None, 0, x, d, F32, row_of, weights, 0, k, d)
    q4lib.q4_moe_combine_backward(x, d, weights, x, d, x, d, F32, row_of, weights, 0, k, d)
    w, dw, dg = (torch.full((d,), 3.0, device="cuda") for _ in range(3))
    q4lib.q4_norm_before_backward(x, d, dw, x, d, None, 0, x, d, F32, w, 0.0, 1e-6, 0, d, None, 0)
    assert bool((dw == 0).all())
    dw.fill_(3.0)
    q4lib.q4_norm_after_backward(x, d, dw, dg, 0, x, d, x, d, F32, w, 0.0, w, 0, q4lib.Q4_GATE_CHANNEL, 1.0, 1e-6, 0, d, None, 0)
    assert bool((dw == 0).all()) and bool((dg == 0).all())
