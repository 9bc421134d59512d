"""The streamed norms under a wait limit of 1 ns, over so many rows that each CTA's
copying warp waits for room in its ring many times: they report
Q4_ERR_DEVICE_TIMEOUT, return, and leave nothing behind that the next call would
meet. (A wait can be over before it is looked at: a call is repeated until one is
not.)"""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEFAULT_NS = 2_000_000_000


@pytest.mark.parametrize("m,d,name", [(3000, 4096, "f32"), (6000, 1031, "bf16")])
@pytest.mark.parametrize("which", ["join", "before backward", "after backward"])
def test_a_wait_that_runs_out_is_reported(q4lib, m, d, name, which):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ty, dtype = (q4lib.Q4_TYPE_F32, torch.float32) if name == "f32" else (q4lib.Q4_TYPE_BF16, torch.bfloat16)
    R, B, dY, gate = (torch.randn(m, d, device="cuda").to(dtype) for _ in range(4))
    w, dw = torch.randn(d, device="cuda"), torch.zeros(d, device="cuda")
    out = [torch.zeros(m, d, device="cuda", dtype=dtype) for _ in range(2)]   # each call writes all of what it writes
    need = q4lib.q4_norm_workspace_size(m, d)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    calls = {
        "join": lambda: q4lib.q4_norm_after_before(out[0], d, out[1], d, ty, None, R, d, B, d, ty, w, 0.0, gate, d, 3, 1.0, w, 0.0,
                                                   1e-6, m, d),
        "before backward": lambda: q4lib.q4_norm_before_backward(out[0], d, dw, dY, d, R, d, B, d, ty, w, 0.0, 1e-6, m, d, ws, need),
        "after backward": lambda: q4lib.q4_norm_after_backward(out[0], d, dw, out[1], d, dY, d, B, d, ty, w, 0.0, gate, d, 3, 1.0,
                                                               1e-6, m, d, ws, need),
    }

    def status_of(ns):
        q4lib.q4_last_device_status(clear=True)
        q4lib.q4_set_wait_limit_ns(ns)
        try:
            calls[which]()
            return q4lib.q4_last_device_status(clear=True)
        finally:
            q4lib.q4_set_wait_limit_ns(DEFAULT_NS)

    assert status_of(DEFAULT_NS) == 0
    right = [t.clone() for t in (*out, dw)]
    seen = 0
    for _ in range(20):
        status = status_of(1)
        assert status in (0, q4lib.Q4_ERR_DEVICE_TIMEOUT)
        seen += status != 0
        assert status_of(DEFAULT_NS) == 0
        assert all(torch.equal(a, b) for a, b in zip((*out, dw), right))
        if seen == 3:
            break
    assert seen > 0
