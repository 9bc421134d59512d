"""The calls around the linear layers as programs make them: captured in a graph
and replayed on new values, from two threads at once, and with more choices a
token than a warp has lanes."""

import threading

import numpy as np
import pytest

from block_testlib import close, f64
from test_gpu_moe import E, choices, dispatch, reference

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, BF16, I8 = 0, 2, 3


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Step:
    """A norm as codes, their product, the join and its gradient; the experts'
    sort, its rows back, and their gradient: buffers of its own."""

    def __init__(self, q4lib, m, seed, d=640, n=900, e=24, k=4):
        self.q4, self.m, self.d, self.n, self.e, self.k = q4lib, m, d, n, e, k
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.x, self.w = torch.randn(m, d, generator=g, device="cuda"), 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
        self.ids = torch.randint(-1, e, (m, k), generator=g, device="cuda")
        self.weights = torch.rand(m, k, generator=g, device="cuda")
        W = torch.randn(n, d, generator=g, device="cuda")
        self.P = torch.empty(q4lib.q4_w8_packed_size(n, d), dtype=torch.uint8, device="cuda")
        q4lib.q4_w8_quantize(self.P, W, n, d)
        self.codes, self.scales = torch.empty((m, d), dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
        self.y, self.z = torch.empty((m, n), device="cuda"), torch.empty((m, n), device="cuda")
        self.r, self.h, self.dx, self.out = (torch.empty((m, d), device="cuda") for _ in range(4))
        self.dw = torch.empty(d, device="cuda")
        self.offsets = torch.empty(e + 1, dtype=torch.int64, device="cuda")
        self.row_of = torch.empty((m, k), dtype=torch.int32, device="cuda")
        self.xs, self.dxs = torch.empty((m * k, d), device="cuda"), torch.empty((m * k, d), device="cuda")
        self.dweights = torch.empty((m, k), device="cuda")
        self.sizes = [q4lib.q4_w8a8_workspace_size(m, d, n), q4lib.q4_norm_workspace_size(m, d), q4lib.q4_moe_workspace_size(m, k, e)]
        self.ws = [torch.empty(max(1, s), dtype=torch.uint8, device="cuda") for s in self.sizes]
        torch.cuda.synchronize()

    def run(self, stream=None):
        q, m, d, n, s = self.q4, self.m, self.d, self.n, stream
        q.q4_norm_before(self.codes, d, I8, self.scales, self.x, d, F32, self.w, 0.0, 1e-6, m, d, stream=s)
        q.q4_w8a8_matmul_codes(self.P, self.codes, self.scales, self.y, n, F32, m, d, n, self.ws[0], self.sizes[0], stream=s)
        q.q4_w8a8_matmul(self.P, self.x, d, F32, self.z, n, F32, m, d, n, self.ws[0], self.sizes[0], stream=s)
        q.q4_norm_after_before(self.r, d, self.h, d, F32, None, self.x, d, self.x, d, F32, self.w, 0.0, None, 0, 0, 0.5, self.w, 0.0,
                               1e-6, m, d, stream=s)
        q.q4_norm_before_backward(self.dx, d, self.dw, self.h, d, None, 0, self.r, d, F32, self.w, 0.0, 1e-6, m, d, self.ws[1],
                                  self.sizes[1], stream=s)
        q.q4_moe_dispatch(self.xs, d, self.offsets, self.row_of, None, self.ids, 8, self.h, d, F32, m, self.k, self.e, d, self.ws[2],
                          self.sizes[2], stream=s)
        q.q4_moe_combine(self.out, d, self.x, d, self.xs, d, F32, self.row_of, self.weights, m, self.k, d, stream=s)
        q.q4_moe_combine_backward(self.dxs, d, self.dweights, self.out, d, self.xs, d, F32, self.row_of, self.weights, m, self.k, d,
                                  stream=s)

    def results(self):
        return [t.clone() for t in (self.codes, self.scales, self.y, self.z, self.r, self.h, self.dx, self.dw, self.offsets, self.row_of,
                                    self.xs, self.out, self.dxs, self.dweights)]


# one launch and three for the sort; a mat-vec, the GEMM, the GEMM in slices;
# norms in registers and streamed
@pytest.mark.parametrize("m", [1, 12, 100, 2500])
def test_captured_and_replayed_on_new_values(q4lib, m):
    step = Step(q4lib, m, seed=m)
    x0, ids0 = step.x.clone(), step.ids.clone()
    x1, ids1 = torch.randn_like(x0), torch.randint(0, step.e, ids0.shape, device="cuda")
    want = []
    for x, ids in ((x0, ids0), (x1, ids1)):
        step.x.copy_(x)
        step.ids.copy_(ids)
        step.run()
        torch.cuda.synchronize()
        want.append(step.results())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    for (x, ids), right in zip(((x0, ids0), (x1, ids1), (x0, ids0)), want + want[:1]):
        step.x.copy_(x)
        step.ids.copy_(ids)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(step.results(), right):
            assert torch.equal(a, b)
    assert q4lib.q4_last_device_status(clear=True) == 0


@pytest.mark.parametrize("m", [3, 200])
def test_from_two_threads(q4lib, m):
    steps = [Step(q4lib, m, seed) for seed in (1, 2)]
    right = []
    for step in steps:
        step.run()
        torch.cuda.synchronize()
        right.append(step.results())
    errors = []

    def work(step, want):
        try:
            stream = torch.cuda.Stream()
            for _ in range(40):
                step.run(stream)
            stream.synchronize()
            with torch.cuda.stream(stream):
                got = step.results()
            stream.synchronize()
            errors.extend("results differ" for a, b in zip(got, want) if not torch.equal(a, b))
        except Exception as e:   # noqa: BLE001 (reported below, in the test's own thread)
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=a) for a in zip(steps, right)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    assert q4lib.q4_last_device_status(clear=True) == 0


@pytest.mark.parametrize("t,k,e,d", [(7, 33, 40, 72), (3, 64, 9, 1), (20, 100, 300, 130), (2, 1024, 4096, 40)])
@pytest.mark.parametrize("name,odd", [("f32", 0), ("bf16", 0), ("bf16", 1)])
def test_more_choices_than_lanes(q4lib, t, k, e, d, name, odd):
    dtype, ty = (torch.float32, F32) if name == "f32" else (torch.bfloat16, BF16)
    half = 2.0 ** -24 if name == "f32" else 2.0 ** -8
    rng = np.random.default_rng(k)
    ids = choices(t, k, e, k)
    X = torch.as_tensor(rng.standard_normal((t, d + odd))).to(dtype).cuda()[:, odd:]
    offsets, row_of, pair_of, Xs = dispatch(q4lib, ids, e, X, name)
    want = reference(ids, e)
    for a, b in zip((offsets, row_of, pair_of), want):
        assert np.array_equal(a, b)
    x64, kept = f64(X), want[1] >= 0
    sorted_x = np.where(kept.reshape(-1)[want[2]][:, None], x64[want[2] // k], 0.0)
    assert np.array_equal(f64(Xs), sorted_x)
    w = torch.as_tensor(rng.standard_normal((t, k)), dtype=torch.float32).cuda()
    rd, w64 = torch.as_tensor(row_of).cuda(), np.where(kept, f64(w), 0.0)
    Y = torch.empty((t, d + odd), dtype=dtype, device="cuda")[:, odd:]
    q4lib.q4_moe_combine(Y, d + odd, None, 0, Xs, Xs.stride(0), ty, rd, w, t, k, d)
    y, size = w64.sum(axis=1)[:, None] * x64, np.abs(w64).sum(axis=1)[:, None] * np.abs(x64)
    close(Y, y, (k + 2) * E * size + half * np.abs(y) + 2.0 ** -133)
    dYs, dw = torch.empty_like(Xs), torch.empty_like(w)
    q4lib.q4_moe_combine_backward(dYs, dYs.stride(0), dw, Y, d + odd, Xs, Xs.stride(0), ty, rd, w, t, k, d)
    y64 = f64(Y)
    dys = np.zeros((t * k, d))
    rows_of = np.where(kept, row_of, -1 - row_of).reshape(-1)
    dys[rows_of] = (w64[:, :, None] * y64[:, None, :]).reshape(t * k, d)
    close(dYs, dys, (E + half) * np.abs(dys) + 2.0 ** -133)
    dot, dsize = (y64 * x64).sum(axis=1)[:, None] * kept, np.abs(y64 * x64).sum(axis=1)[:, None] * kept
    close(dw, dot, (d / 32 + 8) * E * dsize + 1e-37)
