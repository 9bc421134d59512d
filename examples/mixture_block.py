"""A mixture feed-forward block around quantised weights, end to end: the norm
before it, a shared expert over int8 weights and int8 tokens, routed experts
over Q4_0 weights, and the norm after it with its gate, the residual scale and
the residual sum, fused with the next block's norm.

    python examples/mixture_block.py [tokens]

The routed experts' rows are sorted on the device; their offsets come to the
host once a block, since q4_0_matmul_experts takes them there.
"""

from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np  # noqa: E402
import torch  # noqa: E402

from q4_quantized_linear_gb300 import binding as q4, synth  # noqa: E402

F32, I8 = q4.Q4_TYPE_F32, q4.Q4_TYPE_I8
EPS = 1e-6


class MixtureBlock:
    """d: model width, f: experts' width, n_experts of which top_k a token, and a
    shared expert of width f for every token. Weights are random."""

    def __init__(self, d: int, f: int, n_experts: int, top_k: int, seed: int = 0):
        self.d, self.f, self.e, self.k = d, f, n_experts, top_k
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda")

        def int8_weights(n, k):
            w = normal(n, k) / k ** 0.5
            packed = torch.empty(q4.q4_w8_packed_size(n, k), dtype=torch.uint8, device="cuda")
            q4.q4_w8_quantize(packed, w, n, k)
            return packed

        def q4_weights(n, k, seed):
            blocks = synth.q4_0_blocks(n, k, seed=seed)
            return blocks, q4.pack(torch.from_numpy(blocks.reshape(-1)).cuda(), n, k)

        self.w_before, self.w_after, self.w_next = (1 + 0.1 * normal(d) for _ in range(3))
        self.gate = 0.5 + 0.1 * normal(d)                  # of the block's output, a channel each
        self.scale = 0.7                                   # of the residual sum
        self.router = normal(n_experts, d) / d ** 0.5
        self.shared_up, self.shared_down = int8_weights(2 * f, d), int8_weights(d, f)
        ups = [q4_weights(2 * f, d, seed=seed + 10 + i) for i in range(n_experts)]
        downs = [q4_weights(d, f, seed=seed + 10 + n_experts + i) for i in range(n_experts)]
        self.up_blocks, self.up = [b for b, _ in ups], [w for _, w in ups]
        self.down_blocks, self.down = [b for b, _ in downs], [w for _, w in downs]

    def _workspace(self, nbytes: int):
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda")

    @staticmethod
    def _gated(x):
        """SiLU of the first half times the second."""
        a, b = x.chunk(2, dim=-1)
        return (torch.nn.functional.silu(a) * b).contiguous()

    def shared(self, codes, scales):
        """The shared expert: tokens that the norm coded, int8 weights."""
        t, d, f = codes.shape[0], self.d, self.f
        ws = self._workspace(max(q4.q4_w8a8_workspace_size(t, d, 2 * f), q4.q4_w8a8_workspace_size(t, f, d)))
        h, y = torch.empty((t, 2 * f), device="cuda"), torch.empty((t, d), device="cuda")
        q4.q4_w8a8_matmul_codes(self.shared_up, codes, scales, h, 2 * f, F32, t, d, 2 * f, ws, ws.numel())
        h = self._gated(h)
        q4.q4_w8a8_matmul(self.shared_down, h, f, F32, y, d, F32, t, f, d, ws, ws.numel())
        return y

    def route(self, h):
        top = torch.topk(h @ self.router.t(), self.k, dim=1)
        return top.indices.contiguous(), torch.softmax(top.values, dim=1).contiguous()

    def forward(self, x):
        """x [tokens x d] fp32, the residual stream: (the stream after the block,
        the next block's normed input)."""
        t, d, f, k = x.shape[0], self.d, self.f, self.k
        h, codes, scales = torch.empty_like(x), torch.empty((t, d), dtype=torch.int8, device="cuda"), torch.empty(t, device="cuda")
        q4.q4_norm_before(h, d, F32, None, x, d, F32, self.w_before, 0.0, EPS, t, d)
        q4.q4_norm_before(codes, d, I8, scales, x, d, F32, self.w_before, 0.0, EPS, t, d)
        ids, weights = self.route(h)
        offsets = torch.empty(self.e + 1, dtype=torch.int64, device="cuda")
        row_of = torch.empty((t, k), dtype=torch.int32, device="cuda")
        xs = torch.empty((t * k, d), device="cuda")
        ws = self._workspace(q4.q4_moe_workspace_size(t, k, self.e))
        q4.q4_moe_dispatch(xs, d, offsets, row_of, None, ids, 8, h, d, F32, t, k, self.e, d, ws, ws.numel())
        base = self.shared(codes, scales)
        host = offsets.tolist()
        hs, ys = torch.empty((t * k, 2 * f), device="cuda"), torch.empty((t * k, d), device="cuda")
        q4.q4_0_matmul_experts(self.up, host, xs, hs, d, 2 * f)
        hs = self._gated(hs)
        q4.q4_0_matmul_experts(self.down, host, hs, ys, f, d)
        out = torch.empty_like(x)
        q4.q4_moe_combine(out, d, base, d, ys, d, F32, row_of, weights, t, k, d)
        y, h_next = torch.empty_like(x), torch.empty_like(x)
        q4.q4_norm_after_before(y, d, h_next, d, F32, None, x, d, out, d, F32, self.w_after, 0.0, self.gate, 0,
                                q4.Q4_GATE_CHANNEL, self.scale, self.w_next, 0.0, EPS, t, d)
        return y, h_next


def main() -> None:
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 64
    block = MixtureBlock(d=1024, f=512, n_experts=16, top_k=4)
    x = torch.randn(tokens, block.d, device="cuda")
    y, h = block.forward(x)
    torch.cuda.synchronize()
    status = q4.q4_last_device_status()
    if status:
        raise SystemExit(q4.q4_status_string(status))
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(20):
        block.forward(x)
    end.record()
    torch.cuda.synchronize()
    print(f"{tokens} tokens, {block.e} experts, {block.k} a token: {start.elapsed_time(end) / 20 * 1e3:.0f} us a block, "
          f"|y| {float(y.norm()) / np.sqrt(y.numel()):.3f}, |h| {float(h.norm()) / np.sqrt(h.numel()):.3f}")


if __name__ == "__main__":
    main()
