"""The mixture block of the examples, end to end, against the same block in 64
bits from the oracle's weights.

The routed experts run the library's Q4_0 products, whose own tolerance is 1e-3
(up to 16 rows an expert) or 1e-2 of a sum's terms, so the block is held to 2e-2
of its values' root mean square; what the block adds to those products is held
to tight bounds in its own tests. Routing is taken from the block itself: a tie
in the router's fp32 scores may fall to either side."""

import os
import sys

import numpy as np
import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def block(q4lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import mixture_block
    return mixture_block.MixtureBlock(d=256, f=128, n_experts=6, top_k=2, seed=3)


def dense(oracle_mod, blocks, n, k):
    eye = np.eye(k, dtype=np.float32)
    return oracle_mod.matmul(blocks, eye, n, k)[0].T      # [n x k], fp64


def int8_dense(q4lib, packed, n, k):
    codes, scales = torch.empty((n, k), dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
    q4lib.q4_w8_unpack(codes, scales, packed, n, k)
    return codes.double().cpu().numpy() * scales.double().cpu().numpy()[:, None]


def unit(x):
    return x / np.sqrt((x * x).mean(axis=1, keepdims=True) + 1e-6)


def silu_gated(x):
    a, b = np.split(x, 2, axis=1)
    return a / (1 + np.exp(-a)) * b


def as_coded(x):
    s = np.abs(x).max(axis=1, keepdims=True) / 127
    return np.rint(x / s) * s


@pytest.mark.parametrize("tokens", [1, 9, 50, 200])
def test_block_against_64_bits(q4lib, oracle_mod, block, tokens):
    d, f, k = block.d, block.f, block.k
    x = torch.randn(tokens, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(tokens)) * 2
    y, h_next = block.forward(x)
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
    n64 = lambda t: t.double().cpu().numpy()   # noqa: E731
    X = n64(x)
    h = unit(X) * n64(block.w_before)
    hd = torch.empty_like(x)
    q4lib.q4_norm_before(hd, d, 0, None, x, d, 0, block.w_before, 0.0, 1e-6, tokens, d)
    ids, weights = (t.cpu().numpy() for t in block.route(hd))
    up, down = int8_dense(q4lib, block.shared_up, 2 * f, d), int8_dense(q4lib, block.shared_down, d, f)
    out = as_coded(silu_gated(as_coded(h) @ up.T)) @ down.T
    for e in range(block.e):
        t, j = np.nonzero(ids == e)
        if t.size:
            hid = silu_gated(h[t] @ dense(oracle_mod, block.up_blocks[e], 2 * f, d).T)
            np.add.at(out, t, weights[t, j, None].astype(np.float64) * (hid @ dense(oracle_mod, block.down_blocks[e], d, f).T))
    ref = X + block.scale * n64(block.gate) * unit(out) * n64(block.w_after)
    ref_h = unit(ref) * n64(block.w_next)
    for got, want in ((n64(y), ref), (n64(h_next), ref_h)):
        rms = np.sqrt((want * want).mean())
        assert np.sqrt(((got - want) ** 2).mean()) <= 2e-2 * rms
        assert np.abs(got - want).max() <= 0.2 * rms
