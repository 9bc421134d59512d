"""Probabilities at temperatures at the ends of fp32, and rows that are NaN whole."""

import numpy as np
import pytest
import torch

from block_testlib import TYPES, f64
from test_gpu_draft import probs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [7, 1000, 151936])
def test_temperatures_at_the_ends(q4lib, name, n):
    """Next to nothing: all on the largest logit, shared by equal ones. Infinite: the
    same for every logit but -inf. -inf has probability 0 at any."""
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.round(torch.randn(6, n, generator=g, device="cuda") * 2).to(TYPES[name])
    x[:, 1] = float("-inf")
    t = torch.tensor([2.0 ** -149, 1e-40, 2.0 ** -126, 3e38, float("inf"), 1e-30], device="cuda")
    p = f64(probs(q4lib, x, name, t))
    for i in range(6):
        z = f64(x[i])
        want = (z == z.max()).astype(np.float64) if i not in (3, 4) else (z > -np.inf).astype(np.float64)
        want /= want.sum()
        assert np.abs(p[i] - want).max() <= 2.0 ** -18 * want.max() and not p[i][want == 0].any(), f"temperature {float(t[i])}"


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [5, 9000, 151936])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_that_are_nan_whole(q4lib, name, n, bad):
    """A NaN or +inf logit, wherever it stands; a temperature that is NaN or below 0."""
    x = torch.zeros(6, n, device="cuda", dtype=TYPES[name])
    x[0, 0], x[1, n - 1], x[2, n // 2] = bad, bad, bad
    x[2, 0] = float("-inf")
    t = torch.tensor([1.0, 2.0, float("inf"), float("nan"), -1.0, 1.0], device="cuda")
    p = probs(q4lib, x, name, t)
    assert bool(torch.isnan(p[:5]).all()) and bool(torch.isfinite(p[5]).all())
