"""The acceptance of drafted tokens where probabilities are none."""

import numpy as np
import pytest
import torch

from test_gpu_draft import verify, verify64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [4, 3000, 60000])
def test_acceptance_where_probabilities_are_none(q4lib, n):
    """NaN and negative ones count as 0 and those above 1 as 1, in the acceptance as in
    the draw: the tokens are those of rows where they were 0 and 1."""
    kinds = [float("nan"), -0.5, -float("inf"), 0.0, 0.25, 0.5, 1.0, 3.0, float("inf")]
    pairs = [(a, b) for a in kinds for b in kinds]
    s = len(pairs)
    p = torch.full((s, 2, n), 0.1 / n, device="cuda")
    q = torch.full((s, n), 0.1 / n, device="cuda")
    for i, (a, b) in enumerate(pairs):
        p[i, 0, 2], q[i, 2] = a, b
    p = p.reshape(-1, n)

    def clean(x):
        return torch.nan_to_num(x, nan=0.0, posinf=1.0, neginf=0.0).clamp(0.0, 1.0)

    drafted = torch.full((s, 1), 2, dtype=torch.int32, device="cuda")
    sample = torch.full((s,), 0.75, device="cuda")
    for u in (0.0, 0.3, 0.99):
        accept = torch.full((s, 1), u, device="cuda")
        for given in (q, None):
            got = verify(q4lib, p, given, drafted, None, accept, sample, n)
            want = verify64(clean(p), None if given is None else clean(q), drafted, None, accept, sample, n)
            assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])
