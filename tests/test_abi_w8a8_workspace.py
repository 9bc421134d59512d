"""The int8 product's workspace: its size is known without a device, holds the
tokens' tiles, and never falls as the batch grows."""

import pytest

LAYERS = [(9728, 2560), (2560, 9728), (14336, 4096), (4096, 4096), (151936, 2560), (1, 32), (130, 96), (4096, 131072)]


@pytest.mark.parametrize("n,k", LAYERS)
def test_a_larger_batch_never_needs_less(q4lib, n, k):
    sizes = [q4lib.q4_w8a8_workspace_size(m, k, n) for m in range(1, 700)]
    sizes += [q4lib.q4_w8a8_workspace_size(m, k, n) for m in range(701, 1 << 20, 4999)]
    assert sizes == sorted(sizes) and sizes[0] > 0


@pytest.mark.parametrize("n,k", LAYERS)
@pytest.mark.parametrize("m", [17, 40, 257, 4096])
def test_the_tokens_tiles_are_in_it(q4lib, m, n, k):
    # codes, scales, and each token as fp16 in rows of whole 64 columns
    assert q4lib.q4_w8a8_workspace_size(m, k, n) >= m * k + 4 * m + m * ((k + 63) // 64) * 128
