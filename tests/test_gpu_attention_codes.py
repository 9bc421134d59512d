"""Many query rows over codes: denominators beside tiles of zero values."""

import numpy as np
import pytest
import torch

from block_testlib import ROUND, TINY, TYPES, blank, close, f64
from cache_testlib import Cache, attend64, held
from test_gpu_attention import FOLDED, ROUND_P

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("size", [1.0, 500.0, 30000.0])
@pytest.mark.parametrize("rest", [0.0, 1e-30])
def test_terms_of_tiles_without_values(q4lib, name, size, rest):
    """One tile of values and a long tail of none (or next to none): what the tail's
    terms, 2^-14 of the largest each, add to the denominator halves the result. Heads
    enough that a sequence's tiles are few CTAs' work."""
    d, length, new, heads = 64, 16384, 128, 160
    if name == "f16" and rest:
        pytest.skip("not a number of fp16")
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.zeros(length, 1, d, device="cuda")
    k[:, 0, 0] = 6.0
    k[0, 0, 0] = 20.0
    v = torch.full((length, 1, d), rest, device="cuda")
    v[:128] = size * (1 + 0.5 * torch.rand(128, 1, d, generator=g, device="cuda"))
    k, v = k.to(TYPES[name]), v.to(TYPES[name])
    q = torch.zeros(new, d, device="cuda")
    q[:, 0] = 1.0
    q = q.to(TYPES[name])
    scale = float(np.float32(np.log(2.0)))                  # scores in powers of two
    c = Cache(q4lib, [length], heads, d, 64, "i8")
    c.write(k.expand(length, heads, d).reshape(length, -1), v.expand(length, heads, d).reshape(length, -1), name, [length], [length])
    o = blank(new, heads * d, name)
    c.attend(o, q.repeat(1, heads), name, heads, scale, 0, [length], [new])
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
    ref, tol = attend64(q, held(k, "i8"), held(v, "i8"), 1, 1, d, scale, 0, [length], [new], ROUND_P[name, "i8"], 1, (name, "i8") == FOLDED)
    assert float(ref.abs().max()) < 0.8 * size              # (the first tile alone: more than size)
    ref, tol = f64(ref.repeat(1, heads)), f64(tol.repeat(1, heads))
    close(o, ref, tol + ROUND[name] * np.abs(ref) * 1.01 + TINY[name])
