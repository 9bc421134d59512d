"""Waits of the attention that run out for sure: shapes whose kernels wait longer
than the shortest limit, each of which has to say so; and the probabilities, whose
waits are for their own copies and have a limit of their own."""

import pytest
import torch

from block_testlib import TYPES, blank
from cache_testlib import Cache
from test_gpu_attention import KINDS

pytestmark = pytest.mark.gpu


@pytest.fixture
def limit(q4lib):
    yield q4lib.q4_set_wait_limit_ns
    q4lib.q4_set_wait_limit_ns(2_000_000_000)


@pytest.mark.parametrize("name,cache", KINDS)
@pytest.mark.parametrize("d,new,length", [(256, 2, 60000), (128, 16, 60000), (128, 200, 20000), (256, 200, 20000)])
def test_attention_says_so(q4lib, limit, name, cache, d, new, length):
    """Blocks of 16, 64 and 256 query rows: every call returns, some of five say that a
    wait ran out, and the calls between them are as ever."""
    heads, kv_heads = 8, 2
    g = torch.Generator(device="cuda").manual_seed(7)
    c = Cache(q4lib, [length], kv_heads, d, 64, cache)
    k = torch.randn(length, kv_heads * d, generator=g, device="cuda").to(TYPES[name])
    c.write(k, k, name, [length], [length])
    q = torch.randn(new, heads * d, generator=g, device="cuda").to(TYPES[name])
    good, o = blank(new, heads * d, name), blank(new, heads * d, name)
    c.attend(good, q, name, heads, 0.1, 0, [length], [new])
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
    out = 0
    for _ in range(5):
        limit(1)
        c.attend(o, q, name, heads, 0.1, 0, [length], [new])
        torch.cuda.synchronize()
        status = q4lib.q4_last_device_status(clear=True)
        assert status in (0, q4lib.Q4_ERR_DEVICE_TIMEOUT)
        out += status != 0
        limit(2_000_000_000)
        c.attend(o, q, name, heads, 0.1, 0, [length], [new])
        torch.cuda.synchronize()
        assert q4lib.q4_last_device_status(clear=True) == 0 and torch.equal(o, good)
    assert out > 0


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("rows_,n", [(4, 151936), (300, 50000), (2, 2000000)])
def test_probabilities_do_not(q4lib, limit, name, rows_, n):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows_, n, generator=g, device="cuda").to(TYPES[name])
    t = torch.rand(rows_, generator=g, device="cuda") + 0.5
    t[0] = 0.0
    want, got = torch.empty(rows_, n, device="cuda"), torch.empty(rows_, n, device="cuda")
    type_ = {"f32": q4lib.Q4_TYPE_F32, "bf16": q4lib.Q4_TYPE_BF16}[name]
    q4lib.q4_token_probs(want, n, x, n, type_, t, rows_, n)
    limit(1)
    for _ in range(5):
        got.fill_(-1.0)
        q4lib.q4_token_probs(got, n, x, n, type_, t, rows_, n)
        torch.cuda.synchronize()
        assert q4lib.q4_last_device_status(clear=True) == 0 and torch.equal(got, want)
