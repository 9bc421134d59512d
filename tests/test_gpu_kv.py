"""The paged cache: written values and codes are what the rule gives, to the bit;
everything else in the pages is left as it was."""

import numpy as np
import pytest
import torch

from block_testlib import TYPES, blank, gaps_kept, rows
from cache_testlib import CTYPES, Cache, held, starts_of

pytestmark = pytest.mark.gpu


def values(total, heads, d, name, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(total, heads * d, generator=g, device="cuda") * (1 + 5 * torch.rand(total, 1, generator=g, device="cuda"))
    return x.to(TYPES[name])


def split(x, lens, counts, heads, d):
    """The last counts[i] of each sequence's lens[i] rows."""
    at, out = 0, []
    for n, m in zip(lens, counts):
        out.append(x[at + n - m:at + n])
        at += n
    return torch.cat(out)


def status_ok(q4):
    torch.cuda.synchronize()
    assert q4.q4_last_device_status(clear=True) == 0


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cache", CTYPES)
@pytest.mark.parametrize("heads,d,page,pad,shift", [(2, 64, 16, 0, 0), (1, 128, 64, 8, 0), (3, 80, 32, 1, 0), (2, 256, 16, 0, 3),
                                                    (1, 192, 128, 0, 0), (5, 8, 16, 0, 0), (2, 40, 1024, 4, 1)])
def test_write_and_read(q4lib, name, cache, heads, d, page, pad, shift):
    lens, counts = [70, 0, 1, 33, 16], [70, 0, 1, 5, 16]
    total = sum(lens)
    k, v = values(total, heads, d, name), values(total, heads, d, name, 2)
    c = Cache(q4lib, lens, heads, d, page, cache)
    old = [n - m for n, m in zip(lens, counts)]
    # what was there before, then the batch's new tokens
    before = [lens[i] - counts[i] for i in range(len(lens))]
    at = starts_of(lens)
    first_k = torch.cat([k[at[i]:at[i] + before[i]] for i in range(len(lens))])
    first_v = torch.cat([v[at[i]:at[i] + before[i]] for i in range(len(lens))])
    c.write(first_k, first_v, name, old, before)
    new_k, new_v = rows(split(k, lens, counts, heads, d), name, pad, shift), rows(split(v, lens, counts, heads, d), name, pad, shift)
    c.write(new_k, new_v, name, lens, counts)
    for out in {name, "f32"}:
        bk, bv = blank(total, heads * d, out, pad, shift), blank(total, heads * d, out, pad, shift)
        c.read(bk, bv, out, None, lens)
        status_ok(q4lib)
        for got, want in ((bk, k), (bv, v)):
            ref = held(want.reshape(total, heads, d), cache).float().to(TYPES[out]).reshape(total, -1)
            assert torch.equal(got, ref)
            assert gaps_kept(got)
    # some tokens from the middle on
    bk, bv = blank(7, heads * d, name), blank(7, heads * d, name)
    c.read(bk, bv, name, [61, 0, 0, 30, 0], [4, 0, 0, 3, 0])
    ref = held(k.reshape(total, heads, d), cache).float().to(TYPES[name]).reshape(total, -1)
    assert torch.equal(bk[:4], ref[61:65]) and torch.equal(bk[4:], ref[at[3] + 30:at[3] + 33])


@pytest.mark.parametrize("cache", CTYPES)
def test_only_the_batch_is_touched(q4lib, cache):
    """Rows past the last sequence are not read, other places of the pages keep
    their bytes, rows of the outputs past the last sequence theirs."""
    heads, d, page = 2, 64, 32
    lens, counts = [40, 7], [3, 2]
    c = Cache(q4lib, lens, heads, d, page, cache, fill=17)
    k = values(9, heads, d, "bf16")
    k[5:] = float("nan")
    c.write(k, k, "bf16", lens, counts)
    status_ok(q4lib)
    changed = (c.pages != 17).reshape(c.n_pages, -1).sum(dim=1)
    touched = {int(c.table[0, 1]), int(c.table[1, 0])}
    assert {i for i in range(c.n_pages) if changed[i] > 0} == touched
    per_token = c.nbytes // page
    assert int(changed[int(c.table[0, 1])]) <= 3 * per_token and int(changed[int(c.table[1, 0])]) <= 2 * per_token
    bk, bv = rows(torch.full((9, heads * d), 5.0), "f32"), rows(torch.full((9, heads * d), 5.0), "f32")
    c.read(bk, bv, "f32", [37, 5], counts)
    status_ok(q4lib)
    assert torch.equal(bk[:5], held(k[:5].reshape(5, heads, d), cache).float().reshape(5, -1))
    assert bool((bk[5:] == 5.0).all()) and bool((bv[5:] == 5.0).all())


@pytest.mark.parametrize("cache", CTYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 1e30])
def test_what_is_not_finite(q4lib, cache, bad):
    """A head's token with such a key or value: NaN keys, zero values; its other
    heads and tokens as ever. 1e30 is finite in fp32 and bf16 alone."""
    heads, d = 2, 64
    k, v = values(4, heads, d, "f32"), values(4, heads, d, "f32", 2)
    rk, rv = k.clone(), v.clone()
    v[1, 3] = bad
    k[2, d + 5] = bad
    if cache == "f16" or bad != 1e30:
        rk[1, :d], rv[1, :d] = float("nan"), 0.0
        rk[2, d:], rv[2, d:] = float("nan"), 0.0
    else:
        rk, rv = k, v
    c = Cache(q4lib, [4], heads, d, 16, cache)
    c.write(k, v, "f32", [4], [4])
    bk, bv = blank(4, heads * d, "f32"), blank(4, heads * d, "f32")
    c.read(bk, bv, "f32", None, [4])
    status_ok(q4lib)
    for got, want in ((bk, rk), (bv, rv)):
        ref = held(want.reshape(4, heads, d), cache).float().reshape(4, -1)
        assert torch.equal(torch.isnan(got), torch.isnan(ref)) and torch.equal(torch.nan_to_num(got), torch.nan_to_num(ref))


def test_bad_pages_and_places(q4lib):
    """A page or place that the cache does not have is recorded and skipped."""
    heads, d, page = 1, 64, 16
    k = values(6, heads, d, "f32")
    for table, lens, lost in (([[0, -1]], [18], [4, 5]), ([[0, 3]], [18], [4, 5]), ([[0, 1]], [34], [4, 5]), ([[0, 1]], [4], [0, 1])):
        c = Cache(q4lib, [20], heads, d, page, "f16", spare=0, fill=0)
        c.table = torch.tensor(table, dtype=torch.int32, device="cuda")
        c.n_pages, counts = 2, [6]
        before = c.pages.clone()
        c.write(k, k, "f32", lens, counts)
        torch.cuda.synchronize()
        assert q4lib.q4_last_device_status(clear=True) == q4lib.Q4_ERR_DEVICE_CHECK
        bk, bv = blank(6, d, "f32"), blank(6, d, "f32")
        c.read(bk, bv, "f32", [lens[0] - 6], counts)
        torch.cuda.synchronize()
        assert q4lib.q4_last_device_status(clear=True) == q4lib.Q4_ERR_DEVICE_CHECK
        ref = held(k.reshape(6, 1, d), "f16").float().reshape(6, -1)
        for i in range(6):
            assert torch.equal(bk[i], torch.zeros_like(bk[i]) if i in lost else ref[i])
        assert before.numel() == c.pages.numel()


def test_large_offsets(q4lib):
    """Pages past 2^32 bytes."""
    heads, d, page = 8, 128, 64
    nbytes = q4lib.q4_kv_page_size(page, heads, d, q4lib.Q4_TYPE_BF16)
    n_pages = (1 << 32) // nbytes + 5
    c = Cache(q4lib, [40], heads, d, page, "bf16", spare=0)
    c.pages = torch.zeros(n_pages * nbytes, dtype=torch.uint8, device="cuda")
    c.n_pages = n_pages
    c.table = torch.tensor([[n_pages - 1]], dtype=torch.int32, device="cuda")
    k = values(40, heads, d, "bf16")
    c.write(k, k, "bf16", [40], [40])
    bk, bv = blank(40, heads * d, "bf16"), blank(40, heads * d, "bf16")
    c.read(bk, bv, "bf16", None, [40])
    status_ok(q4lib)
    assert torch.equal(bk, k) and torch.equal(bv, k)
    assert not bool(c.pages[:(n_pages - 1) * nbytes].any())


def test_many_sequences(q4lib):
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 40, 1024)]
    counts = [int(rng.integers(0, n + 1)) for n in lens]
    heads, d = 1, 64
    k = values(sum(lens), heads, d, "f16")
    c = Cache(q4lib, lens, heads, d, 16, "i8")
    old = [n - m for n, m in zip(lens, counts)]
    at = starts_of(lens)
    c.write(torch.cat([k[at[i]:at[i] + old[i]] for i in range(1024)]), torch.cat([k[at[i]:at[i] + old[i]] for i in range(1024)]), "f16", old, old)
    c.write(split(k, lens, counts, heads, d), split(k, lens, counts, heads, d), "f16", lens, counts)
    bk, bv = blank(sum(lens), d, "f32"), blank(sum(lens), d, "f32")
    c.read(bk, bv, "f32", None, lens)
    status_ok(q4lib)
    ref = held(k.reshape(-1, heads, d), "i8").float().reshape(-1, d)
    assert torch.equal(bk, ref) and torch.equal(bv, ref)
