"""Helpers of the tests of the paged cache and the attention over it: a cache
with its sequences in pages at random places, and both operators in 64 bits."""

import math

import numpy as np
import torch

from block_testlib import TYPES, type_of

CTYPES = ("f16", "bf16", "i8")


def ctype_of(q4, name):
    return q4.Q4_TYPE_I8 if name == "i8" else type_of(q4, name)


def ints(values):
    return torch.tensor([int(v) for v in values], dtype=torch.int32, device="cuda")


def starts_of(counts):
    return [0] + [int(v) for v in np.cumsum(counts)]


def held(x, cache):
    """Rows of a head ([.., d], any type) as the cache gives them back, in 64 bits."""
    x = x.float()
    if cache != "i8":
        return x.to(TYPES[cache]).double()
    top = x.abs().amax(dim=-1, keepdim=True)
    inv = torch.where(top > 0, torch.full_like(top, 127.0) / top, torch.zeros_like(top))
    return torch.round(x * inv).double() * (top / torch.full_like(top, 127.0)).double()


class Cache:
    """Pages filled with a byte (255: NaN), and a table of random distinct pages."""

    def __init__(self, q4, lens, kv_heads, d, page, cache, seed=0, spare=2, fill=255, wide=0):
        self.q4, self.heads, self.d, self.page, self.cache = q4, kv_heads, d, page, cache
        self.ctype = ctype_of(q4, cache)
        need = [max(0, -(-int(n) // page)) for n in lens]
        self.n_pages = sum(need) + spare
        self.nbytes = q4.q4_kv_page_size(page, kv_heads, d, self.ctype)
        self.pages = torch.full((self.n_pages * self.nbytes,), fill, dtype=torch.uint8, device="cuda")
        order = np.random.default_rng(seed).permutation(self.n_pages)
        width = max(1, max(need, default=0)) + wide
        table = np.full((max(1, len(lens)), width), -7, dtype=np.int32)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        self.table = torch.from_numpy(table).cuda()

    def args(self):
        return (self.pages, self.n_pages, self.page, self.heads, self.d, self.ctype, self.table, self.table.stride(0))

    def write(self, k, v, name, lens, counts, rows=None, **kw):
        self.q4.q4_kv_write(*self.args(), ints(lens), ints(starts_of(counts)), len(counts), k, k.stride(0), v, v.stride(0),
                            type_of(self.q4, name), k.shape[0] if rows is None else rows, **kw)

    def read(self, k, v, name, first, counts, **kw):
        self.q4.q4_kv_read(k, k.stride(0), v, v.stride(0), type_of(self.q4, name), *self.args(),
                           None if first is None else ints(first), ints(starts_of(counts)), len(counts), k.shape[0], **kw)

    def attend(self, o, q, name, heads, scale, window, lens, counts, max_new=None, ws=None, **kw):
        need = self.q4.q4_attention_workspace_size(q.shape[0], len(counts), heads, self.heads, self.d)
        if ws is None:
            ws = torch.full((max(1, need),), 255, dtype=torch.uint8, device="cuda")   # it needs no initialisation
        self.q4.q4_attention(o, o.stride(0), q, q.stride(0), type_of(self.q4, name), heads, scale, window, *self.args(),
                             ints(lens), ints(starts_of(counts)), len(counts), q.shape[0],
                             max(counts) if max_new is None else max_new, ws, ws.numel(), **kw)
        return ws


def attend64(q, k, v, heads, kv_heads, d, scale, window, lens, counts, round_p, terms, folded=False):
    """The attention in 64 bits and what an output may be off by beyond its own
    rounding. q [rows, heads d], k and v [tokens of all sequences, kv_heads, d] in
    64 bits, as the cache holds them. For a row with scores s_y, B_y = scale sum_i
    |q_i k_yi|, p its softmax and A = sum_y p_y |v_y|:
      - a score's products add up in fp32, 16 at a time, cut to it: (d / 16 + 3)
        2^-23 B, times log2(e) rounded (2 roundings of |s|): in all at most (d / 16 +
        6) 2^-23 B absolute; fp32 queries as two terms: 2^-21 B more;
      - a term is 2^x with 2^-22 relative error, and its argument's last place,
        which the bound of the score holds;
      - a term is rounded to `round_p` relative (2^-21 for two terms). In fp16 (all but
        bf16 over bf16) a term has a smallest step too: it is held as 2^7 times its
        share of the largest term so far (with codes, times the value scale over a power
        of two at most twice the largest that the row has seen), and fp16's step below
        2^-14 is 2^-24, so up to 2^-25 2^-7 = 2^-32 of the largest term is lost, and with
        codes twice that: a term of the denominator is 1, so a row's sum is off by at
        most n 2^-31 max |v| over what it sees;
      - the sums add n terms in fp32, 16 at a time: (n / 16 + 8) 2^-23.
      - `folded` (bf16 queries over codes): a key or value may be code x factor, the
        factor (its scale over the power of two above the largest that stands near it)
        and the product each rounded to fp16, 2^-11: 2^-10 relative. A factor below
        2^-14 is in steps of 2^-24, so off by 2^-25 of that power of two, which is at
        most twice the largest scale seen: 127 codes of it 2^-24 of the largest key or
        value seen. For the scores 2^-10 B and 2^-24 scale |q|_1 max |k|, for the values
        2^-10 A and 2^-24 max |v|.
    A relative error e of every term moves numerator and denominator: 2 e A."""
    group = heads // kv_heads
    out = torch.zeros((sum(counts), heads * d), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    row, at = 0, 0
    for n, m in zip(lens, counts):
        n = max(n, 0)
        pos = torch.arange(n - m, n, device=q.device)[:, None]
        y = torch.arange(n, device=q.device)[None, :]
        sees = y <= pos
        if window:
            sees &= y > pos - window
        for h in range(heads if m else 0):
            kk, vv = k[at:at + n, h // group], v[at:at + n, h // group]
            qq = q[row:row + m, h * d:(h + 1) * d].double()
            s = (qq @ kk.t()) * scale
            s = torch.where(sees, s, torch.full_like(s, -math.inf))
            top = s.amax(dim=1, keepdim=True) if n else torch.full((m, 1), -math.inf, device=q.device, dtype=torch.float64)
            e = torch.where(sees, torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top)), torch.zeros_like(s))
            total = e.sum(dim=1, keepdim=True)
            p = e / torch.where(total == 0, torch.ones_like(total), total)
            clean = torch.where(torch.isfinite(vv), vv, torch.zeros_like(vv))
            out[row:row + m, h * d:(h + 1) * d] = p @ clean
            b = torch.where(sees, (qq.abs() @ kk.abs().t()) * scale, torch.zeros_like(s))
            worst = b.amax(dim=1, keepdim=True) if n else torch.zeros_like(top)
            eps = ((d / 16 + 6) * 2.0 ** -23 + (2.0 ** -21 if terms == 2 else 0.0)) * worst + 2.0 ** -22 + round_p + (n / 16 + 8) * 2.0 ** -23
            eps = eps + (2.0 ** -10 * worst + 2.0 ** -24 * scale * qq.abs().sum(dim=1, keepdim=True) * (kk.abs().max() if n else 0.0) if folded else 0.0)
            step = 0.0 if round_p == 2.0 ** -8 else n * 2.0 ** -31
            largest = (torch.where(sees, clean.abs().amax(dim=1)[None, :], torch.zeros_like(s)).amax(dim=1, keepdim=True)
                       if n else torch.zeros_like(top))
            tol[row:row + m, h * d:(h + 1) * d] = 2 * eps * (p @ clean.abs()) + step * largest
            if folded:
                tol[row:row + m, h * d:(h + 1) * d] += 2.0 ** -10 * (p @ clean.abs()) + 2.0 ** -24 * largest
        row, at = row + m, at + n
    return out, tol
