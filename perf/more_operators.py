"""Cases of the operators between the linear layers of a generating model: what
is timed, the plain form of each, and its value in 64 bits.

A pass of a server over its slots takes new tokens of some sequences (a prompt's
chunk, one token, or a few drafted ones), keeps their keys and values in a cache
of pages, lets them attend to all that their sequence holds there, and turns the
logit head's output into accepted tokens:

  step      new tokens' keys and values into the cache, coded to int8 where the
            cache holds codes, and the new tokens' attention over it
  attend    the attention alone: a chunk of new tokens over a paged cache
  store     a prompt's keys and values into the cache, and read back as values
  fetch     the values of whole sequences out of the cache, as a program does
            that moves a conversation or looks at what is cached
  probs     logits over a temperature to probabilities
  verify    drafted tokens against the target's probabilities, from given random
            numbers: how many are kept, and the token after them

Plain forms: elementary torch operations in fp32 (in 64 bits where a token is
chosen by a sum over the vocabulary), rounded once at the end.
"""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "i8": 1}

# The largest cases; a drawn case stays within them.
MAX_PRODUCTS = 2048 * 15360 * 32 * 128      # query rows x keys x dims
MAX_BYTES = 320 * 151936 * 6
MAX_PROBS = 320 * 151936


def listed():
    return [
        # a single conversation's decode step behind a fp32 projection
        dict(name="step one token", kind="step", seqs=1, new=1, len=1000, ragged=0.0, heads=32, kv_heads=8, d=128,
             page=64, type="f32", cache="f16", window=0, pad=0),
        # sixteen conversations' tokens in one decode step, the cache in int8
        dict(name="step 16 slots", kind="step", seqs=16, new=1, len=8192, ragged=0.9, heads=32, kv_heads=8, d=128,
             page=64, type="bf16", cache="i8", window=0, pad=2048),
        # four drafted tokens and one more for each of sixteen conversations
        dict(name="attend drafted tokens", kind="attend", seqs=16, new=5, len=4096, ragged=0.5, heads=32, kv_heads=8,
             d=128, page=16, type="bf16", cache="bf16", window=0, pad=0),
        # a prompt of 540 tokens behind a cached conversation in int8
        dict(name="attend chunk, int8", kind="attend", seqs=1, new=540, len=8100, ragged=0.0, heads=32, kv_heads=8,
             d=128, page=64, type="bf16", cache="i8", window=0, pad=0),
        # four prompts of odd lengths from their start, a window, small heads
        dict(name="attend prompts, window", kind="attend", seqs=4, new=2000, len=2000, ragged=0.6, heads=16,
             kv_heads=2, d=64, page=32, type="f16", cache="f16", window=1024, pad=64),
        # a long chunk of a long document
        dict(name="attend long chunk", kind="attend", seqs=1, new=2048, len=16384, ragged=0.0, heads=32, kv_heads=8,
             d=128, page=64, type="bf16", cache="bf16", window=0, pad=0),
        # prompts into an int8 cache, straight from a fp32 projection
        dict(name="store prompts", kind="store", seqs=4, new=2048, len=4096, ragged=0.4, heads=8, kv_heads=8, d=128,
             page=64, type="f32", cache="i8", window=0, pad=0),
        # conversations out of an int8 cache
        dict(name="fetch conversations", kind="fetch", seqs=3, new=0, len=8000, ragged=0.7, heads=8, kv_heads=8, d=128,
             page=64, type="bf16", cache="i8", window=0, pad=0),
        # the logit head's rows of four slots
        dict(name="probs 4 slots", kind="probs", rows=4, n=151936, type="f32", pad=0),
        # sixty-four slots with four drafted tokens each
        dict(name="probs 64 slots drafted", kind="probs", rows=320, n=151936, type="bf16", pad=0),
        # one conversation's drafted tokens
        dict(name="verify one slot", kind="verify", seqs=1, draft=4, n=151936, agree=0.7, given=True),
        # sixty-four conversations'
        dict(name="verify 64 slots", kind="verify", seqs=64, draft=4, n=151936, agree=0.7, given=True),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(["step", "step", "attend", "attend", "attend", "store", "fetch", "probs", "verify"])
    if kind == "probs":
        n = _spread(rng, 2, 200000)
        type_ = rng.choice(["f32", "f16", "bf16"])
        rows = max(1, min(_spread(rng, 1, 512), MAX_BYTES // (n * (SIZE[type_] + 4))))
        return dict(kind=kind, rows=rows, n=n, type=type_, pad=rng.choice([0, 0, 8, 1]))
    if kind == "verify":
        draft = rng.randint(1, 8)
        n = _spread(rng, 2, 200000)
        seqs = max(1, min(_spread(rng, 1, 128), MAX_PROBS // (n * (draft + 1))))
        return dict(kind=kind, seqs=seqs, draft=draft, n=n, agree=rng.choice([0.2, 0.7, 0.95]), given=rng.random() < 0.8)
    type_ = rng.choice(["f32", "f16", "bf16"])
    cache = rng.choice(["i8", "bf16" if type_ == "bf16" else "f16"])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8])
    d = rng.choice([32, 64, 64, 80, 96, 128, 128, 128, 192, 256])
    # a step takes one token or a few, an attention up to long chunks
    new = (rng.choice([1, 1, 1, 2, 3, 5, 8]) if kind == "step" else 0 if kind == "fetch" else
           rng.choice([1, 2, 5, 9, 17, _spread(rng, 32, 2048)]) if kind == "attend" else _spread(rng, 1, 4096))
    length = _spread(rng, max(1, new), max(new, 32768))
    c = dict(kind=kind, seqs=_spread(rng, 1, 64), new=new, len=length, ragged=rng.choice([0.0, 0.5, 0.95]),
             heads=heads, kv_heads=kv_heads, d=d, page=rng.choice([16, 32, 64, 128]), type=type_, cache=cache,
             window=rng.choice([0, 0, _spread(rng, 1, 4096)]) if kind in ("step", "attend") else 0,
             pad=rng.choice([0, 0, 8, 1]))
    # products in fp32 cost four times those of 16 bits
    heavy = heads * d * (4 if type_ == "f32" else 1)
    while work(c)["bytes"] > MAX_BYTES or c["seqs"] * c["new"] * c["len"] * heavy > MAX_PRODUCTS:
        if c["seqs"] > 1:
            c["seqs"] //= 2
        else:
            c["len"], c["new"] = max(1, c["len"] // 2), min(c["new"], max(1, c["new"] // 2))
    return c


def _batch(c):
    """(tokens each sequence holds, its new ones among them): the last ones are
    the shortest; a ragged batch's new tokens fall with the lengths."""
    s = c["seqs"]
    lens = [max(1, round(c["len"] * (1.0 - c["ragged"] * i / max(1, s - 1)))) for i in range(s)]
    if c["new"] <= 8:
        new = [min(c["new"], n) for n in lens]
    else:
        new = [max(1, min(n, round(c["new"] * n / c["len"]))) for n in lens]
    return lens, new


# ------------------------------------------------------------------ inputs --

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _rows(x, type_, pad):
    """`x` in its type, as rows of a buffer with `pad` values more a row."""
    x = x.to(TYPES[type_])
    if not pad:
        return x
    buf = torch.full((x.shape[0], x.shape[1] + pad), 3.0, dtype=x.dtype, device=x.device)
    buf[:, :x.shape[1]] = x
    return buf[:, :x.shape[1]]


def _empty(rows, cols, type_, pad):
    return torch.zeros((rows, cols + pad), dtype=TYPES[type_], device="cuda")[:, :cols]


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _starts(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def _inputs(c, seed):
    """What the model hands over. Sequences are kept in pages at random places
    of the cache; the keys have a few large channels, as keys have."""
    g = _generator(seed)
    if c["kind"] == "probs":
        n = c["n"]
        peaks = 9.0 * _normal(g, c["rows"], 1) * (_uniform(g, c["rows"], n) < 0.001)
        return {"logits": _rows(2.5 * _normal(g, c["rows"], n) + peaks.abs(), c["type"], c["pad"]),
                "temperature": 0.5 + _uniform(g, c["rows"])}
    if c["kind"] == "verify":
        return _drafted(c, g)
    lens, new = _batch(c)
    h, d, total = c["kv_heads"], c["d"], sum(lens)
    scale = torch.ones(d, device="cuda")
    scale[:: max(1, d // 4)] = 4.0
    s = {"k": (_normal(g, total, h, d) * scale).to(TYPES[c["type"]]),
         "v": (_normal(g, total, h, d) + 0.3 * _normal(g, 1, h, d)).to(TYPES[c["type"]])}
    # (where query heads share keys, each has a query of its own)
    s["q"] = _rows(0.6 * _normal(g, sum(new), c["heads"] * d), c["type"], c["pad"])
    pages = [-(-n // c["page"]) for n in lens]
    spare = 3                                           # pages that no sequence has
    order = torch.randperm(sum(pages) + spare, generator=g, device="cuda").to(torch.int32)
    table = torch.full((c["seqs"], max(pages)), -1, dtype=torch.int32, device="cuda")
    at = _starts(pages)
    for i in range(c["seqs"]):
        table[i, :pages[i]] = order[at[i]:at[i + 1]]
    s["table"], s["n_pages"] = table, sum(pages) + spare
    s["lens"], s["starts"], s["all"] = _ints(lens), _ints(_starts(new)), _ints(_starts(lens))
    # the new tokens among all: the last ones of each sequence
    ends = _starts(lens)[1:]
    s["fresh"] = torch.cat([torch.arange(e - n, e, device="cuda") for e, n in zip(ends, new)])
    return s


def _drafted(c, g):
    """A target's and a draft's probabilities that agree in part, tokens drawn
    from the draft's, and the random numbers that decide."""
    s, t, n = c["seqs"], c["draft"], c["n"]
    target = 3.0 * _normal(g, s, t + 1, n)
    other = 3.0 * _normal(g, s, t, n)
    a = c["agree"]
    p = torch.softmax(target, dim=2)
    q = torch.softmax(a * target[:, :t] + (1.0 - a) * other, dim=2)
    pick = torch.multinomial(q.reshape(s * t, n), 1, generator=g).reshape(s, t).to(torch.int32)
    counts = torch.full((s,), t, dtype=torch.int32, device="cuda")
    counts[1::3] = max(0, t - 1)                        # some slots had fewer to draft
    return {"p": p.reshape(s * (t + 1), n), "q": q.reshape(s * t, n) if c["given"] else None, "drafted": pick,
            "counts": counts, "accept": _uniform(g, s, t), "sample": _uniform(g, s)}


def prepare(case, seed):
    c = case
    s = _inputs(c, seed)
    s["case"] = dict(c)
    if c["kind"] == "probs":
        s["probs"] = torch.empty((c["rows"], c["n"]), device="cuda")
    elif c["kind"] == "verify":
        s["tokens"] = torch.empty((c["seqs"], c["draft"] + 1), dtype=torch.int32, device="cuda")
        s["kept"] = torch.empty(c["seqs"], dtype=torch.int32, device="cuda")
    else:
        _prepare_cache(s, c)
    return s


def _prepare_cache(s, c):
    """The new tokens' rows as the projection gives them, what is cached
    already, and the buffers of the results. What no token was written to holds
    NaN."""
    lens, new = _batch(c)
    h, d = c["kv_heads"], c["d"]
    s["new_k"] = _rows(s["k"][s["fresh"]].reshape(-1, h * d), c["type"], c["pad"])
    s["new_v"] = _rows(s["v"][s["fresh"]].reshape(-1, h * d), c["type"], c["pad"])
    cached = {"store": [n - m for n, m in zip(lens, new)], "step": [n - m for n, m in zip(lens, new)]}.get(c["kind"], lens)
    starts = _starts(lens)
    at = torch.cat([torch.arange(starts[i], starts[i] + cached[i], device="cuda") for i in range(c["seqs"])])
    old_k, old_v = s["k"][at].reshape(-1, h * d), s["v"][at].reshape(-1, h * d)
    old_lens, old_starts = _ints(cached), _ints(_starts(cached))
    rows = sum(new)
    if c["kind"] in ("step", "attend"):
        s["out"] = _empty(rows, c["heads"] * d, c["type"], c["pad"])
    else:
        rows = rows if c["kind"] == "store" else sum(lens)
        s["back_k"], s["back_v"] = _empty(rows, h * d, c["type"], 0), _empty(rows, h * d, c["type"], 0)
        s["first"] = s["lens"] - _ints(new) if c["kind"] == "store" else None
    if own:
        from q4_quantized_linear_gb300 import binding as q4
        s["q4"] = q4
        names = {"f32": q4.Q4_TYPE_F32, "f16": q4.Q4_TYPE_F16, "bf16": q4.Q4_TYPE_BF16, "i8": q4.Q4_TYPE_I8}
        s["type"], s["ctype"] = names[c["type"]], names[c["cache"]]
        nbytes = q4.q4_kv_page_size(c["page"], h, d, s["ctype"])
        s["pages"] = torch.full((s["n_pages"] * nbytes,), 255, dtype=torch.uint8, device="cuda")
        _own_write(s, old_k, old_v, old_lens, old_starts, old_k.shape[0])
        if "out" in s:
            need = q4.q4_attention_workspace_size(rows, c["seqs"], c["heads"], h, d)
            s["ws"] = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
    else:
        shape = (s["n_pages"] * c["page"], h, d)
        for x in ("k", "v"):
            if c["cache"] == "i8":
                s["c" + x] = torch.full(shape, -1, dtype=torch.int8, device="cuda")
                s["s" + x] = torch.full(shape[:2], float("nan"), device="cuda")
            else:
                s["c" + x] = torch.full(shape, float("nan"), dtype=TYPES[c["cache"]], device="cuda")
        if old_k.shape[0]:
            _plain_write(s, old_k, old_v, old_lens, old_starts)
    del s["k"], s["v"]


# --------------------------------------------------------------------- run --

def run(s):
    return _OWN[s["case"]["kind"]](s) if own else _PLAIN[s["case"]["kind"]](s)


def _own_write(s, k, v, lens, starts, rows):
    c = s["case"]
    s["q4"].q4_kv_write(s["pages"], s["n_pages"], c["page"], c["kv_heads"], c["d"], s["ctype"], s["table"],
                        s["table"].stride(0), lens, starts, c["seqs"], k, k.stride(0), v, v.stride(0), s["type"], rows)


def _own_read(s, first, starts):
    c, k, v = s["case"], s["back_k"], s["back_v"]
    s["q4"].q4_kv_read(k, k.stride(0), v, v.stride(0), s["type"], s["pages"], s["n_pages"], c["page"], c["kv_heads"],
                       c["d"], s["ctype"], s["table"], s["table"].stride(0), first, starts, c["seqs"], k.shape[0])
    return {"k": k, "v": v}


def _own_attend(s):
    c, q, o = s["case"], s["q"], s["out"]
    s["q4"].q4_attention(o, o.stride(0), q, q.stride(0), s["type"], c["heads"], c["d"] ** -0.5, c["window"], s["pages"],
                         s["n_pages"], c["page"], c["kv_heads"], c["d"], s["ctype"], s["table"], s["table"].stride(0),
                         s["lens"], s["starts"], c["seqs"], q.shape[0], c["new"], s["ws"], s["ws"].numel())
    return o


def _own_step(s):
    _own_write(s, s["new_k"], s["new_v"], s["lens"], s["starts"], s["new_k"].shape[0])
    return _own_attend(s)


def _own_store(s):
    _own_write(s, s["new_k"], s["new_v"], s["lens"], s["starts"], s["new_k"].shape[0])
    return _own_read(s, s["first"], s["starts"])


def _own_fetch(s):
    return _own_read(s, None, s["all"])


def _own_probs(s):
    from q4_quantized_linear_gb300 import binding as q4
    c, x = s["case"], s["logits"]
    ty = {"f32": q4.Q4_TYPE_F32, "f16": q4.Q4_TYPE_F16, "bf16": q4.Q4_TYPE_BF16}[c["type"]]
    q4.q4_token_probs(s["probs"], c["n"], x, x.stride(0), ty, s["temperature"], c["rows"], c["n"])
    return s["probs"]


def _own_verify(s):
    from q4_quantized_linear_gb300 import binding as q4
    c = s["case"]
    q4.q4_draft_verify(s["tokens"], c["draft"] + 1, s["kept"], s["p"], c["n"], s["q"], c["n"], s["drafted"], c["draft"],
                       s["counts"], s["accept"], c["draft"], s["sample"], c["seqs"], c["draft"], c["n"])
    return {"tokens": s["tokens"], "kept": s["kept"]}


_OWN = {"step": _own_step, "attend": _own_attend, "store": _own_store, "fetch": _own_fetch, "probs": _own_probs,
        "verify": _own_verify}


def _codes(x):
    """Symmetric int8 codes of each row and its scale, every step one fp32
    operation."""
    amax = x.abs().amax(dim=-1, keepdim=True)
    top = torch.full_like(amax, 127.0)    # a tensor: a number would be divided by way of its reciprocal
    inv = torch.where(amax > 0, top / amax, torch.zeros_like(amax))
    return torch.round(x * inv).to(torch.int8), (amax / top).squeeze(-1)


def _places(s, first, starts, rows):
    """The place in the cache of each row of a ragged batch whose sequence s
    has its rows at positions first[s] and on."""
    c = s["case"]
    row = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(starts.to(torch.int64), row, right=True) - 1
    pos = first.to(torch.int64)[seq] + row - starts.to(torch.int64)[seq]
    return s["table"][seq, pos // c["page"]].to(torch.int64) * c["page"] + pos % c["page"]


def _plain_write(s, k, v, lens, starts):
    c = s["case"]
    first = lens - (starts[1:] - starts[:-1])
    at = _places(s, first, starts, k.shape[0])
    for name, x in (("k", k), ("v", v)):
        x = x.reshape(-1, c["kv_heads"], c["d"]).float()
        if c["cache"] == "i8":
            s["c" + name][at], s["s" + name][at] = _codes(x)
        else:
            s["c" + name][at] = x.to(TYPES[c["cache"]])


def _plain_values(s, name, at):
    """The cache's values at these places, in fp32."""
    x = s["c" + name][at].float()
    return x * s["s" + name][at][..., None] if s["case"]["cache"] == "i8" else x


def _plain_attend(s):
    c = s["case"]
    h, d, group = c["kv_heads"], c["d"], c["heads"] // c["kv_heads"]
    lens, new = _batch(c)
    most, width, seqs = max(lens), max(new), c["seqs"]
    length, starts = s["lens"].to(torch.int64), s["starts"].to(torch.int64)
    count = starts[1:] - starts[:-1]
    pos = torch.arange(most, device="cuda")
    held = pos[None, :] < length[:, None]                                        # [seqs, most]
    at = s["table"][:, pos // c["page"]].to(torch.int64) * c["page"] + pos % c["page"]
    at = torch.where(held, at, torch.zeros_like(at))
    zero = torch.zeros((), device="cuda")
    k = torch.where(held[..., None, None], _plain_values(s, "k", at), zero).transpose(1, 2)   # [seqs, h, most, d]
    v = torch.where(held[..., None, None], _plain_values(s, "v", at), zero).transpose(1, 2)
    i = torch.arange(width, device="cuda")
    row = torch.minimum(starts[:-1, None] + i[None, :], starts[1:, None] - 1)    # [seqs, width], padded
    q = s["q"][row].float().reshape(seqs, width, h, group, d).permute(0, 2, 1, 3, 4).reshape(seqs, h, width * group, d)
    score = torch.matmul(q, k.transpose(2, 3)) * (d ** -0.5)
    mine = length[:, None] - count[:, None] + i[None, :]                         # a new token's position
    sees = (pos[None, None, :] <= mine[:, :, None]) & held[:, None, :]
    if c["window"]:
        sees &= pos[None, None, :] > mine[:, :, None] - c["window"]
    sees = sees[:, None, :, None, :].expand(seqs, 1, width, group, most).reshape(seqs, 1, width * group, most)
    score.masked_fill_(~sees, float("-inf"))
    top = score.amax(dim=-1, keepdim=True)
    e = torch.exp_(score.sub_(torch.where(top == float("-inf"), zero, top)))
    o = torch.matmul(e, v) / e.sum(dim=-1, keepdim=True)
    o = o.reshape(seqs, h, width, group, d).permute(0, 2, 1, 3, 4).reshape(seqs, width, c["heads"] * d)
    s["out"].copy_(o[i[None, :] < count[:, None]])
    return s["out"]


def _plain_step(s):
    _plain_write(s, s["new_k"], s["new_v"], s["lens"], s["starts"])
    return _plain_attend(s)


def _plain_read(s, first, starts):
    c, rows = s["case"], s["back_k"].shape[0]
    at = _places(s, first, starts, rows)
    ty = TYPES[c["type"]]
    return {"k": _plain_values(s, "k", at).to(ty).reshape(rows, -1), "v": _plain_values(s, "v", at).to(ty).reshape(rows, -1)}


def _plain_store(s):
    _plain_write(s, s["new_k"], s["new_v"], s["lens"], s["starts"])
    return _plain_read(s, s["first"], s["starts"])


def _plain_fetch(s):
    return _plain_read(s, torch.zeros_like(s["lens"]), s["all"])


def _plain_probs(s):
    x = s["logits"].float() / s["temperature"][:, None]
    e = torch.exp(x - x.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _plain_verify(s):
    """A drafted token x stays while u q(x) < p(x); the first that does not is
    replaced by a draw from what p has more than q, and after the last one a
    token is drawn from p."""
    c, D = s["case"], torch.float64
    seqs, t, n = c["seqs"], c["draft"], c["n"]
    p, drafted = s["p"].reshape(seqs, t + 1, n), s["drafted"].to(torch.int64)
    px = p[:, :t].gather(2, drafted[:, :, None]).squeeze(2).to(D)
    if c["given"]:
        q = s["q"].reshape(seqs, t, n)
        qx = q.gather(2, drafted[:, :, None]).squeeze(2).to(D)
    else:
        qx = torch.ones_like(px)                        # the draft was sure of its token
    i = torch.arange(t, device="cuda")
    stays = (s["accept"].to(D) * qx < px) & (i[None, :] < s["counts"][:, None])
    kept = torch.cumprod(stays.to(torch.int64), dim=1).sum(dim=1)
    slot = torch.arange(seqs, device="cuda")
    left = p[slot, kept].to(D)
    refused = kept < s["counts"]
    at = torch.minimum(kept, torch.full_like(kept, t - 1))
    if c["given"]:
        less = q[slot, at].to(D)
    else:
        less = torch.zeros_like(left)
        less[slot, drafted[slot, at]] = 1.0
    rest = torch.where(refused[:, None], (left - less).clamp(min=0.0), left)
    total = rest.sum(dim=1, keepdim=True)
    rest = torch.where(total > 0, rest, left)
    run_ = torch.cumsum(rest, dim=1)
    above = run_ > s["sample"].to(D)[:, None] * run_[:, -1:]
    drawn = above.to(torch.uint8).argmax(dim=1)
    j = torch.arange(t + 1, device="cuda")[None, :]
    wide = torch.cat([drafted, torch.zeros((seqs, 1), dtype=drafted.dtype, device="cuda")], dim=1)
    tokens = torch.where(j < kept[:, None], wide, torch.where(j == kept[:, None], drawn[:, None], torch.full_like(wide, -1)))
    return {"tokens": tokens.to(torch.int32), "kept": kept.to(torch.int32)}


_PLAIN = {"step": _plain_step, "attend": _plain_attend, "store": _plain_store, "fetch": _plain_fetch,
          "probs": _plain_probs, "verify": _plain_verify}


# -------------------------------------------------------------------- work --

def work(case):
    """Every input read once, every output written once; the products and sums."""
    c = case
    if c["kind"] == "probs":
        return {"bytes": c["rows"] * c["n"] * (SIZE[c["type"]] + 4), "flops": 4 * c["rows"] * c["n"]}
    if c["kind"] == "verify":
        # the row that is drawn from, of the target's and the draft's
        return {"bytes": c["seqs"] * c["n"] * 4 * (2 if c["given"] else 1), "flops": 3 * c["seqs"] * c["n"]}
    lens, new = _batch(c)
    h, d, z = c["kv_heads"], c["d"], SIZE[c["type"]]
    token = 2 * h * (d * SIZE[c["cache"]] + (4 if c["cache"] == "i8" else 0))     # of the cache
    if c["kind"] == "store":
        return {"bytes": sum(new) * (4 * h * d * z + 2 * token), "flops": 6 * sum(new) * h * d}
    if c["kind"] == "fetch":
        return {"bytes": sum(lens) * (2 * h * d * z + token), "flops": 2 * sum(lens) * h * d}
    seen = pairs = 0
    for n, m in zip(lens, new):
        if c["window"]:
            w = c["window"]
            seen += min(n, m - 1 + w)
            # sum over the new tokens' positions p of min(p + 1, w)
            lo, hi = n - m + 1, n
            full = max(0, hi - max(lo, w) + 1)
            pairs += full * w + (lo + hi - full) * (m - full) // 2
        else:
            seen += n
            pairs += m * (n - m) + m * (m + 1) // 2
    nbytes = seen * token + 2 * sum(new) * c["heads"] * d * z
    if c["kind"] == "step":
        nbytes += sum(new) * 2 * h * d * z              # what it caches is read from the rows
    return {"bytes": nbytes, "flops": 4 * pairs * c["heads"] * d}


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    """The definitions in 64 bits. What the cache holds follows the coding rule's
    own fp32 steps, or one rounding to the cache's type."""
    c = case
    s = _inputs(c, seed)
    D = torch.float64
    if c["kind"] == "verify":
        return None                                     # whole numbers
    if c["kind"] == "probs":
        out = []
        for i in range(c["rows"]):
            z = s["logits"][i].to(D) / s["temperature"][i].to(D)
            out.append((z - torch.logsumexp(z, dim=0)).exp())
        return torch.stack(out)
    lens, new = _batch(c)
    h, d, group = c["kv_heads"], c["d"], c["heads"] // c["kv_heads"]
    ends = _starts(lens)

    def held(x):
        """A sequence's tokens of a head as the cache gives them back."""
        x = x.float()
        if c["cache"] != "i8":
            return x.to(TYPES[c["cache"]]).to(D)
        top = x.abs().max(dim=-1, keepdim=True).values
        factor = torch.where(top == 0, torch.zeros_like(top), torch.full_like(top, 127.0) / top)
        return (x * factor).round().to(D) * (top / torch.full_like(top, 127.0)).to(D)

    if c["kind"] in ("store", "fetch"):
        parts = {"k": [], "v": []}
        for i in range(c["seqs"]):
            lo = ends[i + 1] - new[i] if c["kind"] == "store" else ends[i]
            for name in parts:
                parts[name].append(held(s[name][lo:ends[i + 1]]).reshape(ends[i + 1] - lo, h * d))
        return {name: torch.cat(v) for name, v in parts.items()}
    if 8 * 4 * c["heads"] * d * sum(n * m for n, m in zip(lens, new)) > 8e12:
        return None
    q = s["q"].to(D)
    out = torch.zeros((sum(new), c["heads"] * d), dtype=D, device=q.device)
    row = 0
    for i in range(c["seqs"]):
        n, m = lens[i], new[i]
        mine = torch.arange(n - m, n, device=q.device).unsqueeze(1)
        theirs = torch.arange(n, device=q.device).unsqueeze(0)
        hidden = theirs > mine
        if c["window"]:
            hidden |= theirs <= mine - c["window"]
        for j in range(h):
            keys, values = (held(s[x][ends[i]:ends[i + 1], j]) for x in ("k", "v"))
            for b in range(j * group, (j + 1) * group):
                z = q[row:row + m, b * d:(b + 1) * d] @ keys.t() / math.sqrt(d)
                z[hidden] = -math.inf
                out[row:row + m, b * d:(b + 1) * d] = (z - torch.logsumexp(z, dim=1, keepdim=True)).exp() @ values
        row += m
    return out
