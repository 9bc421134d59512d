"""Cases of the operators around the quantised linear layers: what is timed,
the plain form of each, and its value in 64 bits.

A transformer block of the models this library serves is a norm, a linear
layer over quantised weights or a mixture of such layers, and a norm again:

  linear            X coded per token to int8, times per-channel int8 weights
  norm_linear       the norm before a block written as int8 codes, times such
                    weights (the decode step of a block's first projection)
  norm_join         the norm after a block, with its gate, the residual scale
                    and the residual sum, and the next block's norm, in one pass
  norm_before_bwd   the gradient of the norm before a block, with the residual
                    stream's gradient added
  norm_after_bwd    the gradient of the norm after a block: of the block's
                    output, the norm's weights and the gate
  dispatch          tokens sorted by expert, their rows copied in that order
  combine           the experts' rows back in token order, weighted and summed
  combine_bwd       the gradient of combine: of the experts' rows and weights

Plain forms: elementary torch operations in fp32, rounded once at the end.
"""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6

# The largest cases; a drawn case stays within them.
MAX_MACS = 4096 * 14336 * 4096
MAX_WEIGHTS = 14336 * 4096
MAX_NORM = 8192 * 4096
MAX_PAIRS = 8192 * 8 * 4096


def listed():
    return [
        # a single conversation's decode step: one token through a
        # feed-forward projection, fp32 as the other products of the library
        dict(name="linear one token", kind="linear", m=1, n=9728, k=2560, type="f32", pad=0),
        # sixteen conversations' tokens in one decode step, norm first
        dict(name="norm and linear, 16 slots", kind="norm_linear", m=16, n=14336, k=4096, type="bf16", pad=0),
        # a prompt of 540 tokens through the same projection
        dict(name="linear prompt", kind="linear", m=540, n=9728, k=2560, type="f32", pad=0),
        # several prompts in one pass, the widest projection
        dict(name="linear prompts", kind="linear", m=4096, n=14336, k=4096, type="bf16", pad=0),
        # between two blocks of one token's decode step
        dict(name="norm join one token", kind="norm_join", m=1, d=2560, type="f32", gate="channel", pad=0),
        # between two blocks of a long prompt, a gate of its own for each value
        dict(name="norm join prompts", kind="norm_join", m=4096, d=4096, type="bf16", gate="full", pad=0),
        # tuning the norms of a model whose weights stay quantised: an odd batch in fp32
        dict(name="norm before, backward", kind="norm_before_bwd", m=2049, d=2560, type="f32", pad=0),
        # the same on a large batch, the gate shared by all tokens
        dict(name="norm after, backward", kind="norm_after_bwd", m=8192, d=4096, type="bf16", gate="channel", pad=0),
        # a mixture layer's decode step: one token, eight of 128 experts
        dict(name="dispatch one token", kind="dispatch", t=1, k=8, e=128, d=2560, type="f32", ids=64, drop=0.0, pad=0),
        # prompts through a mixture layer, some tokens padding or over capacity
        dict(name="dispatch prompts", kind="dispatch", t=8192, k=8, e=128, d=4096, type="bf16", ids=64, drop=0.02, pad=0),
        # the experts' rows back, next to a shared expert's output
        dict(name="combine prompt", kind="combine", t=4099, k=4, e=32, d=2560, type="f32", drop=0.02, base=True, pad=0),
        # and their gradient in a training step
        dict(name="combine, backward", kind="combine_bwd", t=4096, k=8, e=128, d=4096, type="bf16", drop=0.02, pad=0),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(["linear", "linear", "norm_linear", "norm_join", "norm_before_bwd", "norm_after_bwd",
                       "dispatch", "dispatch", "combine", "combine_bwd"])
    type_ = rng.choice(["f32", "f16", "bf16"])
    pad = rng.choice([0, 0, 8, 1])   # values between two rows beyond their own
    if kind in ("linear", "norm_linear"):
        if kind == "norm_linear" and type_ == "f32":
            type_ = "bf16"           # codes of a norm differ in their last place by the order of its sum
        k = 32 * _spread(rng, 1, 448)
        n = _spread(rng, 1, min(151936, MAX_WEIGHTS // k))
        m = _spread(rng, 1, 4096)
        m = max(1, min(m, MAX_MACS // (n * k), 67108864 // n))
        return dict(kind=kind, m=m, n=n, k=k, type=type_, pad=8 if pad else 0)
    if kind.startswith("norm"):
        d = _spread(rng, 32, 16384)
        m = max(1, min(_spread(rng, 1, 16384), MAX_NORM // d))
        c = dict(kind=kind, m=m, d=d, type=type_, pad=pad)
        if kind != "norm_before_bwd":
            c["gate"] = rng.choice(["none", "channel", "token", "full"])
        return c
    e = _spread(rng, 2, 512)
    k = rng.randint(1, min(8, e))
    d = _spread(rng, 32, 8192)
    t = max(1, min(_spread(rng, 1, 16384), MAX_PAIRS // (k * d * (1 if type_ != "f32" else 2))))
    c = dict(kind=kind, t=t, k=k, e=e, d=d, type=type_, drop=rng.choice([0.0, 0.02, 0.3]), pad=pad)
    if kind == "dispatch":
        c["ids"] = rng.choice([32, 64])
    if kind == "combine":
        c["base"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------ inputs --

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rows(x, type_, pad):
    """`x` in its type, as rows of a buffer with `pad` values more a row."""
    x = x.to(TYPES[type_])
    if not pad:
        return x
    buf = torch.full((x.shape[0], x.shape[1] + pad), 3.0, dtype=x.dtype, device=x.device)
    buf[:, :x.shape[1]] = x
    return buf[:, :x.shape[1]]


def _empty(m, d, type_, pad):
    return torch.empty((m, d + pad), dtype=TYPES[type_], device="cuda")[:, :d]


def _hidden(g, m, d):
    """A residual stream: tokens of different sizes, a few large channels."""
    x = _normal(g, m, d) * (0.5 + 2.0 * torch.rand(m, 1, generator=g, device="cuda"))
    x[:, :: max(1, d // 5)] *= 8.0
    return x


def _codes(w):
    """Symmetric int8 codes and scale of each row: the coding of the weights
    and of the tokens, every step one fp32 operation."""
    amax = w.abs().amax(dim=1, keepdim=True)
    top = torch.full_like(amax, 127.0)    # a tensor: a number would be divided by way of its reciprocal
    inv = torch.where(amax > 0, top / amax, torch.zeros_like(amax))
    return torch.round(w * inv).to(torch.int8), (amax / top).squeeze(1)


def _router(g, case):
    """Expert ids and weights as a router gives them: the top k of skewed
    scores, softmax weights; padding tokens and pairs over capacity are -1."""
    t, k, e = case["t"], case["k"], case["e"]
    scores = _normal(g, t, e) + 1.5 * _normal(g, e)
    top = torch.topk(scores, k, dim=1)
    ids = top.indices
    weights = torch.softmax(top.values, dim=1)
    if case["drop"] > 0:
        gone = torch.rand(t, k, generator=g, device="cuda") < case["drop"] / 2
        gone |= torch.rand(t, 1, generator=g, device="cuda") < case["drop"] / 2
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return ids, weights.contiguous()


def _inputs(case, seed):
    g, c = _generator(seed), case
    kind, type_, pad = c["kind"], c["type"], c["pad"]
    s = {}
    if kind in ("linear", "norm_linear"):
        s["W"] = _normal(g, c["n"], c["k"]) * (0.02 * (0.5 + torch.rand(c["n"], 1, generator=g, device="cuda")))
        s["X"] = _rows(_hidden(g, c["m"], c["k"]), type_, pad)
        if kind == "norm_linear":
            s["w"] = 1.0 + 0.2 * _normal(g, c["k"])
        return s
    if kind.startswith("norm"):
        m, d = c["m"], c["d"]
        if kind == "norm_before_bwd":
            s["X"] = _rows(_hidden(g, m, d), type_, pad)
            s["w"] = 0.2 * _normal(g, d)                      # the model holds the weight's distance from 1
            s["dH"] = _rows(_normal(g, m, d), type_, pad)
            s["dR"] = _rows(_normal(g, m, d), type_, pad)
            return s
        s["B"] = _rows(_hidden(g, m, d), type_, pad)
        s["w"] = 1.0 + 0.2 * _normal(g, d)
        gate = c["gate"]
        s["gate"] = (None if gate == "none" else 0.5 + 0.5 * _normal(g, d) if gate == "channel" else
                     torch.sigmoid(_normal(g, m)) if gate == "token" else
                     _rows(torch.sigmoid(_normal(g, m, d)), type_, pad))
        if kind == "norm_join":
            s["R"] = _rows(_hidden(g, m, d), type_, pad)
            s["w_next"] = 1.0 + 0.2 * _normal(g, d)
        else:
            s["dY"] = _rows(_normal(g, m, d), type_, pad)
        return s
    t, k, d = c["t"], c["k"], c["d"]
    ids, s["weights"] = _router(g, c)
    if kind == "dispatch":
        s["ids"] = ids if c["ids"] == 64 else ids.to(torch.int32)
        s["X"] = _rows(_hidden(g, t, d), type_, pad)
        return s
    s["row_of"] = _sorted_rows(ids, c["e"])[1]
    rows = _normal(g, t * k, d)
    kept = (s["row_of"] >= 0).sum()
    rows[torch.arange(t * k, device="cuda") >= kept] = float("nan")   # rows that no expert wrote
    s["Ys"] = _rows(rows, type_, pad)
    if kind == "combine":
        s["base"] = _rows(_normal(g, t, d), type_, pad) if c["base"] else None
    else:
        s["dY"] = _rows(_normal(g, t, d), type_, pad)
    return s


def _sorted_rows(ids, experts):
    """offsets [e + 1]; row_of [t, k]: the row of each pair, -1 - row where the
    pair has no expert (its row then is one of those after the last expert's);
    pair_of: the pair at each row."""
    flat = ids.reshape(-1).to(torch.int64)
    valid = (flat >= 0) & (flat < experts)
    key = torch.where(valid, flat, torch.full_like(flat, experts))
    pair_of = torch.argsort(key, stable=True)
    row = torch.empty_like(pair_of)
    row[pair_of] = torch.arange(flat.numel(), device=flat.device)
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=flat.device)
    counts.index_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = torch.cumsum(counts[:experts], 0)
    row_of = torch.where(valid, row, -1 - row).to(torch.int32).reshape(ids.shape)
    return offsets, row_of, pair_of.to(torch.int32)


def prepare(case, seed):
    s = _inputs(case, seed)
    c = case
    s["case"] = dict(c)
    if c["kind"] in ("linear", "norm_linear"):
        s["codes"], s["scales"] = _codes(s["W"])
    if own:
        _prepare_own(s, c)
    s.pop("W", None)
    return s


def _prepare_own(s, c):
    """What a program of the library keeps: packed weights, output buffers and
    workspaces."""
    from q4_quantized_linear_gb300 import binding as q4
    s["q4"] = q4
    s["type"] = {"f32": q4.Q4_TYPE_F32, "f16": q4.Q4_TYPE_F16, "bf16": q4.Q4_TYPE_BF16}[c["type"]]
    kind, type_, pad = c["kind"], c["type"], c["pad"]

    def workspace(nbytes):
        return torch.empty(max(1, nbytes), dtype=torch.uint8, device="cuda"), nbytes

    if kind in ("linear", "norm_linear"):
        m, n, k = c["m"], c["n"], c["k"]
        s["packed"] = torch.empty(q4.q4_w8_packed_size(n, k), dtype=torch.uint8, device="cuda")
        q4.q4_w8_quantize(s["packed"], s["W"].contiguous(), n, k)
        s["Y"] = _empty(m, n, type_, 0)
        s["ws"], s["ws_bytes"] = workspace(q4.q4_w8a8_workspace_size(m, k, n))
        if kind == "norm_linear":
            s["H"] = torch.empty((m, k), dtype=torch.int8, device="cuda")
            s["h_scale"] = torch.empty(m, dtype=torch.float32, device="cuda")
        torch.cuda.current_stream().synchronize()
    elif kind.startswith("norm"):
        m, d = c["m"], c["d"]
        s["gate_kind"] = {"none": q4.Q4_GATE_NONE, "channel": q4.Q4_GATE_CHANNEL, "token": q4.Q4_GATE_TOKEN,
                          "full": q4.Q4_GATE_FULL}[c.get("gate", "none")]
        if kind == "norm_join":
            s["Y"], s["H"] = _empty(m, d, type_, pad), _empty(m, d, type_, pad)
            return
        s["ws"], s["ws_bytes"] = workspace(q4.q4_norm_workspace_size(m, d))
        s["dw"] = torch.empty(d, dtype=torch.float32, device="cuda")
        if kind == "norm_before_bwd":
            s["dX"] = _empty(m, d, type_, pad)
            return
        s["dB"] = _empty(m, d, type_, pad)
        gate = c["gate"]
        s["dgate"] = (None if gate == "none" else torch.empty(d, device="cuda") if gate == "channel" else
                      torch.empty(m, device="cuda") if gate == "token" else _empty(m, d, type_, pad))
    else:
        t, k, d = c["t"], c["k"], c["d"]
        if kind == "dispatch":
            s["Xs"] = _empty(t * k, d, type_, pad)
            s["offsets"] = torch.empty(c["e"] + 1, dtype=torch.int64, device="cuda")
            s["row_of"] = torch.empty((t, k), dtype=torch.int32, device="cuda")
            s["pair_of"] = torch.empty(t * k, dtype=torch.int32, device="cuda")
            s["ws"], s["ws_bytes"] = workspace(q4.q4_moe_workspace_size(t, k, c["e"]))
        elif kind == "combine":
            s["Y"] = _empty(t, d, type_, pad)
        else:
            s["dYs"] = _empty(t * k, d, type_, pad)
            s["dweights"] = torch.empty((t, k), dtype=torch.float32, device="cuda")


# --------------------------------------------------------------------- run --

SCALE = 0.7       # the residual scale
OFFSET = 1.0      # what the model adds to the weights of the norm before


def run(s):
    return _OWN[s["case"]["kind"]](s) if own else _PLAIN[s["case"]["kind"]](s)


def _ld(x):
    return 0 if x is None else x.stride(0)


def _own_linear(s):
    c, q4, X, Y, ty = s["case"], s["q4"], s["X"], s["Y"], s["type"]
    q4.q4_w8a8_matmul(s["packed"], X, X.stride(0), ty, Y, c["n"], ty, c["m"], c["k"], c["n"], s["ws"], s["ws_bytes"])
    return Y


def _own_norm_linear(s):
    c, q4, X, Y, ty = s["case"], s["q4"], s["X"], s["Y"], s["type"]
    m, n, k = c["m"], c["n"], c["k"]
    q4.q4_norm_before(s["H"], k, q4.Q4_TYPE_I8, s["h_scale"], X, X.stride(0), ty, s["w"], 0.0, EPS, m, k)
    q4.q4_w8a8_matmul_codes(s["packed"], s["H"], s["h_scale"], Y, n, ty, m, k, n, s["ws"], s["ws_bytes"])
    return Y


def _own_norm_join(s):
    c, q4, Y, H, R, B, g, ty = s["case"], s["q4"], s["Y"], s["H"], s["R"], s["B"], s["gate"], s["type"]
    ldg = g.stride(0) if s["gate_kind"] == q4.Q4_GATE_FULL else 0
    q4.q4_norm_after_before(Y, Y.stride(0), H, H.stride(0), ty, None, R, R.stride(0), B, B.stride(0), ty, s["w"], 0.0,
                            g, ldg, s["gate_kind"], SCALE, s["w_next"], 0.0, EPS, c["m"], c["d"])
    return {"y": Y, "h": H}


def _own_norm_before_bwd(s):
    c, q4, dX, dH, dR, X, ty = s["case"], s["q4"], s["dX"], s["dH"], s["dR"], s["X"], s["type"]
    q4.q4_norm_before_backward(dX, dX.stride(0), s["dw"], dH, dH.stride(0), dR, dR.stride(0), X, X.stride(0), ty,
                               s["w"], OFFSET, EPS, c["m"], c["d"], s["ws"], s["ws_bytes"])
    return {"dx": dX, "dw": s["dw"]}


def _own_norm_after_bwd(s):
    c, q4, dB, dY, B, g, dg, ty = s["case"], s["q4"], s["dB"], s["dY"], s["B"], s["gate"], s["dgate"], s["type"]
    full = s["gate_kind"] == q4.Q4_GATE_FULL
    q4.q4_norm_after_backward(dB, dB.stride(0), s["dw"], dg, dg.stride(0) if full else 0, dY, dY.stride(0), B,
                              B.stride(0), ty, s["w"], 0.0, g, g.stride(0) if full else 0, s["gate_kind"], SCALE, EPS,
                              c["m"], c["d"], s["ws"], s["ws_bytes"])
    out = {"db": dB, "dw": s["dw"]}
    if dg is not None:
        out["dgate"] = dg
    return out


def _own_dispatch(s):
    c, q4, Xs, X, ids = s["case"], s["q4"], s["Xs"], s["X"], s["ids"]
    q4.q4_moe_dispatch(Xs, Xs.stride(0), s["offsets"], s["row_of"], s["pair_of"], ids, c["ids"] // 8, X, X.stride(0),
                       s["type"], c["t"], c["k"], c["e"], c["d"], s["ws"], s["ws_bytes"])
    return {"offsets": s["offsets"], "row_of": s["row_of"], "pair_of": s["pair_of"], "xs": Xs}


def _own_combine(s):
    c, q4, Y, base, Ys = s["case"], s["q4"], s["Y"], s["base"], s["Ys"]
    q4.q4_moe_combine(Y, Y.stride(0), base, _ld(base), Ys, Ys.stride(0), s["type"], s["row_of"], s["weights"], c["t"],
                      c["k"], c["d"])
    return Y


def _own_combine_bwd(s):
    c, q4, dYs, dY, Ys = s["case"], s["q4"], s["dYs"], s["dY"], s["Ys"]
    q4.q4_moe_combine_backward(dYs, dYs.stride(0), s["dweights"], dY, dY.stride(0), Ys, Ys.stride(0), s["type"],
                               s["row_of"], s["weights"], c["t"], c["k"], c["d"])
    return {"dys": dYs, "dweights": s["dweights"]}


_OWN = {"linear": _own_linear, "norm_linear": _own_norm_linear, "norm_join": _own_norm_join,
        "norm_before_bwd": _own_norm_before_bwd, "norm_after_bwd": _own_norm_after_bwd, "dispatch": _own_dispatch,
        "combine": _own_combine, "combine_bwd": _own_combine_bwd}


def _product(xq, sx, s):
    y = xq.float() @ s["codes"].float().t()
    return (y * (sx[:, None] * s["scales"][None, :])).to(TYPES[s["case"]["type"]])


def _plain_linear(s):
    xq, sx = _codes(s["X"].float())
    return _product(xq, sx, s)


def _unit(x):
    """x over its root mean square, and the reciprocal of that."""
    r = torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS)
    return x * r, r


def _plain_norm_linear(s):
    xq, sx = _codes(_unit(s["X"].float())[0] * s["w"])
    return _product(xq, sx, s)


def _gate32(s):
    g, gate = s["gate"], s["case"]["gate"]
    if gate == "none":
        return 1.0
    return g[None, :] if gate == "channel" else g[:, None] if gate == "token" else g.float()


def _plain_norm_join(s):
    ty = TYPES[s["case"]["type"]]
    y = (s["R"].float() + SCALE * _gate32(s) * (_unit(s["B"].float())[0] * s["w"])).to(ty)
    h = _unit(y.float())[0] * s["w_next"]
    return {"y": y, "h": h.to(ty)}


def _unit_grad(u, r, dn):
    """The gradient of x for n = x r: `dn` is n's, u = n."""
    return r * (dn - u * (dn * u).mean(dim=1, keepdim=True))


def _plain_norm_before_bwd(s):
    x, dh = s["X"].float(), s["dH"].float()
    u, r = _unit(x)
    dx = s["dR"].float() + _unit_grad(u, r, dh * (OFFSET + s["w"]))
    return {"dx": dx.to(TYPES[s["case"]["type"]]), "dw": (dh * u).sum(dim=0)}


def _plain_norm_after_bwd(s):
    ty, gate = TYPES[s["case"]["type"]], s["case"]["gate"]
    dn, g = SCALE * s["dY"].float(), _gate32(s)
    u, r = _unit(s["B"].float())
    out = {"db": _unit_grad(u, r, dn * g * s["w"]).to(ty), "dw": (dn * g * u).sum(dim=0)}
    if gate != "none":
        dg = dn * u * s["w"]
        out["dgate"] = dg.sum(dim=0) if gate == "channel" else dg.sum(dim=1) if gate == "token" else dg.to(ty)
    return out


def _plain_dispatch(s):
    c = s["case"]
    offsets, row_of, pair_of = _sorted_rows(s["ids"], c["e"])
    at = pair_of.to(torch.int64)
    kept = row_of.reshape(-1)[at] >= 0
    xs = s["X"][torch.div(at, c["k"], rounding_mode="floor")]
    xs = torch.where(kept[:, None], xs, torch.zeros((), dtype=xs.dtype, device=xs.device))
    return {"offsets": offsets, "row_of": row_of, "pair_of": pair_of, "xs": xs}


def _plain_combine(s):
    row_of = s["row_of"].to(torch.int64)
    v = s["Ys"].float()[row_of.clamp(min=0)] * s["weights"][:, :, None]
    y = torch.where((row_of >= 0)[:, :, None], v, torch.zeros((), device=v.device)).sum(dim=1)
    if s["base"] is not None:
        y = y + s["base"].float()
    return y.to(TYPES[s["case"]["type"]])


def _plain_combine_bwd(s):
    c = s["case"]
    row_of = s["row_of"].to(torch.int64)
    kept = row_of >= 0
    row = torch.where(kept, row_of, -1 - row_of)
    zero = torch.zeros((), device=row.device)
    dy = s["dY"].float()[:, None, :]
    g = torch.where(kept[:, :, None], dy * s["weights"][:, :, None], zero)
    dys = torch.empty((c["t"] * c["k"], c["d"]), dtype=TYPES[c["type"]], device=row.device)
    dys[row.reshape(-1)] = g.reshape(-1, c["d"]).to(dys.dtype)
    dw = torch.where(kept, (dy * s["Ys"].float()[row]).sum(dim=2), zero)
    return {"dys": dys, "dweights": dw}


_PLAIN = {"linear": _plain_linear, "norm_linear": _plain_norm_linear, "norm_join": _plain_norm_join,
          "norm_before_bwd": _plain_norm_before_bwd, "norm_after_bwd": _plain_norm_after_bwd,
          "dispatch": _plain_dispatch, "combine": _plain_combine, "combine_bwd": _plain_combine_bwd}


# -------------------------------------------------------------------- work --

def work(case):
    """Every input read once, every output written once; the products and sums."""
    c = case
    kind, z = c["kind"], SIZE[c["type"]]
    if kind in ("linear", "norm_linear"):
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": n * k + 4 * n + z * (m * k + m * n) + (4 * k if kind == "norm_linear" else 0),
                "flops": 2 * m * n * k}
    if kind.startswith("norm"):
        m, d, gate = c["m"], c["d"], c.get("gate", "none")
        g = {"none": 0, "channel": 4 * d, "token": 4 * m, "full": z * m * d}[gate]
        if kind == "norm_join":
            return {"bytes": 4 * m * d * z + g + 8 * d, "flops": 10 * m * d}
        if kind == "norm_before_bwd":
            return {"bytes": 4 * m * d * z + 8 * d, "flops": 10 * m * d}
        return {"bytes": 3 * m * d * z + 2 * g + 8 * d, "flops": 12 * m * d}
    t, k, d = c["t"], c["k"], c["d"]
    if kind == "dispatch":
        return {"bytes": t * k * (c["ids"] // 8 + 8) + 8 * (c["e"] + 1) + z * d * (t + t * k), "flops": t * k}
    if kind == "combine":
        return {"bytes": 8 * t * k + z * d * (t * k + t + (t if c["base"] else 0)), "flops": 2 * t * k * d}
    return {"bytes": 12 * t * k + z * d * (t + 2 * t * k), "flops": 3 * t * k * d}


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    """The definitions in 64 bits. Tokens and weights are coded by the rule's
    own fp32 steps; a norm in front of the coding is taken in 64 bits and its
    result coded by the same rule."""
    s = _inputs(case, seed)
    c, kind = case, case["kind"]
    D = torch.float64
    if kind in ("linear", "norm_linear"):
        def code(rows):
            top = rows.abs().max(dim=1).values
            factor = torch.where(top == 0, torch.zeros_like(top), torch.full_like(top, 127.0) / top)
            return (rows * factor.unsqueeze(1)).round().to(D), top.to(D) / 127.0

        x = s["X"].float()
        if kind == "norm_linear":
            x64 = x.to(D)
            x = (x64 / (x64.pow(2).sum(dim=1, keepdim=True) / c["k"] + EPS).sqrt() * s["w"].to(D)).float()
        a, sa = code(x)
        parts = []
        step = max(1, (1 << 27) // c["k"])
        for lo in range(0, c["n"], step):
            b, sb = code(s["W"][lo:lo + step])
            parts.append(torch.einsum("mk,nk->mn", a, b) * sa.unsqueeze(1) * sb.unsqueeze(0))
        return torch.cat(parts, dim=1)
    if kind.startswith("norm"):
        d = c["d"]
        w = s["w"].to(D)

        def rms(v):
            return (v.pow(2).sum(dim=1, keepdim=True) / d + EPS).sqrt()

        if kind == "norm_before_bwd":
            x, dh, w = s["X"].to(D), s["dH"].to(D), w + OFFSET
            r = rms(x)
            dot = (dh * w * x).sum(dim=1, keepdim=True)
            return {"dx": s["dR"].to(D) + dh * w / r - x * dot / (d * r.pow(3)), "dw": (dh * x / r).sum(dim=0)}
        b, gate = s["B"].to(D), c["gate"]
        g = torch.ones((), dtype=D, device=b.device) if gate == "none" else s["gate"].to(D)
        g = g.unsqueeze(1) if gate == "token" else g
        if kind == "norm_join":
            y = (s["R"].to(D) + SCALE * g * b / rms(b) * w)
            # the next norm reads the residual stream as it is stored
            stored = y.to(torch.float32).to(TYPES[c["type"]]).to(D)
            return {"y": y, "h": stored / rms(stored) * s["w_next"].to(D)}
        dy, r = s["dY"].to(D) * SCALE, rms(b)
        dn = dy * g * w
        out = {"db": dn / r - b * (dn * b).sum(dim=1, keepdim=True) / (d * r.pow(3)), "dw": (dy * g * b / r).sum(dim=0)}
        if gate != "none":
            dg = dy * w * b / r
            out["dgate"] = dg.sum(dim=0) if gate == "channel" else dg.sum(dim=1) if gate == "token" else dg
        return out
    if kind == "dispatch":
        return None          # whole numbers and copies
    row_of, w = s["row_of"].to(torch.int64), s["weights"].to(D)
    t, k, d = c["t"], c["k"], c["d"]
    if kind == "combine":
        y = torch.zeros((t, d), dtype=D, device=w.device) if s["base"] is None else s["base"].to(D)
        for j in range(k):
            has = (row_of[:, j] >= 0).nonzero().squeeze(1)
            y[has] += w[has, j].unsqueeze(1) * s["Ys"][row_of[has, j]].to(D)
        return y
    dys = torch.zeros((t * k, d), dtype=D, device=w.device)
    dw = torch.zeros((t, k), dtype=D, device=w.device)
    for j in range(k):
        has = (row_of[:, j] >= 0).nonzero().squeeze(1)
        at = row_of[has, j]
        dy = s["dY"][has].to(D)
        dys[at] = w[has, j].unsqueeze(1) * dy
        dw[has, j] = (dy * s["Ys"][at].to(D)).sum(dim=1)
    return {"dys": dys, "dweights": dw}
