"""The cache, the attention, the probabilities and the verification as a server
uses them: one behind the other, in captured graphs whose batches change between
replays, on other streams, from two threads, and with waits that run out."""

import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from block_testlib import ROUND, TINY, TYPES, blank, close, f64, rows, type_of
from cache_testlib import Cache, attend64, held, ints, starts_of
from q4_quantized_linear_gb300 import synth
from test_gpu_draft import verify64

pytestmark = pytest.mark.gpu


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def pack(q4, n, k, seed):
    blocks = synth.q4_0_blocks(n, k, seed=seed)
    return q4.pack(torch.from_numpy(blocks.reshape(-1)).cuda(), n, k)


@pytest.mark.parametrize("cache", ["f16", "i8"])
def test_a_drafting_server(q4lib, cache):
    """Slots with drafted tokens: projections over Q4_0 weights, keys and values
    cached, attention, the logit head, probabilities, verification; then the
    sequences are rewound to what was kept and go on. Each stage against 64 bits of
    its own inputs; and at the end the cache holds what a fresh one would."""
    q4 = q4lib
    g = torch.Generator(device="cuda").manual_seed(1)
    heads, kv_heads, d, width, vocab, page, slots, draft = 4, 2, 64, 256, 500, 16, 3, 4
    qkv, head = pack(q4, (heads + 2 * kv_heads) * d, width, 1), pack(q4, vocab, heads * d, 2)
    kept_k, kept_v = [[] for _ in range(slots)], [[] for _ in range(slots)]
    lens = [0] * slots
    c = Cache(q4, [200] * slots, kv_heads, d, page, cache)
    w = 1 + 0.1 * normal(g, width)
    counts = [37, 5, 20]                                  # prompts first
    for step in range(6):
        n = sum(counts)
        x, h = normal(g, n, width), blank(n, width, "f32")
        q4.q4_norm_before(h, width, q4.Q4_TYPE_F32, None, x, width, q4.Q4_TYPE_F32, w, 0.0, 1e-6, n, width)
        y = q4.matmul(qkv, h.contiguous(), (heads + 2 * kv_heads) * d)
        q, k, v = y[:, :heads * d], y[:, heads * d:(heads + kv_heads) * d], y[:, (heads + kv_heads) * d:]
        lens = [a + b for a, b in zip(lens, counts)]
        c.write(k, v, "f32", lens, counts)
        o = blank(n, heads * d, "f32")
        c.attend(o, q, "f32", heads, d ** -0.5, 0, lens, counts)
        at = starts_of(counts)
        for s in range(slots):
            kept_k[s] += list(k[at[s]:at[s + 1]].clone())
            kept_v[s] += list(v[at[s]:at[s + 1]].clone())
        all_k = torch.cat([torch.stack(t) for t in kept_k]).reshape(-1, kv_heads, d)
        all_v = torch.cat([torch.stack(t) for t in kept_v]).reshape(-1, kv_heads, d)
        ref, tol = attend64(q, held(all_k, cache), held(all_v, cache), heads, kv_heads, d, d ** -0.5, 0, lens, counts, 2.0 ** -21, 2)
        close(o, f64(ref), f64(tol) + ROUND["f32"] * np.abs(f64(ref)) * 1.01 + TINY["f32"], "attention")
        # the last draft + 1 rows of each slot: the drafted tokens' places and the one after
        last = torch.cat([torch.arange(at[s + 1] - min(counts[s], draft + 1), at[s + 1]) for s in range(slots)])
        each = [min(counts[s], draft + 1) for s in range(slots)]
        logits = q4.matmul(head, o[last.cuda()].contiguous(), vocab)
        p = blank(sum(each), vocab, "f32")
        q4.q4_token_probs(p, vocab, logits, vocab, q4.Q4_TYPE_F32, None, sum(each), vocab)
        close(p, f64(torch.softmax(logits.double(), dim=1)), 1e-5 * np.abs(f64(torch.softmax(logits.double(), dim=1))) + 1e-30, "probabilities")
        padded = torch.zeros(slots, draft + 1, vocab, device="cuda")
        first = starts_of(each)
        for s in range(slots):
            padded[s, :each[s]] = p[first[s]:first[s + 1]]
        padded = padded.reshape(-1, vocab)
        drafted = torch.stack([padded[s * (draft + 1) + i].argmax() if (s + i + step) % 3 else torch.tensor(7, device="cuda")
                               for s in range(slots) for i in range(draft)]).reshape(slots, draft).to(torch.int32)
        n_draft = ints([m - 1 for m in each])
        accept, sample = torch.rand(slots, draft, generator=g, device="cuda"), torch.rand(slots, generator=g, device="cuda")
        tokens, kept = torch.empty((slots, draft + 1), dtype=torch.int32, device="cuda"), torch.empty(slots, dtype=torch.int32, device="cuda")
        q4.q4_draft_verify(tokens, draft + 1, kept, padded, vocab, None, 0, drafted, draft, n_draft, accept, draft, sample, slots, draft, vocab)
        want = verify64(padded, None, drafted, n_draft.tolist(), accept, sample, vocab)
        assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(kept.cpu().numpy(), want[1])
        assert q4.q4_last_device_status(clear=True) == 0
        # what was not kept is taken back; the next pass writes over it
        for s in range(slots):
            back = each[s] - 1 - int(kept[s])
            lens[s] -= back
            if back:
                del kept_k[s][-back:], kept_v[s][-back:]
        counts = [5, 5, 3]
    bk, bv = blank(sum(lens), kv_heads * d, "f32"), blank(sum(lens), kv_heads * d, "f32")
    c.read(bk, bv, "f32", None, lens)
    for got, want in ((bk, kept_k), (bv, kept_v)):
        ref = held(torch.cat([torch.stack(t) for t in want]).reshape(-1, kv_heads, d), cache).float().reshape(sum(lens), -1)
        assert torch.equal(got, ref)


def batch(g, lens, counts, name, heads, kv_heads, d):
    n = sum(counts)
    return (normal(g, n, heads * d).to(TYPES[name]), normal(g, n, kv_heads * d).to(TYPES[name]), normal(g, n, kv_heads * d).to(TYPES[name]))


class Step:
    """Static buffers of a write and an attention, as a captured program has them."""

    def __init__(self, q4, cache, name, heads, rows_, n_seq, max_new):
        self.q4, self.c, self.heads, self.rows, self.n_seq, self.max_new = q4, cache, heads, rows_, n_seq, max_new
        self.type = type_of(q4, name)
        self.q, self.o = blank(rows_, heads * cache.d, name), blank(rows_, heads * cache.d, name)
        self.k, self.v = blank(rows_, cache.heads * cache.d, name), blank(rows_, cache.heads * cache.d, name)
        self.lens, self.starts = ints([0] * n_seq), ints([0] * (n_seq + 1))
        need = q4.q4_attention_workspace_size(rows_, n_seq, heads, cache.heads, cache.d)
        self.ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")

    def set(self, lens, counts, q, k, v):
        n = sum(counts)
        self.lens.copy_(ints(lens))
        self.starts.copy_(ints(starts_of(counts)))
        self.q[:n], self.k[:n], self.v[:n] = q, k, v

    def run(self):
        c = self.c
        self.q4.q4_kv_write(*c.args(), self.lens, self.starts, self.n_seq, self.k, self.k.stride(0), self.v, self.v.stride(0), self.type, self.rows)
        self.q4.q4_attention(self.o, self.o.stride(0), self.q, self.q.stride(0), self.type, self.heads, c.d ** -0.5, 0, *c.args(), self.lens,
                             self.starts, self.n_seq, self.rows, self.max_new, self.ws, self.ws.numel())


@pytest.mark.parametrize("name,cache", [("bf16", "i8"), ("bf16", "bf16"), ("f32", "f16")])
@pytest.mark.parametrize("new", [4, 150])
def test_captured_steps_with_other_batches(q4lib, name, cache, new):
    """A captured pass replays with other lengths, tables and rows: the results are
    the eager call's, to the bit."""
    heads, kv_heads, d, n_seq = 4, 2, 128, 3
    g = torch.Generator(device="cuda").manual_seed(3)
    caches = [Cache(q4lib, [1500] * n_seq, kv_heads, d, 64, cache, seed=5) for _ in range(2)]
    captured, eager = (Step(q4lib, c, name, heads, 3 * new, n_seq, new) for c in caches)
    captured.set([1, 1, 1], [1, 1, 1], *batch(g, None, [1, 1, 1], name, heads, kv_heads, d))
    captured.run()                                        # kernels are loaded before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.run()
    lens = [0] * n_seq
    for counts in ([new, 1, new], [1, 1, 1], [new, 0, new // 2], [2, new, 0]):
        lens = [a + b for a, b in zip(lens, counts)]
        data = batch(g, lens, counts, name, heads, kv_heads, d)
        captured.set(lens, counts, *data)
        eager.set(lens, counts, *data)
        graph.replay()
        eager.run()
        torch.cuda.synchronize()
        n = sum(counts)
        assert torch.equal(captured.o[:n], eager.o[:n]) and bool(torch.isfinite(captured.o[:n].float()).all())
    assert torch.equal(caches[0].pages, caches[1].pages)
    assert q4lib.q4_last_device_status(clear=True) == 0


def test_two_graphs_on_two_streams(q4lib):
    """Graphs with a workspace each, replayed at the same time."""
    heads, kv_heads, d = 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(4)
    steps, graphs, alone = [], [], []
    for i in range(2):
        c = Cache(q4lib, [3000, 900], kv_heads, d, 32, "bf16", seed=i)
        k = normal(g, 3900, kv_heads * d).bfloat16()
        c.write(k, k, "bf16", [3000, 900], [3000, 900])
        s = Step(q4lib, c, "bf16", heads, 40, 2, 20)
        s.set([3000, 900], [20, 20], *batch(g, None, [20, 20], "bf16", heads, kv_heads, d))
        s.run()
        torch.cuda.synchronize()
        alone.append(s.o.clone())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(5):
                s.run()
        steps.append(s)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for s, want in zip(steps, alone):
        assert torch.equal(s.o, want)
    assert q4lib.q4_last_device_status(clear=True) == 0


def test_two_threads(q4lib):
    """Calls from two threads, on streams of their own."""
    heads, kv_heads, d = 4, 1, 64
    results, errors = [None, None], []

    def work(i):
        try:
            g = torch.Generator(device="cuda").manual_seed(10 + i)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                c = Cache(q4lib, [700], kv_heads, d, 16, "f16", seed=i)
                k = normal(g, 700, kv_heads * d).half()
                q = normal(g, 30, heads * d).half()
                c.write(k, k, "f16", [700], [700])
                o = [blank(30, heads * d, "f16") for _ in range(20)]
                for x in o:
                    c.attend(x, q, "f16", heads, 0.125, 0, [700], [30])
                stream.synchronize()
            results[i] = (q, k, o)
        except Exception as e:                            # noqa: BLE001 (shown below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for q, k, o in results:
        kk = held(k.reshape(700, kv_heads, d), "f16")
        ref, tol = attend64(q, kk, kk, heads, kv_heads, d, 0.125, 0, [700], [30], 2.0 ** -11, 1)
        for x in o:
            assert torch.equal(x, o[0])
        close(o[0], f64(ref), f64(tol) + ROUND["f16"] * np.abs(f64(ref)) * 1.01 + TINY["f16"])


def test_tokens_captured(q4lib):
    """Probabilities and verification in a graph."""
    n, s, t = 20000, 5, 3
    g = torch.Generator(device="cuda").manual_seed(6)
    logits, p = torch.empty(s * (t + 1), n, device="cuda"), torch.empty(s * (t + 1), n, device="cuda")
    q = torch.softmax(normal(g, s * t, n), dim=1)
    drafted = torch.randint(0, n, (s, t), generator=g, device="cuda").to(torch.int32)
    accept, sample = torch.rand(s, t, generator=g, device="cuda"), torch.rand(s, generator=g, device="cuda")
    tokens, kept = torch.empty((s, t + 1), dtype=torch.int32, device="cuda"), torch.empty(s, dtype=torch.int32, device="cuda")

    def run():
        q4lib.q4_token_probs(p, n, logits, n, q4lib.Q4_TYPE_F32, None, s * (t + 1), n)
        q4lib.q4_draft_verify(tokens, t + 1, kept, p, n, q, n, drafted, t, None, accept, t, sample, s, t, n)

    logits.zero_()
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        logits.copy_(normal(g, s * (t + 1), n) * 2)
        accept.copy_(torch.rand(s, t, generator=g, device="cuda") * 0.3)
        graph.replay()
        torch.cuda.synchronize()
        want = verify64(p, q, drafted, None, accept, sample, n)
        assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(kept.cpu().numpy(), want[1])


@pytest.mark.parametrize("name,cache", [("f16", "f16"), ("f32", "f16"), ("bf16", "bf16"), ("bf16", "i8"), ("f32", "i8")])
@pytest.mark.parametrize("new", [2, 200])
def test_waits_that_run_out(q4lib, name, cache, new):
    """With a limit of a nanosecond waits may run out: the call returns, says so in
    the status word, and the next call is as ever."""
    heads, kv_heads, d, length = 4, 2, 128, 2000
    g = torch.Generator(device="cuda").manual_seed(7)
    c = Cache(q4lib, [length], kv_heads, d, 64, cache)
    k = normal(g, length, kv_heads * d).to(TYPES[name])
    c.write(k, k, name, [length], [length])
    q = normal(g, new, heads * d).to(TYPES[name])
    good, o = blank(new, heads * d, name), blank(new, heads * d, name)
    c.attend(good, q, name, heads, 0.1, 0, [length], [new])
    torch.cuda.synchronize()
    assert q4lib.q4_last_device_status(clear=True) == 0
    try:
        for _ in range(5):
            q4lib.q4_set_wait_limit_ns(1)
            c.attend(o, q, name, heads, 0.1, 0, [length], [new])
            torch.cuda.synchronize()
            assert q4lib.q4_last_device_status(clear=True) in (0, q4lib.Q4_ERR_DEVICE_TIMEOUT)
            q4lib.q4_set_wait_limit_ns(2_000_000_000)
            c.attend(o, q, name, heads, 0.1, 0, [length], [new])
            torch.cuda.synchronize()
            assert q4lib.q4_last_device_status(clear=True) == 0 and torch.equal(o, good)
    finally:
        q4lib.q4_set_wait_limit_ns(2_000_000_000)


_FIRST = """
import torch
from q4_quantized_linear_gb300 import binding as q4
heads, kv_heads, d, page, n, rows = 8, 2, 128, 32, 5000, 300
g = torch.Generator(device="cuda").manual_seed(5)
ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
K, V, Q = (torch.randn(rows, h * d, generator=g, device="cuda").to(torch.bfloat16) for h in (kv_heads, kv_heads, heads))
pages = torch.zeros((10, q4.q4_kv_page_size(page, kv_heads, d, q4.Q4_TYPE_I8)), dtype=torch.uint8, device="cuda")
cache = (pages, 10, page, kv_heads, d, q4.Q4_TYPE_I8, torch.arange(10, dtype=torch.int32, device="cuda"), 10)
batch = (ints(rows), ints(0, rows), 1)
need = q4.q4_attention_workspace_size(rows, 1, heads, kv_heads, d)
ws = torch.empty(need, dtype=torch.uint8, device="cuda")
O, k, v = torch.zeros_like(Q), torch.zeros_like(K), torch.zeros_like(V)
logits = torch.randn(4, n, generator=g, device="cuda")
P, tokens, kept = torch.zeros(4, n, device="cuda"), torch.zeros((1, 4), dtype=torch.int32, device="cuda"), ints(0)
accept, sample, drafted = torch.full((1, 3), 0.5, device="cuda"), torch.full((1,), 0.5, device="cuda"), ints(1, 2, 3).reshape(1, 3)


def step():
    q4.q4_kv_write(*cache, *batch, K, kv_heads * d, V, kv_heads * d, q4.Q4_TYPE_BF16, rows)
    q4.q4_attention(O, heads * d, Q, heads * d, q4.Q4_TYPE_BF16, heads, d ** -0.5, 0, *cache, *batch, rows, 0, ws, need)
    q4.q4_kv_read(k, kv_heads * d, v, kv_heads * d, q4.Q4_TYPE_BF16, *cache, None, ints_0, 1, rows)
    q4.q4_token_probs(P, n, logits, n, q4.Q4_TYPE_F32, None, 4, n)
    q4.q4_draft_verify(tokens, 4, kept, P, n, None, 0, drafted, 3, None, accept, 3, sample, 1, 3, n)


ints_0 = batch[1]
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    step()
out = (O, k, v, P, tokens, kept)
graph.replay()
torch.cuda.synchronize()
first = [x.clone() for x in out]
for x in out:
    x.zero_()
step()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(first, out)) and bool(first[0].any()) and bool(first[3].any())
assert q4.q4_last_device_status(clear=True) == 0
print("same")
"""


def test_first_call_is_captured(q4lib):
    """A process whose first calls are captured gives what the plain calls give."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", _FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "same" in done.stdout, done.stderr[-2000:]
