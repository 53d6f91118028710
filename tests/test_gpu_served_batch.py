"""The rotated append, the attention over a shared prefix, the routing and the
adapters together, as the example runs them."""
import importlib.util
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
FOLDER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


@pytest.fixture(scope="module")
def example(require_gpu):
    sys.path.insert(0, FOLDER)
    spec = importlib.util.spec_from_file_location("served_batch", os.path.join(FOLDER, "served_batch.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


SYSTEM = list(range(200, 300))
PROMPTS = [[1, 2, 3], [70, 80], list(range(100, 110))]


def plain_logits(m, tokens, adapter, system):
    """Logits after each token of one request, in 64 bits on the CPU, from the
    definitions: no cache, no pages, the weights dequantized."""
    def dense(w):
        codes, scales, biases = (t.cpu() for t in w)
        q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
        g = q.view(*q.shape[:-1], -1, 64) * scales.double()[..., None] + biases.double()[..., None]
        return g.flatten(-2)

    T, D, Hq = len(tokens), m.D, m.H * m.G
    x = m.embedding.cpu()[torch.tensor(tokens)].double()
    qkv = x @ dense(m.qkv).T
    if adapter >= 0:
        more = (x @ m.a.cpu()[adapter].double().T) @ m.b.cpu()[adapter].double().T
        qkv[system:] += more[system:]
    qkv = qkv.view(T, -1, D)
    pairs = m.freq.numel()
    angle = torch.arange(T)[:, None].double() * m.freq.cpu().double()
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    turned = qkv.clone()
    a, b = qkv[..., :pairs], qkv[..., pairs:2 * pairs]
    turned[..., :pairs], turned[..., pairs:2 * pairs] = a * c - b * s, a * s + b * c
    q, k, v = turned[:, :Hq], turned[:, Hq:Hq + m.H], qkv[:, Hq + m.H:]
    k, v = (t.repeat_interleave(m.G, 1) for t in (k, v))
    score = torch.einsum("thd,jhd->htj", q, k) * D ** -0.5
    score = score.masked_fill(torch.ones(T, T, dtype=torch.bool).triu(1), float("-inf"))
    out = torch.einsum("htj,jhd->thd", torch.softmax(score, -1), v).reshape(T, -1)
    y = out @ dense(m.o).T + x
    gate = torch.sigmoid(y @ dense(m.router).T)
    weight, chosen = gate.topk(m.chosen, -1)
    weight = weight / weight.sum(-1, keepdim=True)
    up, down = dense(m.up), dense(m.down)
    for t in range(T):
        for e, w in zip(chosen[t].tolist(), weight[t]):
            y[t] += w * (down[e] @ torch.relu(up[e] @ y[t]))
    return y @ dense(m.head).T


@pytest.mark.parametrize("cache", [torch.bfloat16, torch.float8_e4m3fn])
def test_sharing_and_drafts_change_the_speed_and_not_the_text(example, cache):
    """At a low temperature the text is the model's own, whether the prompt's pages
    are shared or each request has its own, with drafts or without."""
    m = example.ServedDecoder()
    shared = example.ServedBatch(m, SYSTEM, PROMPTS, [0, 1, -1], drafts=3, cache=cache)
    apart = example.ServedBatch(m, SYSTEM, PROMPTS, [0, 1, -1], share=False, drafts=0, cache=cache)
    assert torch.equal(shared.cache.table[1, :6], shared.cache.table[0, :6])  # 96 of the 100 tokens
    gained = [shared.step() for _ in range(20)]
    while any(len(a) < len(b) for a, b in zip(apart.tokens, shared.tokens)):
        apart.step()
    for a, b in zip(apart.tokens, shared.tokens):
        assert a[:len(b)] == b
    assert all(1 <= n <= 4 for s in gained for n in s)


def test_a_step_against_the_plain_model(example):
    """Logits of a prompt's last tokens against 64 bits.  Between the two lie
    bf16 roundings of the embedding's products' inputs (queries, keys, values,
    weights of the softmax, the attention's output, the experts' inputs: half a step,
    2^-8, of a value each), which the peaks of the output layer stand far above: the
    logits agree within 1/16 of their own spread, and their greatest is the same."""
    m = example.ServedDecoder()
    for adapter in (-1, 2):
        g = example.ServedBatch(m, SYSTEM, [[5, 6, 7, 8]], [adapter], drafts=3)
        rows, lens = [[8, 9, 10]], [g.cached[0] + 3]
        logits, _, _ = g._layer(rows, lens)
        want = plain_logits(m, SYSTEM + [5, 6, 7] + rows[0], adapter, len(SYSTEM))[-3:]
        got = logits.double().cpu()
        assert ((got - want).norm(dim=-1) <= want.norm(dim=-1) / 16).all()
        assert torch.equal(got.argmax(-1), want.argmax(-1))


def test_adapters_change_their_own_rows_alone(example):
    m = example.ServedDecoder()
    one = example.ServedBatch(m, SYSTEM, PROMPTS, [0, -1, -1], drafts=3)
    two = example.ServedBatch(m, SYSTEM, PROMPTS, [1, -1, -1], drafts=3)
    rows = [t[-1:] for t in one.tokens]
    lens = [c + 1 for c in one.cached]
    a, b = one._layer(rows, lens)[0], two._layer(rows, lens)[0]
    assert not torch.equal(a[0], b[0]) and torch.equal(a[1:], b[1:])
