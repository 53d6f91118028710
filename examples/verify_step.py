"""A small decoder that generates with drafted tokens, every step of it on the
library's kernels: 4-bit products, the cache append, attention over the paged
cache and the acceptance of the drafts.

    python examples/verify_step.py [--steps 40] [--drafts 3] [--cache bf16|e4m3] [--window 64]

One layer with random weights stands in for a model: its output layer follows
its embedding through a permutation of the vocabulary with short cycles, so that
the text repeats itself after a while and the drafter (what followed the last
occurrence of the last token) begins to be right.  The order of a step is that of a serving loop:

  1. rows of all sequences: the last token and the drafts after it
  2. q, k, v = one product; the new keys and values go to their pages
  3. attention of the rows over the cache, each up to its own token
  4. output projection with the residual sum, logits, probabilities
  5. acceptance: the tokens that stay, and one more

A refused draft leaves a key and a value behind; the next step's rows overwrite
them, since len counts only what was accepted.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from few_row_quantized_amd import qgemv  # noqa: E402

BITS, GROUP = 4, 64


def quantized(w):
    """codes, scales and biases of the 4-bit affine format for w [N, K]."""
    N, K = w.shape
    g = w.float().view(N, K // GROUP, GROUP)
    low, high = g.amin(-1), g.amax(-1)
    scales = ((high - low) / 15).clamp(min=1e-6).half()
    biases = low.half()
    q = ((g - biases.float()[..., None]) / scales.float()[..., None]).round().clamp(0, 15).to(torch.uint8).view(N, K)
    return q[:, ::2] | q[:, 1::2] << 4, scales, biases


class Decoder:
    def __init__(self, vocabulary=2048, width=512, kv_heads=2, group=4, dim=64, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)
        self.V, self.H, self.G, self.D, self.device = vocabulary, kv_heads, group, dim, device
        self.embedding = torch.randn(vocabulary, width, generator=g).bfloat16().to(device)
        heads = kv_heads * (group + 2)
        cycles = torch.randperm(vocabulary, generator=g).view(-1, 16)
        follow = torch.empty(vocabulary, dtype=torch.long)  # the token after each
        follow[cycles] = cycles.roll(-1, 1)
        head = torch.randn(vocabulary, width, generator=g) * 0.1
        head[follow] += self.embedding.cpu().float() / width ** 0.5
        to = lambda ws: tuple(x.to(device).contiguous() for x in ws)  # noqa: E731
        self.qkv = to(quantized(torch.randn(heads * dim, width, generator=g) / width ** 0.5))
        self.o = to(quantized(torch.randn(width, kv_heads * group * dim, generator=g) * 0.1 / width ** 0.5))
        self.head = to(quantized(head))

    def product(self, weights, x, residual=None):
        return qgemv.small(*weights, x, BITS, GROUP, residual=residual)


class Generation:
    """Sequences in progress: their tokens, their pages and what a step reuses."""

    def __init__(self, model, prompts, drafts=3, cache=torch.bfloat16, window=0, sinks=0, page=16, longest=1024,
                 temperature=0.05, seed=1):
        if len(prompts) * (drafts + 1) > 16:
            raise ValueError("the rows of a step, drafts + 1 a sequence, are at most 16 in all")
        self.slots = -(-longest // page) * page  # of a sequence's pages
        for b, p in enumerate(prompts):
            self._fits(b, len(p))
        self.m, self.window, self.sinks, self.temperature = model, window, sinks, temperature
        self.tokens = [list(p) for p in prompts]
        self.cached = [0] * len(prompts)  # tokens whose keys and values are in the cache
        self.drafts, self.M = drafts, drafts + 1
        dev, B, width = model.device, len(prompts), -(-longest // page)
        shape = (B * width, page, model.H, model.D)
        pages = torch.randperm(B * width, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        scale = None
        if cache == torch.float8_e4m3fn:
            scale = torch.full((model.H,), 1 / 64, device=dev)
        self.cache = qgemv.KvCache(torch.zeros(shape, dtype=cache, device=dev), torch.zeros(shape, dtype=cache, device=dev),
                                   pages.view(B, width).to(dev), scale, scale)
        self.attend_work = qgemv.attend_workspace(self.cache, 16, model.H * model.G, 16)
        self.verify_work = torch.zeros(0, dtype=torch.uint8, device=dev)
        self.random = torch.Generator(device=dev).manual_seed(seed)
        while any(len(t) - 1 > c for t, c in zip(self.tokens, self.cached)):
            self._prefill()

    def _fits(self, b, tokens):
        if tokens > self.slots:
            raise ValueError(f"sequence {b} has pages for {self.slots} tokens, not for {tokens}")

    def _layer(self, rows, lens):
        """Logits of the rows of all sequences; their keys and values enter the
        cache on the way."""
        m, dev = self.m, self.m.device
        start = torch.tensor([0] + [len(r) for r in rows], dtype=torch.int32).cumsum(0, dtype=torch.int32).to(dev)
        length = torch.tensor(lens, dtype=torch.int32, device=dev)
        fed = torch.tensor([t for r in rows for t in r], dtype=torch.int32, device=dev)
        T, Hq = fed.numel(), m.H * m.G
        x = m.embedding[fed]
        qkv = m.product(m.qkv, x).view(T, Hq + 2 * m.H, m.D)
        qgemv.append(self.cache, qkv[:, Hq:Hq + m.H], qkv[:, Hq + m.H:], start, length)
        out = qgemv.attend(self.cache, qkv[:, :Hq].bfloat16(), start, length, max(map(len, rows)), window=self.window,
                           sinks=self.sinks, workspace=self.attend_work)
        y = m.product(m.o, out.view(T, -1), residual=x.float())
        return m.product(m.head, y.bfloat16()), fed, start

    def _prefill(self):
        """Up to 16 prompt tokens in all into the cache, but for each sequence's last."""
        room, rows = 16, []
        for t, c in zip(self.tokens, self.cached):
            rows.append(t[c:max(c, min(len(t) - 1, c + room))])
            room -= len(rows[-1])
        self.cached = [c + len(r) for c, r in zip(self.cached, rows)]
        self._layer(rows, self.cached)

    def _draft(self, tokens):
        """What followed the last earlier occurrence of the last token."""
        for i in range(len(tokens) - 2, -1, -1):
            if tokens[i] == tokens[-1]:
                return tokens[i + 1:i + 1 + self.drafts]
        return []

    def step(self):
        """One verify step of all sequences; returns how many tokens each gained.
        Drafts end where a sequence's pages do; a sequence whose last token has no
        place left ends the generation with a ValueError, before anything is changed."""
        for b, c in enumerate(self.cached):
            self._fits(b, c + 1)
        rows = [t[-1:] + self._draft(t)[:self.slots - c - 1] for t, c in zip(self.tokens, self.cached)]
        lens = [c + len(r) for c, r in zip(self.cached, rows)]
        logits, fed, start = self._layer(rows, lens)
        p = torch.softmax(logits / self.temperature, -1)
        u = torch.rand(fed.numel(), device=p.device, generator=self.random)
        if not self.verify_work.numel():
            self.verify_work = qgemv.verify_workspace(p, len(rows))
        out, count = qgemv.verify(p, None, fed, u, start, self.M, workspace=self.verify_work)
        out, count = out.tolist(), count.tolist()
        at = 0
        for b, (r, n) in enumerate(zip(rows, count)):
            self.tokens[b] += out[at:at + n]
            self.cached[b] += n
            at += len(r)
        return count


def main():
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    a.add_argument("--steps", type=int, default=40)
    a.add_argument("--drafts", type=int, default=3)
    a.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    a.add_argument("--window", type=int, default=0)
    a = a.parse_args()
    cache = torch.bfloat16 if a.cache == "bf16" else torch.float8_e4m3fn
    prompts = [[1, 2, 3], [70, 80], list(range(100, 140))]
    longest = max(map(len, prompts)) + a.steps * (a.drafts + 1)
    g = Generation(Decoder(), prompts, a.drafts, cache, a.window, min(a.window, 4), longest=longest)
    gained = [g.step() for _ in range(a.steps)]
    for b, t in enumerate(g.tokens):
        n = sum(s[b] for s in gained)
        print(f"sequence {b}: {n} tokens in {a.steps} steps ({n / a.steps:.2f} a step), {len(t)} in all: ... {t[-8:]}")


if __name__ == "__main__":
    main()
