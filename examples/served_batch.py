"""A batch of requests on one system prompt, each with an adapter of its own, on a
small decoder with rotated positions and experts: every step on the library's
kernels, those of verify_step.py and

  1. q, k, v = one product + the request's adapter
  2. queries and keys turned by their positions, keys and values to their pages
  3. attention of all rows over the common prompt at once, and over their own tokens
  4. routing of the rows to experts, whose two products read each expert once

    python examples/served_batch.py [--steps 20] [--drafts 3] [--cache bf16|e4m3]

The pages of the system prompt are in every request's page table and are filled
once.  The layer's weights are random; its output layer follows the embedding
through a permutation of the vocabulary (verify_step.py).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import verify_step  # noqa: E402
from few_row_quantized_amd import qgemv  # noqa: E402
from verify_step import BITS, GROUP, quantized  # noqa: E402


class ServedDecoder(verify_step.Decoder):
    """verify_step's decoder with rotated positions, adapters on the q, k, v
    product, and experts after the attention."""

    def __init__(self, adapters=3, rank=8, experts=8, chosen=2, inner=256, rotated=32, **kw):
        super().__init__(**kw)
        g = torch.Generator().manual_seed(kw.get("seed", 0) + 100)
        dev, width, N = self.device, self.embedding.shape[1], self.qkv[0].shape[0]
        self.freq = (10000.0 ** (-torch.arange(rotated // 2, dtype=torch.float64) / (rotated // 2))).float().to(dev)
        self.a = (torch.randn(adapters, rank, width, generator=g) / width ** 0.5).bfloat16().to(dev)
        self.b = (0.3 * torch.randn(adapters, N, rank, generator=g) / rank ** 0.5).bfloat16().to(dev)
        self.E, self.chosen = experts, chosen
        self.router = tuple(x.to(dev).contiguous() for x in quantized(torch.randn(experts, width, generator=g) / width ** 0.5))
        self.up = self._experts(torch.randn(experts, inner, width, generator=g) / width ** 0.5)
        self.down = self._experts(0.1 * torch.randn(experts, width, inner, generator=g) / inner ** 0.5)

    def _experts(self, w):
        parts = zip(*(quantized(x) for x in w))
        return tuple(torch.stack(p).to(self.device).contiguous() for p in parts)

    def gather(self, weights, x, x_idx, e_idx):
        """The product of row x_idx[p] with expert e_idx[p], 0 where it is not there."""
        codes, scales, biases = weights
        E, N, K = codes.shape[0], codes.shape[1], codes.shape[2] * 8 // BITS
        y = torch.zeros((x_idx.numel(), N), device=x.device)
        qgemv.qgemv_gather(codes, scales, biases, x, x_idx, e_idx, y, x_idx.numel(), x.shape[0], E, N, K, BITS, GROUP)
        return y

    def experts_of(self, x):
        """The rows x (bfloat16) through their experts."""
        T, k = x.shape[0], self.chosen
        experts, weights = qgemv.route(self.product(self.router, x), k, score="sigmoid")
        pairs = torch.arange(T * k, dtype=torch.int32, device=x.device)
        h = self.gather(self.up, x, pairs // k, experts.view(-1))
        y = self.gather(self.down, torch.relu(h).bfloat16(), pairs, experts.view(-1))
        return (y.view(T, k, -1) * weights[..., None]).sum(1)


class ServedBatch(verify_step.Generation):
    """Requests on one system prompt, adapters[b] the adapter of request b (-1:
    none)."""

    def __init__(self, model, system, prompts, adapters, share=True, **kw):
        self.adapters, self.system = adapters, len(system)
        self.share = share
        page = kw.get("page", 16)
        # (a request's last token is its own: it is fed with the first step)
        whole = min(len(system), len(system) + min(map(len, prompts)) - 1) // page if share and len(system) else 0
        self.common = torch.tensor([whole * page], dtype=torch.int32, device=model.device)
        self.pages = whole
        super().__init__(model, [list(system) + list(p) for p in prompts], **kw)

    def _prefill(self):
        """The first request's rows alone until the common pages are full, which the
        others then have too; after that verify_step's way."""
        common = self.pages * (self.slots // self.cache.table.shape[1])
        if self.cached[0] >= common:
            return super()._prefill()
        if self.cached[0] == 0:
            self.cache.table[:, :self.pages] = self.cache.table[0, :self.pages].clone()
        rows = [self.tokens[0][self.cached[0]:min(self.cached[0] + 16, common)]] + [[]] * (len(self.tokens) - 1)
        self.cached[0] += len(rows[0])
        self._layer(rows, self.cached)
        if self.cached[0] == common:
            self.cached = [common] * len(self.tokens)

    def _layer(self, rows, lens):
        m, dev = self.m, self.m.device
        start = torch.tensor([0] + [len(r) for r in rows], dtype=torch.int32).cumsum(0, dtype=torch.int32).to(dev)
        length = torch.tensor(lens, dtype=torch.int32, device=dev)
        fed = torch.tensor([t for r in rows for t in r], dtype=torch.int32, device=dev)
        # (the system prompt is read without an adapter: its keys are everyone's)
        which = torch.tensor([a if n - len(r) + i >= self.system else -1
                              for a, r, n in zip(self.adapters, rows, lens) for i in range(len(r))],
                             dtype=torch.int32, device=dev)
        T, Hq = fed.numel(), m.H * m.G
        x = m.embedding[fed]
        qkv = m.product(m.qkv, x)
        qkv = qgemv.adapt(qkv, x, m.a, m.b, which, out=qkv).view(T, Hq + 2 * m.H, m.D)
        q = qgemv.append_rotated(self.cache, qkv[:, :Hq], qkv[:, Hq:Hq + m.H], qkv[:, Hq + m.H:], start, length, m.freq,
                                 out=torch.empty((T, Hq, m.D), dtype=torch.bfloat16, device=dev))
        most = max(map(len, rows))
        if self.share:
            out = qgemv.attend_shared(self.cache, q, start, length, most, self.common)
        else:
            out = qgemv.attend(self.cache, q, start, length, most)
        y = m.product(m.o, out.view(T, -1), residual=x.float())
        y = y + m.experts_of(y.bfloat16())
        return m.product(m.head, y.bfloat16()), fed, start


def main():
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    a.add_argument("--steps", type=int, default=20)
    a.add_argument("--drafts", type=int, default=3)
    a.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    a = a.parse_args()
    cache = torch.bfloat16 if a.cache == "bf16" else torch.float8_e4m3fn
    system, prompts = list(range(200, 300)), [[1, 2, 3], [70, 80], list(range(100, 110))]
    g = ServedBatch(ServedDecoder(), system, prompts, [0, 1, -1], drafts=a.drafts, cache=cache)
    gained = [g.step() for _ in range(a.steps)]
    for b, t in enumerate(g.tokens):
        n = sum(s[b] for s in gained)
        print(f"request {b}: {n} tokens in {a.steps} steps ({n / a.steps:.2f} a step), {len(t)} in all: ... {t[-8:]}")


if __name__ == "__main__":
    main()
