"""Seeded problems of the verify step's cache operators, and the bounds their
results are held to."""
import numpy as np
import torch

import oracle

STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


class KvProblem:
    """Random pages, rows and lengths on the CPU.  `rows` and `lens` are lists;
    page ids are shuffled over more pages than are used.  poison: every slot
    that no row sees holds NaN (keys and values)."""

    def __init__(self, rows, lens, H=2, G=2, D=128, page=16, q_dtype=torch.bfloat16, dtype=None, window=0, sinks=0,
                 seed=0, poison=False, spare=3, extra_width=1, spread=2.0):
        g = torch.Generator().manual_seed(seed)
        dtype = q_dtype if dtype is None else dtype
        self.rows, self.lens, self.H, self.G, self.D, self.page = list(rows), list(lens), H, G, D, page
        self.window, self.sinks, self.q_dtype, self.dtype = window, sinks, q_dtype, dtype
        self.B, self.M, self.T = len(self.rows), max(max(self.rows), 1), sum(self.rows)
        need = [max(0, -(-n // page)) for n in self.lens]
        self.P = sum(need) + spare
        f8 = dtype == torch.float8_e4m3fn
        k, v = (torch.randn((self.P, page, H, D), generator=g) * (4.0 if f8 else 1.0) for _ in range(2))
        self.k, self.v = k.to(dtype), v.to(dtype)
        self.table = torch.full((self.B, max(1, max(need)) + extra_width), -1, dtype=torch.int32)
        ids = torch.randperm(self.P, generator=g).to(torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.start = torch.tensor([0] + list(np.cumsum(self.rows)), dtype=torch.int32)
        self.len = torch.tensor(self.lens, dtype=torch.int32)
        self.k_scale = (0.25 + 0.05 * torch.rand(H, generator=g)) if f8 else None
        self.v_scale = (0.25 + 0.05 * torch.rand(H, generator=g)) if f8 else None
        self.q = (spread * torch.randn((self.T, H * G, D), generator=g)).to(q_dtype)
        self.scale = D ** -0.5
        if poison:
            self.poison()

    def seen(self):
        """bool [P, page]: the slots that some row sees."""
        m = np.zeros((self.P, self.page), bool)
        table = self.table.numpy()
        for b, r in enumerate(self.rows):
            for i in range(r):
                for j in oracle.visible(self.lens[b] - r + i, self.lens[b], self.window, self.sinks):
                    s = oracle.kv_oracle.slot_of(table, b, int(j), self.page, self.P)
                    if s is not None:
                        m[s] = True
        return torch.from_numpy(m)

    def poison(self):
        hide = ~self.seen()
        for x in (self.k, self.v):
            f = x.float()
            f[hide] = float("nan")
            x.copy_(f.to(x.dtype))

    def reference(self):
        d = lambda x: None if x is None else x.double().numpy()  # noqa: E731
        return oracle.attend_reference(d(self.q), d(self.k), d(self.v), self.table.numpy(), self.start.tolist(),
                                       self.len.tolist(), self.window, self.sinks, self.scale, d(self.k_scale),
                                       d(self.v_scale))

    def check(self, out, lse, ref=None, label=""):
        """The bound counts, for a row that sees n tokens:
        * a score: D products summed in fp32, the scale and the change to
          base 2: ds = (D + 4) 2^-24 size, and 3 roundings of a value up to size;
        * a weight: twice that, the exponential, and one rounding to q's type
          (half a step, relative to the weight; below fp16's normal range
          2^-25 absolute, the largest weight being at least 1);
        * sums of n terms in fp32, once over tokens and once over parts;
        * the output's own rounding (fp16: at least 2^-25)."""
        r = self.reference() if ref is None else ref
        n = r["count"][:, None].astype(np.float64)
        ds = (self.D + 7) * 2.0 ** -24 * r["size"]
        weight = 2 * ds + (2 * n + 16) * 2.0 ** -24
        u = STEP[self.q_dtype]
        tol = u * np.abs(r["out"]) + (weight + u)[..., None] * (1 + u) * r["mass"]
        if self.q_dtype == torch.float16:
            tol = tol + 2.0 ** -25 * (1 + n[..., None] * r["top"])
        o = out.double().cpu().numpy()
        assert o.shape == r["out"].shape
        bad = ~(np.abs(o - r["out"]) <= tol)
        assert not bad.any(), (f"{label}: {bad.sum()} of {bad.size} outputs, first at {tuple(np.argwhere(bad)[0])}: "
                               f"{o[bad][0]} for {r['out'][bad][0]}, tolerance {tol[bad][0]}")
        if lse is not None:
            z = lse.double().cpu().numpy()
            none = np.isneginf(r["lse"])
            assert np.array_equal(np.isneginf(z), none), f"{label}: rows that see nothing"
            ztol = weight + 4 * 2.0 ** -24 * np.abs(np.where(none, 0.0, r["lse"]))
            d = np.abs(np.where(none, 0.0, z) - np.where(none, 0.0, r["lse"]))
            assert (d <= ztol).all(), f"{label}: lse off by {(d / np.maximum(ztol, 1e-300)).max()} of its tolerance"
            assert (o[none] == 0).all(), f"{label}: rows that see nothing give 0"


class KvDevice:
    """A problem's tensors on the GPU."""

    def __init__(self, p, device="cuda:0"):
        from few_row_quantized_amd import qgemv
        to = lambda x: None if x is None else x.to(device)  # noqa: E731
        self.p, self.q, self.start, self.len = p, to(p.q), to(p.start), to(p.len)
        self.k, self.v, self.table = to(p.k), to(p.v), to(p.table)
        self.k_scale, self.v_scale = to(p.k_scale), to(p.v_scale)
        self.cache = qgemv.KvCache(self.k, self.v, self.table, self.k_scale, self.v_scale)

    def attend(self, lse=True, **kw):
        from few_row_quantized_amd import qgemv
        p = self.p
        z = torch.full((p.T, p.H * p.G), float("nan"), device=self.q.device) if lse is True else lse
        kw.setdefault("scale", p.scale)
        out = qgemv.attend(self.cache, self.q, self.start, self.len, kw.pop("M", p.M), window=p.window, sinks=p.sinks,
                           lse=z, **kw)
        torch.cuda.synchronize()
        return out, z


def draft_problem(rows, V, dtype=torch.float32, drafts=True, seed=0, agree=0.7):
    """p, q (or None), tokens, u, start on the CPU: peaked probabilities, a
    draft model near the target."""
    g = torch.Generator().manual_seed(seed)
    T = sum(rows)
    a = 4.0 * torch.randn((T, V), generator=g)
    p = torch.softmax(a, -1).to(dtype)
    b = a + agree * torch.randn((T, V), generator=g)
    q = torch.softmax(b, -1).to(dtype)
    d = torch.multinomial(torch.softmax(b, -1), 1, generator=g)[:, 0].to(torch.int32)
    start = torch.tensor([0] + list(np.cumsum(rows)), dtype=torch.int32)
    return p, q if drafts else None, torch.roll(d, 1).contiguous(), torch.rand(T, generator=g), start
