"""More operators of a verify step, for models and batches as they are served:
attention of a batch whose sequences share a long prefix, the cache append with
the rotation of positions on the way, the routing of rows to experts, and
low-rank adapters of many requests beside a shared projection.

run() computes them in a plain form of elementary torch operations (`own`
false) or through the framework's entry points (`own` true), on what prepare()
hands over.  exact() evaluates the definitions in 64 bits.

Shapes follow a serving engine: B sequences, sequence b with rows[b] <= M new
rows (its last accepted token and the drafts after it) and lens[b] cached
tokens, those rows included; H key-value heads, G query heads on each, D
values a head; pages of `page` slots, found through a page table.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16,
         "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}


# ---------------------------------------------------------------- cases

def _shared(name, B, M, H, G, D, shared, lo, hi, page, q, cache, window=0, sinks=0):
    """lo..hi: a sequence's own tokens after the shared ones."""
    return {"name": name, "op": "shared", "B": B, "M": M, "H": H, "G": G, "D": D, "shared": shared, "lo": lo,
            "hi": hi, "page": page, "q": q, "cache": cache, "window": window, "sinks": sinks}


def _rotate(name, B, M, H, G, D, R, lo, hi, page, new, cache, axes=0, interleaved=False, far=0):
    """R: rotated values of a head; axes: position axes given (0: the row's own
    place in the cache); far: given positions reach this far past the place."""
    return {"name": name, "op": "rotate", "B": B, "M": M, "H": H, "G": G, "D": D, "R": R, "lo": lo, "hi": hi,
            "page": page, "new": new, "cache": cache, "axes": axes, "interleaved": interleaved, "far": far}


def _route(name, T, E, k, logits, score, bias=False, groups=1, keep=1, best=1, renormalise=True, masked=False):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "logits": logits, "score": score, "bias": bias,
            "groups": groups, "keep": keep, "best": best, "renormalise": renormalise, "masked": masked}


def _adapt(name, B, M, n, r, K, N, x, none=False):
    return {"name": name, "op": "adapt", "B": B, "M": M, "n": n, "r": r, "K": K, "N": N, "x": x, "none": none}


def listed():
    return [
        # four requests just begun on one system prompt, one token each: latency
        _shared("shared_decode4", 4, 1, 8, 6, 128, 1000, 20, 200, 16, "bf16", "bf16"),
        # verify of a batch over an 8-bit cache, an odd page size, a prefix that ends inside a page
        _shared("shared_verify4_e4m3", 24, 4, 8, 6, 128, 6001, 0, 2500, 20, "bf16", "e4m3"),
        # a window layer with sinks, the widest verify: the window reaches back into the prefix
        _shared("shared_window_sinks16", 16, 16, 8, 4, 64, 8192, 100, 3900, 64, "f16", "f16", 4096, 4),
        # the largest: a full batch on a long common prompt, eight verified rows each
        _shared("shared_verify8_full", 64, 8, 8, 6, 128, 16384, 500, 2000, 16, "bf16", "bf16"),
        # the rows of one request's verify (products leave fp32)
        _rotate("rotate_one_request", 1, 5, 8, 6, 128, 128, 4000, 4000, 16, "f32", "bf16"),
        # a full batch into an 8-bit cache, positions of three axes (time, height, width)
        _rotate("rotate_batch_axes_e4m3", 256, 16, 8, 6, 128, 128, 100, 700, 32, "f32", "e4m3", 3),
        # neighbours rotated in a quarter of wide heads, far positions, odd pages
        _rotate("rotate_far_partial", 33, 7, 4, 3, 256, 64, 100, 900, 20, "f16", "f16", 1, True, 1 << 20),
        # one request's verify through 128 experts, 8 a row
        _route("route_one_request", 5, 128, 8, "f32", "softmax"),
        # a batch through 256 experts in 8 groups, chosen with a bias for balance
        _route("route_batch_groups", 4096, 256, 8, "bf16", "sigmoid", True, 8, 4, 2),
        # one request's verify beside the query projection of the 27B-class layer
        _adapt("adapt_one_request", 1, 5, 8, 16, 5120, 6144, "bf16"),
        # a batch with an adapter for every other request, beside the up projection
        _adapt("adapt_batch", 64, 8, 32, 64, 5120, 17408, "bf16"),
        # odd sizes, one row a request, some requests without an adapter
        _adapt("adapt_decode_odd", 77, 1, 5, 8, 1000, 2051, "f16", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("shared", "shared", "rotate", "rotate", "route", "adapt", "adapt"))
    M = rng.randint(1, 16)
    H = rng.choice((1, 2, 4, 5, 8))
    D = rng.choice((64, 128, 128, 256))
    page = rng.choice((1, 8, 16, 16, 20, 32, 64, 128))
    if op == "shared":
        G = rng.choice((1, 2, 3, 4, 6, 8, 12))
        q = rng.choice(("bf16", "f16"))
        shared = _log(rng, 40, 16384)
        hi = _log(rng, 1, 3000)
        most = min(64 * 18000 * 1024 // ((shared + hi) * H * D), 64 * 8 * 48 * 18000 // ((shared + hi) * M * H * G))
        B = _log(rng, 1, max(1, min(128, most)))
        window = rng.choice((0, 0, _log(rng, 16, 8192)))
        c = _shared("", B, M, H, G, D, shared, rng.randint(0, hi), hi, page, q, rng.choice((q, q, "e4m3")), window,
                    rng.choice((0, 1, 4, 64)) if window else 0)
    elif op == "rotate":
        hi = _log(rng, 20, 1000)
        axes = rng.choice((0, 1, 3))
        c = _rotate("", _log(rng, 1, 256), M, H, rng.choice((1, 2, 3, 4, 6, 8)), D, 16 * rng.randint(1, D // 16),
                    rng.randint(1, hi), hi, page, rng.choice(("f32", "bf16", "f16")),
                    rng.choice(("bf16", "f16", "e4m3")), axes, rng.random() < 0.5, rng.choice((0, 1 << 20)) if axes else 0)
    elif op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        E = groups * _log(rng, 8, 512 // groups)
        keep = rng.randint(1, groups)
        c = _route("", _log(rng, 1, 4096), E, rng.randint(1, min(12, E // groups * keep)),
                   rng.choice(("f32", "bf16", "f16")), rng.choice(("softmax", "sigmoid")), rng.random() < 0.5, groups,
                   keep, rng.choice((1, 2)) if groups > 1 else 1, rng.random() < 0.8, rng.random() < 0.3)
    else:
        r = rng.choice((8, 16, 16, 32, 64, 128))
        K = 8 * _log(rng, 32, 17408 // 8)
        N = _log(rng, 64, 17408)
        B = _log(rng, 1, max(1, min(128, 512 * 64 * 22528 // (M * r * (K + N)))))
        c = _adapt("", B, M, _log(rng, 1, 64), r, K, N, rng.choice(("bf16", "bf16", "f16")), rng.random() < 0.4)
    del c["name"]
    return c


def _layout(case):
    """rows[b] and lens[b]: from the case alone, so that a case has one size."""
    r = random.Random(1000 * case["B"] + case["M"])
    B, M = case["B"], case["M"]
    rows = [M if b % 3 != 2 else r.randint(1, M) for b in range(B)]
    base = case.get("shared", 0)
    lens = [base + max(rows[b], r.randint(case["lo"], case["hi"])) for b in range(B)]
    lens[0] = base + max(rows[0], case["hi"])
    return rows, lens


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    if case["op"] == "route":
        return _prepare_route(case, dev, g)
    if case["op"] == "adapt":
        return _prepare_adapt(case, dev, g, seed)
    rows, lens = _layout(case)
    B, H, G, D, page = (case[x] for x in ("B", "H", "G", "D", "page"))
    T, need = sum(rows), [-(-n // page) for n in lens]
    both = case.get("shared", 0) // page  # whole pages that all sequences have in common
    P = sum(n - both for n in need) + both + 3
    cache = TYPES[case["cache"]]

    def pages():
        t = torch.empty((P, page, H, D), dtype=cache, device=dev)
        step = max(1, (1 << 28) // (page * H * D))
        for i in range(0, P, step):
            x = torch.randn((min(step, P - i), page, H, D), generator=g, device=dev)
            t[i:i + step] = x.mul_(4.0 if case["cache"] == "e4m3" else 1.0).to(cache)
        return t

    k, v = pages(), pages()
    # page ids in any order; entries past a sequence's length hold nothing
    table = torch.full((B, max(1, max(need))), -1, dtype=torch.int32)
    ids = torch.randperm(P, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    at = both
    for b in range(B):
        table[b, :both] = ids[:both]
        table[b, both:need[b]] = ids[at:at + need[b] - both]
        at += need[b] - both
    if both < -(-case.get("shared", 0) // page):
        # a prefix that ends inside a page: its last tokens stand in each sequence's own page
        own_page = table[:, both].long().to(dev)
        part = case["shared"] - both * page
        k[own_page, :part] = k[own_page[0], :part].clone()
        v[own_page, :part] = v[own_page[0], :part].clone()
    s = {"case": case, "T": T, "k": k, "v": v, "table": table.to(dev)}
    s["len"] = torch.tensor(lens, dtype=torch.int32).to(dev)
    starts = [0]
    for r in rows:
        starts.append(starts[-1] + r)
    s["start"] = torch.tensor(starts, dtype=torch.int32).to(dev)
    s["k_scale"] = s["v_scale"] = None
    if case["cache"] == "e4m3":
        s["k_scale"] = 0.25 + 0.02 * torch.rand(H, generator=g, device=dev)
        s["v_scale"] = 0.25 + 0.02 * torch.rand(H, generator=g, device=dev)
    if case["op"] == "shared":
        # queries twice as long as the keys: scores spread as in a peaked softmax
        s["q"] = (2.0 * torch.randn((T, H * G, D), generator=g, device=dev)).to(TYPES[case["q"]])
        s["scale"] = D ** -0.5
        s["shared"] = torch.tensor([case["shared"]], dtype=torch.int32, device=dev)
    else:
        _prepare_rotate(s, rows, lens, dev, g)
    if own:
        from few_row_quantized_amd import qgemv
        s["cache"] = qgemv.KvCache(k, v, s["table"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        if case["op"] == "shared":
            s["work"] = qgemv.attend_shared_workspace(s["cache"], case["M"], H * G, T)
            s["lse"] = torch.empty((T, H * G), dtype=torch.float32, device=dev)
    return s


def _prepare_rotate(s, rows, lens, dev, g):
    c = s["case"]
    H, G, D, pairs = c["H"], c["G"], c["D"], c["R"] // 2
    new = TYPES[c["new"]]
    # one product's columns: queries, keys, values
    qkv = torch.randn((s["T"], H * (G + 2), D), generator=g, device=dev).to(new)
    s["q"], s["new_k"], s["new_v"] = qkv[:, :H * G], qkv[:, H * G:H * (G + 1)], qkv[:, H * (G + 1):]
    s["freq"] = (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().to(dev)
    s["out_type"] = TYPES["bf16"] if c["cache"] == "e4m3" else TYPES[c["cache"]]
    s["position"] = s["axes"] = None
    if c["axes"]:
        place = torch.tensor([n - r + i for r, n in zip(rows, lens) for i in range(r)], dtype=torch.int32)
        at = torch.randint(0, c["far"] + 1, (s["T"],), generator=g, device=dev, dtype=torch.int32) + place.to(dev)
        if c["axes"] == 1:
            s["position"] = at[None].contiguous()
        else:  # a picture's rows and columns beside the time
            hw = torch.randint(0, 64, (2, s["T"]), generator=g, device=dev, dtype=torch.int32)
            s["position"] = torch.cat([at[None], at[None] + hw]).contiguous()
            # a quarter of the pairs for the time, the rest shared by height and width
            i = torch.arange(pairs)
            first = pairs // 4
            s["axes"] = torch.where(i < first, 0, 1 + (i - first) * 2 // max(1, pairs - first)).to(torch.int32).to(dev)


def _prepare_route(case, dev, g):
    T, E = case["T"], case["E"]
    x = 2.0 * torch.randn((T, E), generator=g, device=dev)
    if case["masked"]:  # experts that are not there for a row
        x[torch.rand((T, E), generator=g, device=dev) < 0.1] = float("-inf")
    s = {"case": case, "logits": x.to(TYPES[case["logits"]]), "bias": None}
    if case["bias"]:
        s["bias"] = 0.1 * torch.randn(E, generator=g, device=dev)
    return s


def _prepare_adapt(case, dev, g, seed):
    t = TYPES[case["x"]]
    B, M, n, r, K, N = (case[x] for x in ("B", "M", "n", "r", "K", "N"))
    choice = random.Random(1000 * B + M)
    rows = [M if b % 3 != 2 else choice.randint(1, M) for b in range(B)]
    of = _adapters(case)
    T = sum(rows)
    s = {"case": case, "T": T}
    s["x"] = torch.randn((T, K), generator=g, device=dev).to(t)
    s["y"] = torch.randn((T, N), generator=g, device=dev)
    s["a"] = (torch.randn((n, r, K), generator=g, device=dev) * K ** -0.5).to(t)
    s["b"] = torch.randn((n, N, r), generator=g, device=dev).mul_(r ** -0.5).to(t)
    s["scales"] = 0.5 + torch.rand(n, generator=g, device=dev)
    s["adapter"] = torch.tensor([a for a, m in zip(of, rows) for _ in range(m)], dtype=torch.int32).to(dev)
    if own:
        from few_row_quantized_amd import qgemv
        s["work"] = qgemv.adapt_workspace(s["a"], T)
    return s


def _adapters(case):
    """The adapter of each sequence."""
    r = random.Random(7000 + case["B"])
    of = [r.randrange(case["n"]) for _ in range(case["B"])]
    if case["none"]:
        of = [-1 if r.random() < 0.3 else a for a in of]
        of[0] = case["n"] - 1
    return of


# ---------------------------------------------------------------- one pass

def run(state):
    return {"shared": _run_shared, "rotate": _run_rotate, "route": _run_route, "adapt": _run_adapt}[
        state["case"]["op"]](state)


def _run_shared(s):
    if not own:
        return _plain_attend(s)
    from few_row_quantized_amd import qgemv
    c = s["case"]
    out = qgemv.attend_shared(s["cache"], s["q"], s["start"], s["len"], c["M"], s["shared"], window=c["window"],
                              sinks=c["sinks"], scale=s["scale"], lse=s["lse"], workspace=s["work"])
    return {"out": out, "lse": s["lse"]}


def _run_rotate(s):
    if own:
        from few_row_quantized_amd import qgemv
        q = qgemv.append_rotated(s["cache"], s["q"], s["new_k"], s["new_v"], s["start"], s["len"], s["freq"],
                                 position=s["position"], axes=s["axes"], interleaved=s["case"]["interleaved"])
    else:
        q = _plain_rotate(s)
    return {"q": q, "k": s["k"], "v": s["v"]}


def _run_route(s):
    if not own:
        return _plain_route(s)
    from few_row_quantized_amd import qgemv
    c = s["case"]
    experts, weights = qgemv.route(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                                   keep=c["keep"], best=c["best"], renormalise=c["renormalise"], scale=2.5)
    return {"experts": experts, "weights": weights}


def _run_adapt(s):
    if not own:
        return {"out": _plain_adapt(s)}
    from few_row_quantized_amd import qgemv
    return {"out": qgemv.adapt(s["y"], s["x"], s["a"], s["b"], s["adapter"], scales=s["scales"], workspace=s["work"])}


# ---------------------------------------------------------------- plain forms

def _row_places(s, dev):
    """For each row: its sequence, and its position in that sequence's cache."""
    t = torch.arange(s["T"], device=dev, dtype=torch.int64)
    start, length = s["start"].long(), s["len"].long()
    seq = torch.searchsorted(start[1:].contiguous(), t, right=True)
    return seq, length[seq] - (start[seq + 1] - t)


def _plain_attend(s):
    c = s["case"]
    B, M, H, G, D, page = (c[x] for x in ("B", "M", "H", "G", "D", "page"))
    dev = s["q"].device
    start, length = s["start"].long(), s["len"].long()
    table = s["table"].long().clamp(min=0)
    L = table.shape[1] * page
    both = c["shared"] // page * page  # tokens in pages that all sequences have
    rows = start[1:] - start[:-1]
    # the rows of each sequence, padded to M
    m = torch.arange(M, device=dev)
    real = m[None, :] < rows[:, None]
    t = (start[:-1, None] + m[None, :]).clamp(max=s["T"] - 1)
    q = s["q"][t].float().view(B, M, H, G, D).permute(0, 2, 1, 3, 4)  # [B, H, M, G, D]
    factor = s["scale"] if s["k_scale"] is None else (s["scale"] * s["k_scale"]).view(1, H, 1, 1, 1)
    pos = (length[:, None] - rows[:, None] + m[None, :])[:, :, None]

    def sees(j):
        j = j[None, None, :]
        x = (j <= pos) & real[:, :, None]
        if c["window"]:
            x &= (j > pos - c["window"]) | (j < c["sinks"])
        return x[:, None, :, None, :]

    none = float("-inf")
    # scores over the common tokens, all sequences' rows as one product a head
    first = table[0, :both // page]
    k = s["k"][first].reshape(both, H, D).permute(1, 2, 0).float()
    score = torch.matmul(q.transpose(0, 1).reshape(H, B * M * G, D), k).view(H, B, M, G, both).transpose(0, 1)
    score = torch.where(sees(torch.arange(both, device=dev)), score * factor, none)
    # and over each sequence's own
    own_table = table[:, both // page:]
    k = s["k"][own_table].reshape(B, L - both, H, D).permute(0, 2, 3, 1).float()
    rest = torch.matmul(q.reshape(B, H, M * G, D), k).view(B, H, M, G, L - both)
    del k
    rest = torch.where(sees(torch.arange(both, L, device=dev)), rest * factor, none)
    top = rest.amax(-1, keepdim=True)
    if both:
        top = torch.maximum(top, score.amax(-1, keepdim=True))
    top = torch.where(top == none, 0.0, top)
    score = torch.exp(score - top)
    rest = torch.exp(rest - top)
    total = score.sum(-1, keepdim=True) + rest.sum(-1, keepdim=True)
    v = s["v"][first].reshape(both, H, D).transpose(0, 1).float()
    out = torch.matmul(score.transpose(0, 1).reshape(H, B * M * G, both), v).view(H, B, M, G, D).transpose(0, 1)
    v = s["v"][own_table].reshape(B, L - both, H, D).permute(0, 2, 1, 3).float()
    # slots past the length may hold anything
    v = torch.where((torch.arange(both, L, device=dev) < length[:, None])[:, None, :, None], v, 0.0)
    out = out + torch.matmul(rest.view(B, H, M * G, L - both), v).view(B, H, M, G, D)
    del v
    out = torch.where(total > 0, out / total, 0.0)
    if s["v_scale"] is not None:
        out = out * s["v_scale"].view(1, H, 1, 1, 1)
    lse = (top + torch.log(total)).squeeze(-1)
    out = out.permute(0, 2, 1, 3, 4).reshape(B, M, H * G, D)[real]
    lse = lse.permute(0, 2, 1, 3).reshape(B, M, H * G)[real]
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _plain_rotate(s):
    c = s["case"]
    k, v, page, R = s["k"], s["v"], c["page"], c["R"]
    seq, pos = _row_places(s, k.device)
    # angles in 64 bits: positions reach millions of turns
    pairs = R // 2
    if s["position"] is None:
        at = pos.double()[:, None]
    else:
        axes = torch.zeros(pairs, dtype=torch.int64, device=k.device) if s["axes"] is None else s["axes"].long()
        at = s["position"].double()[axes].T
    angle = at * s["freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def rotate(x):
        x = x.float()
        y = x.clone()
        if c["interleaved"]:
            a, b = x[..., 0:R:2], x[..., 1:R:2]
            y[..., 0:R:2], y[..., 1:R:2] = a * cos - b * sin, a * sin + b * cos
        else:
            a, b = x[..., :pairs], x[..., pairs:R]
            y[..., :pairs], y[..., pairs:R] = a * cos - b * sin, a * sin + b * cos
        return y

    slot = s["table"].long()[seq, pos // page]
    new_k, new_v = rotate(s["new_k"]), s["new_v"].float()
    if s["k_scale"] is not None:  # 8 bits: the values over the head's scale, at most 448 large
        new_k = (new_k / s["k_scale"][None, :, None]).clamp(-448.0, 448.0)
        new_v = (new_v / s["v_scale"][None, :, None]).clamp(-448.0, 448.0)
    k[slot, pos % page] = new_k.to(k.dtype)
    v[slot, pos % page] = new_v.to(v.dtype)
    return rotate(s["q"]).to(s["out_type"])


def _plain_route(s):
    c = s["case"]
    T, E, k, groups = c["T"], c["E"], c["k"], c["groups"]
    none = float("-inf")
    # 64 bits: values near the border of the choice
    x = s["logits"].double()
    if c["score"] == "softmax":
        top = x.amax(-1, keepdim=True)
        e = torch.exp(x - torch.where(top == none, 0.0, top))
        score = e / e.sum(-1, keepdim=True).clamp(min=1e-300)
    else:
        score = torch.where(x >= 0, 1.0, torch.exp(x)) / (1.0 + torch.exp(-x.abs()))
    choice = x if s["bias"] is None and c["best"] == 1 else score
    if s["bias"] is not None:
        choice = choice + s["bias"].double()
    choice = torch.where(x == none, none, choice)
    if groups > 1:
        each = torch.sort(choice.view(T, groups, E // groups), -1, descending=True)[0][..., :c["best"]]
        some = each[..., 0] > none
        group = torch.where(some, torch.where(each > none, each, 0.0).sum(-1), none)
        order = torch.sort(group, dim=-1, descending=True, stable=True)[1][:, :c["keep"]]
        kept = torch.zeros((T, groups), device=x.device).scatter_(1, order, 1.0) > 0
        choice = torch.where(kept[..., None], choice.view(T, groups, -1), none).view(T, E)
    value, experts = torch.sort(choice, dim=-1, descending=True, stable=True)
    value, experts = value[:, :k], experts[:, :k]
    there = value > none
    w = torch.where(there, score.gather(1, experts), 0.0)
    if c["renormalise"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return {"experts": torch.where(there, experts, -1).to(torch.int32), "weights": (w * 2.5).float()}


def _plain_adapt(s):
    c = s["case"]
    x, out, n = s["x"].float(), s["y"].clone(), c["n"]
    at = s["adapter"].long()
    has = (at >= 0) & (at < n)
    at = at.clamp(0, n - 1)
    factor = torch.where(has, s["scales"][at], 0.0)[:, None]
    step = max(1, (1 << 28) // (c["r"] * max(c["K"], c["N"])))
    for i in range(0, s["T"], step):
        j = at[i:i + step]
        v = torch.matmul(s["a"][j].float(), x[i:i + step, :, None])
        d = torch.matmul(s["b"][j].float(), v)[..., 0]
        out[i:i + step] += factor[i:i + step] * d
    return out


# ---------------------------------------------------------------- cost

def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * SIZE[case["logits"]] + 8 * T * k + (4 * E if case["bias"] else 0), "flops": 6 * T * E}
    if op == "adapt":
        n, r, K, N = (case[x] for x in ("n", "r", "K", "N"))
        choice = random.Random(1000 * case["B"] + case["M"])
        rows = [case["M"] if b % 3 != 2 else choice.randint(1, case["M"]) for b in range(case["B"])]
        of, T = _adapters(case), sum(rows)
        used = len({a for a in of if a >= 0})
        adapted = sum(m for a, m in zip(of, rows) if a >= 0)
        return {"bytes": 2 * used * r * (K + N) + 2 * adapted * K + 8 * T * N + 4 * T,
                "flops": 2 * adapted * r * (K + N)}
    rows, lens = _layout(case)
    H, D, T = case["H"], case["D"], sum(rows)
    Hq = H * case["G"]
    if op == "rotate":
        out = 2 * T * Hq * D
        return {"bytes": T * (Hq + 2 * H) * D * SIZE[case["new"]] + out + 2 * T * H * D * SIZE[case["cache"]],
                "flops": 3 * T * (Hq + H) * D}
    # each token that some row sees once: the common ones of all sequences together
    both = case["shared"] // case["page"] * case["page"]
    pairs = slots = 0
    first = both
    for r, n in zip(rows, lens):
        for i in range(r):
            pos = n - r + i
            low = max(0, pos - case["window"] + 1) if case["window"] else 0
            pairs += pos + 1 - low + min(case["sinks"], low)
        low = max(0, n - r - case["window"] + 1) if case["window"] else 0
        first = min(first, low)
        slots += n - max(low, both) + max(0, min(case["sinks"], low) - both)
    slots += both - first + min(case["sinks"], first)
    return {"bytes": 2 * slots * H * D * SIZE[case["cache"]] + 2 * T * Hq * D * SIZE[case["q"]] + 4 * T * Hq,
            "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"shared": _exact_attend, "rotate": _exact_rotate, "route": _exact_route, "adapt": _exact_adapt}[
        case["op"]](s)


def _exact_attend(s):
    """Row by row over the sequence's whole page list."""
    c = s["case"]
    H, G, D, page = (c[x] for x in ("H", "G", "D", "page"))
    dev = s["q"].device
    starts, lens = s["start"].tolist(), s["len"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.full(s["q"].shape[:2], float("-inf"), dtype=torch.float64, device=dev)
    one = torch.ones(H, device=dev)
    ks = (one if s["k_scale"] is None else s["k_scale"]).double()
    vs = (one if s["v_scale"] is None else s["v_scale"]).double()
    for b, n in enumerate(lens):
        token = torch.arange(n, device=dev)
        flat = s["table"][b].long()[token // page] * page + token % page
        k = s["k"].view(-1, H, D)[flat].double() * ks[:, None]
        v = s["v"].view(-1, H, D)[flat].double() * vs[:, None]
        k, v = k.permute(1, 2, 0).contiguous(), v.transpose(0, 1).contiguous()
        for t in range(starts[b], starts[b + 1]):
            last = n - (starts[b + 1] - t)
            a = torch.matmul(s["q"][t].double().view(H, G, D), k) * s["scale"]
            hide = token > last
            if c["window"]:
                hide |= (token <= last - c["window"]) & (token >= c["sinks"])
            a[..., hide] = float("-inf")
            z = torch.logsumexp(a, -1)
            lse[t] = z.flatten()
            out[t] = torch.matmul(torch.exp(a - z[..., None]), v).view(H * G, D)
    return {"out": out, "lse": lse}


def _exact_rotate(s):
    c = s["case"]
    page, D, R = c["page"], c["D"], c["R"]
    dev = s["k"].device
    starts, lens, table = s["start"].tolist(), s["len"].tolist(), s["table"].tolist()
    places, where = [], []
    for b, n in enumerate(lens):
        for t in range(starts[b], starts[b + 1]):
            p = n - (starts[b + 1] - t)
            places.append(p)
            where.append(table[b][p // page] * page + p % page)
    where = torch.tensor(where, device=dev)
    # the value at d turns with its partner: out = x cos + (sign) partner sin
    pair, partner, sign = [], list(range(D)), [0.0] * D
    for d in range(R):
        i, upper = (d // 2, d % 2 == 1) if c["interleaved"] else (d % (R // 2), d >= R // 2)
        pair.append(i)
        partner[d] = (d ^ 1) if c["interleaved"] else (d + R // 2) % R
        sign[d] = 1.0 if upper else -1.0
    angle = torch.zeros((s["T"], D), dtype=torch.float64, device=dev)
    for d in range(R):
        i = pair[d]
        if s["position"] is None:
            at = torch.tensor(places, dtype=torch.float64, device=dev)
        else:
            at = s["position"][0 if s["axes"] is None else int(s["axes"][i])].double()
        angle[:, d] = at * s["freq"][i].double()
    cos, sin = torch.cos(angle)[:, None], (torch.sin(angle) * torch.tensor(sign, device=dev).double())[:, None]

    def turn(x):
        x = x.double()
        return x * cos + x[..., partner] * sin

    got = {"q": turn(s["q"])}
    for name, new, scale in (("k", turn(s["new_k"]), s["k_scale"]), ("v", s["new_v"].double(), s["v_scale"])):
        x = s[name].double()
        if scale is not None:
            new = (new / scale.double()[:, None]).clamp(-448.0, 448.0)
        x.view(-1, *x.shape[2:])[where] = new
        got[name] = x
    return got


def _exact_route(s):
    import numpy as np
    c = s["case"]
    x = s["logits"].double().cpu().numpy()
    T, E, k, size = c["T"], c["E"], c["k"], c["E"] // c["groups"]
    bias = None if s["bias"] is None else s["bias"].double().cpu().numpy()
    experts, weights = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        there = [e for e in range(E) if x[t, e] > -np.inf]
        if not there:
            continue
        z = x[t] - x[t, there].max()
        p = np.exp(z) / np.exp(z).sum() if c["score"] == "softmax" else 1.0 / (1.0 + np.exp(-x[t]))
        # without a bias the scores' order is the logits'
        value = (p + bias) if bias is not None else (p if c["best"] == 2 else x[t])
        if c["groups"] > 1:
            best = {}
            for g in range(c["groups"]):
                members = sorted((value[e] for e in there if e // size == g), reverse=True)
                if members:
                    best[g] = sum(members[:c["best"]])
            kept = sorted(best, key=lambda g: (-best[g], g))[:c["keep"]]
            there = [e for e in there if e // size in kept]
        chosen = sorted(there, key=lambda e: (-value[e], e))[:k]
        w = p[chosen]
        if c["renormalise"]:
            w = w / w.sum()
        experts[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = 2.5 * w
    dev = s["logits"].device
    return {"experts": torch.tensor(experts, device=dev), "weights": torch.tensor(weights, device=dev)}


def _exact_adapt(s):
    out = s["y"].double()
    for i in range(s["case"]["n"]):
        rows = (s["adapter"] == i).nonzero()[:, 0]
        if rows.numel():
            v = s["x"][rows].double() @ s["a"][i].double().T
            out[rows] += float(s["scales"][i]) * (v @ s["b"][i].double().T)
    return {"out": out}
