"""The operators of a verify step that sit around the quantized products: appending
the draft rows' keys and values to a paged cache, attention of those few rows
over the cache, and the acceptance of the drafted tokens.

run() computes them in a plain form of elementary torch operations (`own`
false) or through the framework's entry points (`own` true), on what prepare()
hands over.  exact() evaluates the definitions in 64 bits, sequence by
sequence.

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

def _attend(name, B, M, H, G, D, lo, hi, page, q, cache, window=0, sinks=0, empty=False):
    return {"name": name, "op": "attend", "B": B, "M": M, "H": H, "G": G, "D": D, "lo": lo, "hi": hi,
            "page": page, "q": q, "cache": cache, "window": window, "sinks": sinks, "empty": empty}


def _append(name, B, M, H, D, lo, hi, page, new, cache):
    return {"name": name, "op": "append", "B": B, "M": M, "H": H, "D": D, "lo": lo, "hi": hi,
            "page": page, "new": new, "cache": cache, "empty": False}


def _verify(name, B, M, V, p, drafts):
    return {"name": name, "op": "verify", "B": B, "M": M, "V": V, "p": p, "drafts": drafts}


def listed():
    return [
        # one request, one token, a short prompt: the call's own latency
        _attend("attend_one_token_short", 1, 1, 8, 6, 128, 200, 200, 16, "bf16", "bf16"),
        # one request, five verified rows, a long prompt: the heads of the 27B-class
        # layer (q 6144, k and v 1024 wide); only splitting the length fills the card
        _attend("attend_verify5_long", 1, 5, 8, 6, 128, 32768, 32768, 16, "bf16", "bf16"),
        # plain decoding of a ragged batch
        _attend("attend_decode_ragged", 64, 1, 8, 6, 128, 300, 8000, 16, "bf16", "bf16"),
        # verify of a batch over an 8-bit cache
        _attend("attend_verify4_e4m3", 32, 4, 8, 6, 128, 1000, 16000, 32, "bf16", "e4m3"),
        # a window layer with sinks over long contexts, the widest verify
        _attend("attend_window_sinks16", 16, 16, 8, 4, 64, 5000, 30000, 64, "f16", "f16", 4096, 4),
        # wide heads, an odd page size and head group, lengths that end anywhere, one
        # sequence with nothing cached
        _attend("attend_odd_d256", 9, 3, 4, 3, 256, 77, 6001, 20, "bf16", "bf16", 0, 0, True),
        # the largest: a full batch of long contexts, eight verified rows each
        _attend("attend_verify8_full", 64, 8, 8, 6, 128, 8000, 16384, 16, "bf16", "bf16"),
        # the rows of one request's verify (products leave fp32)
        _append("append_one_request", 1, 5, 8, 128, 4000, 4000, 16, "f32", "bf16"),
        # the rows of a full batch into an 8-bit cache
        _append("append_batch_e4m3", 256, 16, 8, 128, 500, 2000, 32, "f32", "e4m3"),
        # one request, four drafts, a small vocabulary
        _verify("verify_one_request", 1, 5, 32000, "f32", True),
        # a batch, seven drafts each, a large vocabulary
        _verify("verify_batch", 64, 8, 151936, "f32", True),
        # drafts without probabilities (a lookup drafter), 16-bit probabilities, an odd vocabulary
        _verify("verify_lookup_bf16", 200, 4, 128257, "bf16", False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attend", "attend", "attend", "append", "verify"))
    if op == "verify":
        M = rng.randint(1, 16)
        V = _log(rng, 1000, 160000)
        B = _log(rng, 1, max(1, min(256, 64 * 8 * 151936 // (M * V))))
        c = _verify("", B, M, V, rng.choice(("f32", "f32", "bf16", "f16")), rng.random() < 0.7)
        del c["name"]
        return c
    M = rng.randint(1, 16)
    H = rng.choice((1, 2, 4, 5, 8))
    D = rng.choice((64, 128, 128, 256))
    page = rng.choice((1, 8, 16, 16, 20, 32, 64, 128))
    if op == "append":
        hi = _log(rng, 20, 2000)
        B = _log(rng, 1, 256)
        c = _append("", B, M, H, D, rng.randint(1, hi), hi, page, rng.choice(("f32", "bf16", "f16")),
                    rng.choice(("bf16", "f16", "e4m3")))
        del c["name"]
        return c
    G = rng.choice((1, 2, 3, 4, 6, 8, 12))
    q = rng.choice(("bf16", "f16"))
    hi = _log(rng, 40, 32768)
    # tokens, rows and their products stay below those of the largest listed case
    most = min(64 * 16384 * 1024 // (hi * H * D), 64 * 8 * 48 * 16384 // (hi * M * H * G))
    B = _log(rng, 1, max(1, min(256, most)))
    window = rng.choice((0, 0, _log(rng, 16, 8192)))
    c = _attend("", B, M, H, G, D, rng.randint(1, hi), hi, page, q, rng.choice((q, q, "e4m3")), window,
                rng.choice((0, 1, 4, 64)) if window else 0, rng.random() < 0.3)
    del c["name"]
    return c


def _layout(case):
    """rows[b] and lens[b]: from the case alone, so that a case has one size."""
    r = random.Random(1000 * case["B"] + case["M"])
    B, M = case["B"], case["M"]
    rows = [M if b % 3 != 2 else r.randint(1, M) for b in range(B)]
    lens = [max(rows[b], r.randint(case["lo"], case["hi"])) for b in range(B)]
    lens[0] = max(rows[0], case["hi"])
    if case["empty"]:
        lens[-1] = 0  # its rows see nothing
    return rows, lens


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    if case["op"] == "verify":
        return _prepare_verify(case, dev, g)
    rows, lens = _layout(case)
    B, H, D, page = case["B"], case["H"], case["D"], case["page"]
    T, need = sum(rows), [-(-n // page) for n in lens]
    P = sum(need) + 3
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
    ids = torch.randperm(P, generator=torch.Generator().manual_seed(seed))[:sum(need)].to(torch.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
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
    if case["op"] == "append":
        s["new_k"] = torch.randn((T, H, D), generator=g, device=dev).to(TYPES[case["new"]])
        s["new_v"] = torch.randn((T, H, D), generator=g, device=dev).to(TYPES[case["new"]])
    else:
        # queries twice as long as the keys: scores spread as in a peaked softmax
        s["q"] = (2.0 * torch.randn((T, H * case["G"], D), generator=g, device=dev)).to(TYPES[case["q"]])
        s["scale"] = D ** -0.5
    if own:
        from few_row_quantized_amd import qgemv
        s["cache"] = qgemv.KvCache(k, v, s["table"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        if case["op"] == "attend":
            s["work"] = qgemv.attend_workspace(s["cache"], case["M"], H * case["G"], T)
            s["lse"] = torch.empty((T, H * case["G"]), dtype=torch.float32, device=dev)
    return s


def _prepare_verify(case, dev, g):
    r = random.Random(1000 * case["B"] + case["M"])
    B, M, V = case["B"], case["M"], case["V"]
    rows = [M if b % 3 != 2 else r.randint(1, M) for b in range(B)]
    T = sum(rows)
    p = torch.empty((T, V), dtype=TYPES[case["p"]], device=dev)
    q = torch.empty((T, V), dtype=TYPES[case["p"]], device=dev) if case["drafts"] else None
    drafted = torch.zeros(T, dtype=torch.int32, device=dev)
    step = max(1, (1 << 26) // V)
    for i in range(0, T, step):
        n = min(step, T - i)
        # peaked probabilities, and a draft model that mostly agrees
        a = 6.0 * torch.randn((n, V), generator=g, device=dev)
        p[i:i + n] = torch.softmax(a, -1).to(p.dtype)
        a += 0.7 * torch.randn((n, V), generator=g, device=dev)
        if q is not None:
            q[i:i + n] = torch.softmax(a, -1).to(q.dtype)
        # the draft model's own sample: the largest of its logits with Gumbel noise
        e = torch.rand((n, V), generator=g, device=dev).clamp_(1e-20, 1.0 - 2.0 ** -24)
        drafted[i:i + n] = a.sub_(e.log_().neg_().log_()).argmax(-1).to(torch.int32)
    s = {"case": case, "T": T, "p": p, "q": q}
    s["u"] = torch.rand(T, generator=g, device=dev)
    starts = [0]
    for n in rows:
        starts.append(starts[-1] + n)
    s["start"] = torch.tensor(starts, dtype=torch.int32).to(dev)
    # row t holds the token fed to the model there: the draft made from row t - 1
    s["tokens"] = torch.roll(drafted, 1).contiguous()
    if own:
        from few_row_quantized_amd import qgemv
        s["work"] = qgemv.verify_workspace(p, B)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if op == "attend":
        return _run_attend(state)
    if op == "append":
        return _run_append(state)
    return _run_verify(state)


def _run_attend(s):
    c = s["case"]
    if own:
        from few_row_quantized_amd import qgemv
        out = qgemv.attend(s["cache"], s["q"], s["start"], s["len"], c["M"], window=c["window"],
                           sinks=c["sinks"], scale=s["scale"], lse=s["lse"], workspace=s["work"])
        return {"out": out, "lse": s["lse"]}
    return _plain_attend(s)


def _run_append(s):
    if own:
        from few_row_quantized_amd import qgemv
        qgemv.append(s["cache"], s["new_k"], s["new_v"], s["start"], s["len"])
    else:
        _plain_append(s)
    return {"k": s["k"], "v": s["v"]}


def _run_verify(s):
    c = s["case"]
    if own:
        from few_row_quantized_amd import qgemv
        tokens, count = qgemv.verify(s["p"], s["q"], s["tokens"], s["u"], s["start"], c["M"],
                                     workspace=s["work"])
        return {"tokens": tokens, "count": count}
    return _plain_verify(s)


# ---------------------------------------------------------------- plain forms

def _row_places(s, dev):
    """For each row: its sequence, and its position in that sequence's cache."""
    t = torch.arange(s["T"], device=dev, dtype=torch.int64)
    start, length = s["start"].long(), s["len"].long()
    seq = torch.searchsorted(start[1:].contiguous(), t, right=True)
    return seq, length[seq] - (start[seq + 1] - t)


def _plain_append(s):
    k, v = s["k"], s["v"]
    page = s["case"]["page"]
    seq, pos = _row_places(s, k.device)
    slot = s["table"].long()[seq, pos // page]
    new_k, new_v = s["new_k"].float(), s["new_v"].float()
    if s["k_scale"] is not None:  # 8 bits: the values over the head's scale, at most 448 large
        new_k = (new_k / s["k_scale"][None, :, None]).clamp(-448.0, 448.0)
        new_v = (new_v / s["v_scale"][None, :, None]).clamp(-448.0, 448.0)
    k[slot, pos % page] = new_k.to(k.dtype)
    v[slot, pos % page] = new_v.to(v.dtype)


def _plain_attend(s):
    c = s["case"]
    B, M, H, G, D, page = (c[x] for x in ("B", "M", "H", "G", "D", "page"))
    dev = s["q"].device
    start, length = s["start"].long(), s["len"].long()
    table = s["table"].long().clamp(min=0)
    L = table.shape[1] * page
    rows = start[1:] - start[:-1]
    # the rows of each sequence, padded to M
    m = torch.arange(M, device=dev)
    real = m[None, :] < rows[:, None]
    t = (start[:-1, None] + m[None, :]).clamp(max=s["T"] - 1)
    q = s["q"][t].float().view(B, M, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, M * G, D)
    k = s["k"][table].float().view(B, L, H, D).permute(0, 2, 3, 1)
    score = torch.matmul(q, k).view(B, H, M, G, L)
    del k
    factor = s["scale"] if s["k_scale"] is None else (s["scale"] * s["k_scale"]).view(1, H, 1, 1, 1)
    score = score * factor
    # the keys that a row sees: up to its own, within the window or among the sinks
    j = torch.arange(L, device=dev)[None, None, :]
    pos = (length[:, None] - rows[:, None] + m[None, :])[:, :, None]
    sees = (j <= pos) & real[:, :, None]
    if c["window"]:
        sees &= (j > pos - c["window"]) | (j < c["sinks"])
    score = torch.where(sees[:, None, :, None, :], score, float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    score = torch.exp(score - top)
    total = score.sum(-1, keepdim=True)
    v = s["v"][table].float().view(B, L, H, D).permute(0, 2, 1, 3)
    # slots past the length may hold anything
    v = torch.where((j[0] < length[:, None])[:, None, :, None], v, 0.0)
    out = torch.matmul(score.view(B, H, M * G, L), v).view(B, H, M, G, D)
    del v
    out = torch.where(total > 0, out / total, 0.0)
    if s["v_scale"] is not None:
        out = out * s["v_scale"].view(1, H, 1, 1, 1)
    lse = (top + torch.log(total)).squeeze(-1)
    out = out.permute(0, 2, 1, 3, 4).reshape(B, M, H * G, D)[real]
    lse = lse.permute(0, 2, 1, 3).reshape(B, M, H * G)[real]
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _plain_verify(s):
    p, q, u = s["p"], s["q"], s["u"].double()
    T, V = p.shape
    B, M = s["case"]["B"], s["case"]["M"]
    start = s["start"].long()
    rows = start[1:] - start[:-1]
    m = torch.arange(M, device=p.device)
    t = (start[:-1, None] + m[None, :]).clamp(max=T - 1)
    # row t's draft is the token fed to row t + 1
    draft = s["tokens"].long()[(t + 1).clamp(max=T - 1)]
    pd = p[t, draft].double()
    qd = torch.ones_like(pd) if q is None else q[t, draft].double()
    checked = m[None, :] < rows[:, None] - 1
    accept = checked & (u[t] * qd < pd)
    n = accept.long().cumprod(-1).sum(-1)  # drafts accepted before the first refusal
    at = start[:-1] + n
    refused = n < rows - 1
    w = p[at].double()
    if q is None:
        drop = torch.zeros_like(w).scatter_(1, draft.gather(1, n[:, None]), 1.0)
        rest = torch.where(drop > 0, 0.0, w)
    else:
        rest = (w - q[at].double()).clamp(min=0.0)
    rest = torch.where(refused[:, None], rest, w)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, w)
    c = rest.cumsum(-1)
    # the last row's number draws the token: the first whose running sum passes its share
    share = u[start[1:] - 1] * c[:, -1]
    token = (c <= share[:, None]).sum(-1).clamp(max=V - 1)
    out = torch.where(m[None, :] < n[:, None], draft, -1)
    out = torch.where(m[None, :] == n[:, None], token[:, None], out)
    real = m[None, :] < rows[:, None]
    return {"tokens": out[real].to(torch.int32), "count": (n + 1).to(torch.int32)}


# ---------------------------------------------------------------- cost

def work(case):
    if case["op"] == "verify":
        r = random.Random(1000 * case["B"] + case["M"])
        T = sum(case["M"] if b % 3 != 2 else r.randint(1, case["M"]) for b in range(case["B"]))
        # one row of p and of q for each sequence: the row its last token is drawn from
        n = case["B"] * case["V"] * (2 if case["drafts"] else 1)
        return {"bytes": n * SIZE[case["p"]] + 24 * T, "flops": 3 * n}
    rows, lens = _layout(case)
    H, D, T = case["H"], case["D"], sum(rows)
    if case["op"] == "append":
        return {"bytes": 2 * T * H * D * (SIZE[case["new"]] + SIZE[case["cache"]]), "flops": 4 * T * H * D}
    slots = pairs = 0
    for r, n in zip(rows, lens):
        seen = 0
        for i in range(r):
            pos = n - r + i
            if pos >= 0:
                w = case["window"]
                first = max(0, pos - w + 1) if w else 0
                seen += pos + 1 - first + min(case["sinks"], first)
        pairs += seen
        low = max(0, n - r - case["window"] + 1) if case["window"] else 0
        slots += n - low + min(case["sinks"], low)
    Hq = H * case["G"]
    return {"bytes": 2 * slots * H * D * SIZE[case["cache"]] + 2 * T * Hq * D * SIZE[case["q"]] + 4 * T * Hq,
            "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "verify":
        return _exact_verify(s)
    return _exact_attend(s)


def _exact_attend(s):
    c = s["case"]
    H, G, D, page = (c[x] for x in ("H", "G", "D", "page"))
    starts, lens = s["start"].tolist(), s["len"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["q"].shape[:2], float("-inf"), dtype=torch.float64, device=s["q"].device)
    ks = torch.ones(H) if s["k_scale"] is None else s["k_scale"].cpu()
    vs = torch.ones(H) if s["v_scale"] is None else s["v_scale"].cpu()
    for b, n in enumerate(lens):
        if n == 0:
            continue
        token = torch.arange(n, device=s["q"].device)
        flat = s["table"][b].long()[token // page] * page + token % page
        for h in range(H):
            k = s["k"].view(-1, H, D)[flat, h].double() * float(ks[h])
            v = s["v"].view(-1, H, D)[flat, h].double() * float(vs[h])
            for t in range(starts[b], starts[b + 1]):
                last = n - (starts[b + 1] - t)
                if last < 0:
                    continue
                heads = slice(h * G, (h + 1) * G)
                keep = token[:last + 1]
                if c["window"]:
                    keep = keep[(keep > last - c["window"]) | (keep < c["sinks"])]
                a = (s["q"][t, heads].double() @ k[keep].T) * s["scale"]
                z = torch.logsumexp(a, -1)
                lse[t, heads] = z
                out[t, heads] = torch.exp(a - z[:, None]) @ v[keep]
    return {"out": out, "lse": lse}


def _exact_append(s):
    page = s["case"]["page"]
    k, v = s["k"].double(), s["v"].double()
    starts, lens = s["start"].tolist(), s["len"].tolist()
    table = s["table"].tolist()
    where = []
    for b, n in enumerate(lens):
        for t in range(starts[b], starts[b + 1]):
            pos = n - (starts[b + 1] - t)
            where.append(table[b][pos // page] * page + pos % page)
    where = torch.tensor(where, device=k.device)
    for pages, new, scale in ((k, s["new_k"], s["k_scale"]), (v, s["new_v"], s["v_scale"])):
        x = new.double()
        if scale is not None:
            x = (x / scale.double()[:, None]).clamp(-448.0, 448.0)
        pages.view(-1, *pages.shape[2:])[where] = x
    return {"k": k, "v": v}


def _exact_verify(s):
    import numpy as np
    starts, given = s["start"].tolist(), s["tokens"].tolist()
    u = s["u"].double().tolist()
    T, V = s["p"].shape
    tokens, count = np.full(T, -1, np.int64), []
    for a, e in zip(starts[:-1], starts[1:]):
        t = a
        while t < e - 1:
            pt = float(s["p"][t, given[t + 1]].double())
            qt = 1.0 if s["q"] is None else float(s["q"][t, given[t + 1]].double())
            if not u[t] * qt < pt:
                break
            tokens[t] = given[t + 1]
            t += 1
        p = s["p"][t].double().cpu().numpy()
        w = p
        if t < e - 1:
            if s["q"] is None:
                w = p.copy()
                w[given[t + 1]] = 0.0
            else:
                w = np.maximum(p - s["q"][t].double().cpu().numpy(), 0.0)
            if not w.sum() > 0:
                w = p
        c = np.cumsum(w)
        tokens[t] = min(int(np.searchsorted(c, u[e - 1] * c[-1], side="right")), V - 1)
        count.append(t - a + 1)
    dev = s["p"].device
    return {"tokens": torch.tensor(tokens, dtype=torch.int32, device=dev),
            "count": torch.tensor(count, dtype=torch.int32, device=dev)}
