"""The operators that keep a paged cache within a budget of tokens by the attention that its tokens receive, as cases to measure.

Four calls are measured:

  weights  the attention weight that every key receives from packed queries, into a pool of weights (``attn_weights_packed``)
  decode   one new query per sequence over pages, the weights that the tokens receive accumulated (``paged_attn_decode``)
  select   the tokens that each head keeps: the first, the latest, and those of the largest weights (``paged_kv_select``)
  compact  the kept rows moved to the front of their sequence's pages, in place (``paged_kv_compact``)

With ``own`` false, ``run`` computes them in plain torch operations; with ``own`` true it calls the library.

A weights pool is float32 [num_pages, Hkv, page_tokens], addressed like the pages of K and V: token t of sequence b and KV head h has its
sum at [table[b, t // page_tokens], h, t % page_tokens].  A token's weight is the sum of the probabilities that the queries of its KV
head's group give it.  A call sets the weights of the tokens that are new with it and adds to the others'.

An FP8 page holds, per KV head, ``page_tokens`` rows of D E4M3 codes and then one E8M0 scale byte per row:
value = code * 2^(byte - 127), the exponent being the smallest e with max|row| / 2^e <= 448 (0 for a row of zeros).
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
NEG = float("-inf")


# ---- the cases ----------------------------------------------------------------------------------


def listed():
    return [
        # two short prompts: latency
        dict(name="weights short", op="weights", B=2, T=128, past=0, Hq=16, Hkv=4, D=64, pt=16, add=False, dtype="bf16", mix=1),
        # a batch of prompts, every query counted
        dict(name="weights prompts", op="weights", B=8, T=16384, past=0, Hq=32, Hkv=8, D=128, pt=16, add=False, dtype="bf16", mix=2),
        # long contexts watched by their last 32 queries
        dict(name="weights window", op="weights", B=8, T=256, past=130816, Hq=32, Hkv=8, D=128, pt=32, add=True, dtype="f16", mix=3),
        # a single user's decode step: latency
        dict(name="decode one", op="decode", fmt="fp8", B=1, T=1500, Hq=32, Hkv=8, D=128, pt=16, dtype="bf16", mix=4),
        # a full server, contexts of 1,024 to 32,768 tokens
        dict(name="decode full", op="decode", fmt="fp8", B=64, T=1081344, Hq=32, Hkv=8, D=128, pt=16, dtype="f16", mix=5, even=True),
        # pages that are not quantised
        dict(name="decode plain pages", op="decode", fmt="rows", B=16, T=65536, Hq=16, Hkv=4, D=128, pt=16, dtype="bf16", mix=6),
        # one conversation that has outgrown its budget
        dict(name="select one", op="select", B=1, T=4096, Hkv=8, pt=16, budget=1024, sink=4, recent=256, mix=7),
        # every context of a full server cut to 2,048 tokens
        dict(name="select full", op="select", B=128, T=2162688, Hkv=8, pt=16, budget=2048, sink=4, recent=512, mix=8, even=True),
        # two long documents
        dict(name="select long", op="select", B=2, T=262144, Hkv=4, pt=32, budget=8192, sink=16, recent=1024, mix=9),
        # one conversation, quantised pages
        dict(name="compact one", op="compact", fmt="fp8", B=1, T=4096, Hkv=8, D=128, pt=16, budget=1024, dtype="bf16", mix=10),
        # a full server, each context some hundred tokens over its budget
        dict(name="compact full", op="compact", fmt="fp8", B=128, T=327680, Hkv=8, D=128, pt=16, budget=2048, dtype="bf16", mix=11),
        # long documents, pages that are not quantised
        dict(name="compact long", op="compact", fmt="rows", B=2, T=131072, Hkv=4, D=128, pt=32, budget=16384, dtype="f16", mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["weights", "decode", "select", "compact"])
    c = dict(op=op, mix=rng.randrange(1, 1 << 20), Hkv=rng.choice([1, 2, 3, 4, 8]), pt=rng.choice([16, 32, 64]))
    g = rng.choice([1, 2, 3, 4, 6, 8, 16])
    if op == "weights":
        B = rng.randint(1, 12)
        c.update(B=B, T=max(B, _log(rng, B, 12000)), past=rng.choice([0, 0, _log(rng, 1, 60000)]), Hq=c["Hkv"] * g,
                 D=rng.choice([64, 128]), add=rng.random() < 0.5, dtype=rng.choice(["bf16", "f16", "bf16", "f16", "f32"]))
        most = 2e10 if c["dtype"] == "f32" else 2e11
        while work(c)["flops"] > most or c["Hq"] * B * max(_lens(c)[0]) * max(_lens(c)[1]) > 3e9:
            c["T"], c["past"] = max(B, c["T"] * 2 // 3), c["past"] * 2 // 3
        return c
    if op == "decode":
        B = _log(rng, 1, 128)
        c.update(fmt=rng.choice(["fp8", "fp8", "rows"]), B=B, T=max(B, _log(rng, 4 * B, 200000)), Hq=c["Hkv"] * g, D=rng.choice([64, 128, 256]),
                 dtype=rng.choice(["bf16", "f16"]))
        return c
    if op == "select":
        B = _log(rng, 1, 128)
        T = _log(rng, 64 * B, 1000000)
        budget = _log(rng, 1, min(16384, T // B // 2))  # some contexts are longer
        sink = rng.randint(0, min(16, budget - 1))
        c.update(B=B, T=T, budget=budget, sink=sink, recent=rng.randint(0, budget - sink - 1))
        return c
    B = _log(rng, 1, 128)
    c.update(fmt=rng.choice(["fp8", "rows"]), B=B, T=max(B, _log(rng, 8 * B, 150000)), D=rng.choice([64, 128, 256]),
             budget=_log(rng, 1, 16384), dtype=rng.choice(["bf16", "f16"]))
    return c


def _split(total, parts, rng, most=None):
    """`parts` lengths of 1 or more (at most `most`) that add up to `total`."""
    w = [rng.uniform(0.06, 1.94) for _ in range(parts)]
    n = [max(1, int(total * x / sum(w))) for x in w]
    if most:
        n = [min(x, most) for x in n]
    i = 0
    while sum(n) != total:
        step = 1 if sum(n) < total else -1
        if (step > 0 and (not most or n[i % parts] < most)) or (step < 0 and n[i % parts] > 1):
            n[i % parts] += step
        i += 1
    return n


def _lens(case):
    """(new tokens, contexts) of the sequences of a case, by the case alone."""
    rng = random.Random(case["mix"])
    B, T = case["B"], case["T"]
    if case["op"] == "weights":
        new = [T // B] * B if T % B == 0 and case["past"] > 64 * T else _split(T, B, rng, max(4096, -(-T // B)))
        past = [0] * B if not case["past"] else [int(case["past"] * rng.uniform(0.2, 1.8) / B) for _ in range(B)]
        return new, [n + p for n, p in zip(new, past)]
    if case.get("even"):  # evenly over 1,024 tokens to twice the mean less that, in no order
        c = [1024 + (2 * (T // B) - 2048) * i // (B - 1) for i in range(B)]
        c[0] += T - sum(c)
        rng.shuffle(c)
    elif case["op"] == "compact":  # about as long as one another
        c = [T // B + rng.randint(0, T // B // 8) - T // B // 16 for _ in range(B)]
        c = [max(1, x) for x in c]
    else:
        c = _split(T, B, rng)
    return [1] * B, c


# ---- FP8 pages ---------------------------------------------------------------------------------------


def _quantise(x):
    """Rows [..., D] -> (E4M3 codes, E8M0 bytes [...])."""
    m, e = torch.frexp(x.abs().amax(-1))  # 448 = 0.875 * 2^9
    e = torch.where(m > 0, e - 9 + (m > 0.875).to(e.dtype), torch.zeros_like(e)).clamp(-127, 127)
    codes = torch.ldexp(x, -e.unsqueeze(-1)).to(torch.float32).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def _codes(pool, pt, D):
    return pool[..., : pt * D].unflatten(-1, (pt, D))


def _scales(pool, pt, D):
    return pool[..., pt * D:]


def _values(pool, pt, D):
    """The views that stand for a quantised pool's values: its E4M3 codes and its E8M0 scales."""
    return _codes(pool, pt, D).view(torch.float8_e4m3fn), _scales(pool, pt, D).view(torch.float8_e8m0fnu)


def _pool(case, pages, gen):
    """A pool of K or V as an earlier part of the text left it: rows mostly normal, of several sizes."""
    Hkv, pt, D = case["Hkv"], case["pt"], case["D"]
    fp8 = case["fmt"] == "fp8"
    pool = torch.empty((pages, Hkv, pt * (D + 1)) if fp8 else (pages, Hkv, pt, D), dtype=torch.uint8 if fp8 else DTYPES[case["dtype"]], device=DEV)
    step = max(1, (1 << 28) // (Hkv * pt * D))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn(n, Hkv, pt, D, generator=gen, device=DEV)
        x *= torch.exp2(torch.randint(-3, 3, (n, Hkv, pt, 1), generator=gen, device=DEV).float())
        if fp8:
            c, s = _quantise(x)
            _codes(pool[p:p + n], pt, D).copy_(c.view(torch.uint8))
            _scales(pool[p:p + n], pt, D).copy_(s)
        else:
            pool[p:p + n].copy_(x)
    return pool


def _table(ctx, pt, gen):
    """Pages dealt out in no order, and how many there are (a few more than are used)."""
    need = [-(-c // pt) for c in ctx]
    pages = sum(need) + 5
    host = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32).cpu()
    table = torch.full((len(ctx), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = host[at:at + n]
        at += n
    return table.to(DEV), pages


def _starts(lens):
    s = [0]
    for n in lens:
        s.append(s[-1] + n)
    return torch.tensor(s, dtype=torch.int32, device=DEV)


# ---- prepare -----------------------------------------------------------------------------------------


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed * 7919 + 13)
    op, Hkv, pt = case["op"], case["Hkv"], case["pt"]
    new, ctx = _lens(case)
    s = dict(case=case, op=op, ctx=torch.tensor(ctx, dtype=torch.int32, device=DEV), most=max(ctx))
    s["table"], pages = _table(ctx, pt, gen)
    # sums of probabilities: of very different sizes, some of them 0
    w = torch.exp(2.5 * torch.randn(pages, Hkv, pt, generator=gen, device=DEV) - 3.0)
    s["weights"] = torch.where(torch.rand(pages, Hkv, pt, generator=gen, device=DEV) < 0.05, 0.0, w)
    if op == "weights":
        dt, D = DTYPES[case["dtype"]], case["D"]
        Tq, Tk = sum(new), sum(ctx)
        # keys of one text have a part in common, so that some of them receive much
        k = torch.randn(Tk + 3, Hkv, D, generator=gen, device=DEV) * (0.5 + torch.rand(Tk + 3, 1, 1, generator=gen, device=DEV))
        s.update(q=torch.randn(Tq + 3, case["Hq"], D, generator=gen, device=DEV).to(dt), k=k.to(dt), q_start=_starts(new), k_start=_starts(ctx), most_q=max(new))
    if op in ("decode", "compact"):
        s.update(k_pool=_pool(case, pages, gen), v_pool=_pool(case, pages, gen))
        pools = (s["k_pool"], s["v_pool"])
        s["out"] = sum((_values(p, pt, case["D"]) for p in pools), ()) if case["fmt"] == "fp8" else pools
    if op == "decode":
        s["q"] = torch.randn(case["B"], case["Hq"], 1, case["D"], generator=gen, device=DEV).to(DTYPES[case["dtype"]])
    if op == "compact":
        # what a selection gives: some of the tokens, in order, -1 behind them
        x = torch.rand(case["B"], Hkv, s["most"], generator=gen, device=DEV)
        x[..., :4] += 2.0
        n = s["ctx"].view(-1, 1, 1)
        x = torch.where(torch.arange(s["most"], device=DEV) < n, x, -1.0)
        width = min(case["budget"], s["most"])
        top = x.topk(width, -1).indices
        top = torch.where(torch.arange(width, device=DEV) < n, top, s["most"]).sort(-1).values
        keep = torch.full((case["B"], Hkv, case["budget"]), -1, dtype=torch.int32, device=DEV)
        keep[..., :width] = torch.where(top < s["most"], top, -1).to(torch.int32)
        s["keep"] = keep
    if own:
        import sparse_top_kv_validate_gb300 as sa
        s["sa"] = sa
    return s


# ---- run ---------------------------------------------------------------------------------------------


def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_weights(s):
    s["sa"].attn_weights_packed(s["q"], s["k"], s["weights"], s["table"], s["q_start"], s["k_start"], accumulate=s["case"]["add"])
    return s["weights"]


def _own_decode(s):
    return s["sa"].paged_attn_decode(s["q"], s["k_pool"], s["v_pool"], s["table"], s["ctx"], weights=s["weights"]), s["weights"]


def _own_select(s):
    c = s["case"]
    return s["sa"].paged_kv_select(s["weights"], s["table"], s["ctx"], c["budget"], sink=c["sink"], recent=c["recent"])


def _own_compact(s):
    s["sa"].paged_kv_compact(s["k_pool"], s["v_pool"], s["table"], s["ctx"], s["keep"], weights=s["weights"])
    return s["out"] + (s["weights"],)


_own = dict(weights=_own_weights, decode=_own_decode, select=_own_select, compact=_own_compact)


def _places(s):
    """(which tokens of [B, most] there are, their pages, their slots)."""
    t = torch.arange(s["most"], device=DEV)
    there = t < s["ctx"].unsqueeze(1)
    return there, torch.where(there, s["table"].long()[:, t // s["case"]["pt"]], 0), (t % s["case"]["pt"]).expand(there.shape)


def _put(s, w, old_from):
    """Weights w [B, Hkv, most] set, or added where old_from [B, most] says so."""
    there, page, slot = _places(s)
    at = (page[there], slice(None), slot[there])
    w = w.transpose(1, 2)[there]
    s["weights"][at] = torch.where(old_from[there].unsqueeze(-1), s["weights"][at] + w, w)


def _softmax(x, seen):
    x = x.masked_fill(~seen, NEG)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top > NEG, top, 0.0))
    total = x.sum(-1, keepdim=True)
    return x / torch.where(total > 0, total, 1.0)


def _plain_weights(s):
    c = s["case"]
    B, Hkv, D, g = c["B"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    qs, ks = s["q_start"].long(), s["k_start"].long()
    nq, nk = qs[1:] - qs[:-1], ks[1:] - ks[:-1]
    i, j = torch.arange(s["most_q"], device=DEV), torch.arange(s["most"], device=DEV)
    in_q, in_k = i < nq[:, None], j < nk[:, None]
    rq, rk = torch.where(in_q, qs[:-1, None] + i, 0), torch.where(in_k, ks[:-1, None] + j, 0)
    q = s["q"][rq].float().view(B, -1, Hkv, g, D) / math.sqrt(D)
    x = torch.einsum("bihgd,bjhd->bhgij", q, s["k"][rk].float())
    past = (nk - nq)[:, None]
    seen = in_k[:, None, :] & in_q[:, :, None] & (j <= (i + past)[:, :, None])
    w = _softmax(x, seen[:, None, None]).sum((2, 3))
    _put(s, w, (j < past) & c["add"])
    return s["weights"]


def _rows(s, pool, page, slot):
    """Rows [B, most, Hkv, D] of a pool, 32 bits."""
    c = s["case"]
    if c["fmt"] != "fp8":
        return pool[page, :, slot].float()
    x = _codes(pool, c["pt"], c["D"])[page, :, slot].view(torch.float8_e4m3fn).float()
    return torch.ldexp(x, _scales(pool, c["pt"], c["D"])[page, :, slot].to(torch.int32).unsqueeze(-1) - 127)


def _plain_decode(s):
    c = s["case"]
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    there, page, slot = _places(s)
    q = s["q"].float().view(B, Hkv, c["Hq"] // Hkv, D) / math.sqrt(D)
    p = _softmax(torch.einsum("bhgd,bthd->bhgt", q, _rows(s, s["k_pool"], page, slot)), there[:, None, None])
    v = _rows(s, s["v_pool"], page, slot)
    y = torch.einsum("bhgt,bthd->bhgd", p, v).reshape(B, c["Hq"], 1, D).to(s["q"].dtype)
    _put(s, p.sum(2), torch.arange(s["most"], device=DEV) < s["ctx"].unsqueeze(1) - 1)
    return y, s["weights"]


def _plain_select(s):
    c = s["case"]
    there, page, slot = _places(s)
    n, t = s["ctx"].long().unsqueeze(1), torch.arange(s["most"], device=DEV)
    w = s["weights"][page, :, slot].transpose(1, 2)  # [B, Hkv, most]
    always = (t < c["sink"]) | (t >= n - c["recent"])
    w = torch.where((always & there)[:, None], float("inf"), torch.where(there[:, None], w, -1.0))
    width = min(c["budget"], s["most"])
    top = w.sort(dim=-1, descending=True, stable=True).indices[..., :width]
    top = torch.where(torch.arange(width, device=DEV) < n[:, None], top, s["most"]).sort(-1).values
    keep = torch.full((c["B"], c["Hkv"], c["budget"]), -1, dtype=torch.int32, device=DEV)
    keep[..., :width] = torch.where(top < s["most"], top, -1).to(torch.int32)
    return keep, s["ctx"].clamp(max=c["budget"])


def _plain_compact(s):
    c = s["case"]
    _, page, slot = _places(s)
    b = torch.arange(c["B"], device=DEV).view(-1, 1, 1)
    h = torch.arange(c["Hkv"], device=DEV).view(1, -1, 1)
    i = torch.arange(c["budget"], device=DEV)
    kept = s["keep"] >= 0
    b, h, i = (x.expand(kept.shape)[kept] for x in (b, h, i))
    j = s["keep"][kept].long()
    src, dst = (page[b, j], h, slot[b, j]), (page[b, i], h, slot[b, i])
    planes = [s["weights"]]
    for p in (s["k_pool"], s["v_pool"]):
        planes += [_codes(p, c["pt"], c["D"]), _scales(p, c["pt"], c["D"])] if c["fmt"] == "fp8" else [p]
    for p in planes:
        p[dst] = p[src]
    return s["out"] + (s["weights"],)


_plain = dict(weights=_plain_weights, decode=_plain_decode, select=_plain_select, compact=_plain_compact)


# ---- work ----------------------------------------------------------------------------------------------


def work(case):
    op, Hkv = case["op"], case["Hkv"]
    new, ctx = _lens(case)
    if op == "select":
        return dict(bytes=4 * Hkv * (sum(ctx) + case["B"] * case["budget"]), flops=Hkv * sum(ctx))
    D, es = case["D"], DTYPES[case["dtype"]].itemsize
    if op == "weights":
        pairs = sum(n * (c - n) + n * (n + 1) // 2 for n, c in zip(new, ctx))
        # the sums that are added to are read as well
        old = sum(c - n for n, c in zip(new, ctx)) if case["add"] else 0
        return dict(bytes=(sum(new) * case["Hq"] + sum(ctx) * Hkv) * D * es + 4 * Hkv * (sum(ctx) + old), flops=2 * case["Hq"] * D * pairs)
    row = D + 1 if case["fmt"] == "fp8" else D * es
    if op == "decode":
        return dict(bytes=sum(ctx) * Hkv * (2 * row + 8) + 2 * case["B"] * case["Hq"] * D * es, flops=4 * case["Hq"] * D * sum(ctx))
    kept = sum(min(c, case["budget"]) for c in ctx)
    moved = sum(min(c, case["budget"]) for c in ctx if c > case["budget"])
    return dict(bytes=Hkv * (moved * 2 * (2 * row + 4) + 4 * kept), flops=0)


# ---- exact ---------------------------------------------------------------------------------------------
# From the definitions in 64 bits, one sequence at a time.


def _exact_rows(case, pool, pages, n):
    """The first n rows [Hkv, n, D] of a sequence."""
    x, D = pool[pages], case["D"]
    if case["fmt"] == "fp8":
        codes = x[..., : case["pt"] * D].reshape(-1, case["Hkv"], case["pt"], D).view(torch.float8_e4m3fn).double()
        x = codes * torch.exp2(x[..., case["pt"] * D:].double() - 127)[..., None]
    return x.double().transpose(0, 1).reshape(case["Hkv"], -1, D)[:, :n]


def _exact_add(case, weights, pages, w, fresh):
    """w [Hkv, n] onto a sequence's weights, the last `fresh` of them anew."""
    n, pt = w.shape[1], case["pt"]
    for h in range(case["Hkv"]):
        old = weights[pages, h].reshape(-1)[:n].clone()
        old[n - fresh:] = 0
        line = weights[pages, h].reshape(-1)
        line[:n] = old + w[h]
        weights[pages, h] = line.view(-1, pt)


def exact(case, seed):
    s = prepare(case, seed)
    op, pt = case["op"], case["pt"]
    new, ctx = _lens(case)
    out = s["weights"].double()
    pages = [s["table"][b, : -(-n // pt)].long() for b, n in enumerate(ctx)]
    if op == "weights":
        qa, ka, g = 0, 0, case["Hq"] // case["Hkv"]
        for b, (n, c) in enumerate(zip(new, ctx)):
            w = torch.zeros(case["Hkv"], c, dtype=torch.float64, device=DEV)
            hide = torch.arange(c, device=DEV)[None] > torch.arange(n, device=DEV)[:, None] + (c - n)
            for h in range(case["Hq"]):
                x = s["q"][qa:qa + n, h].double() @ s["k"][ka:ka + c, h // g].double().T / math.sqrt(case["D"])
                w[h // g] += torch.softmax(x.masked_fill(hide, NEG), -1).sum(0)
            _exact_add(case, out, pages[b], w, n if case["add"] else c)
            qa, ka = qa + n, ka + c
        return out
    if op == "decode":
        ys = []
        for b, n in enumerate(ctx):
            q = s["q"][b].double().view(case["Hkv"], -1, case["D"])
            k, v = (_exact_rows(case, p, pages[b], n) for p in (s["k_pool"], s["v_pool"]))
            p = torch.softmax(q @ k.transpose(1, 2) / math.sqrt(case["D"]), -1)
            ys.append((p @ v).reshape(1, case["Hq"], 1, case["D"]))
            _exact_add(case, out, pages[b], p.sum(1), 1)
        return torch.cat(ys), out
    if op == "select":
        return None  # whole numbers
    outs = [x.double() for x in s["out"]] + [out]
    for b, n in enumerate(ctx):
        for h in range(case["Hkv"]):
            keep = s["keep"][b, h].long()
            keep = keep[keep >= 0]
            to = torch.arange(len(keep), device=DEV)
            for x in outs:
                line = x[pages[b], h].flatten(0, 1)
                line[to] = line[keep]
                x[pages[b], h] = line.view(len(pages[b]), pt, *line.shape[1:])
    return tuple(outs)
