"""The serving operators of this library around a paged cache, as cases to measure.

Five calls of one serving step are measured:

  rotary   rotary positions of queries and keys (``rotary_embed``)
  write    new tokens' K and V rotated, quantised to FP8 and put into their pages (``paged_kv_write``)
  read     a context read back from FP8 pages into packed rows (``paged_kv_read``)
  attend   one new query per sequence over FP8 pages (``paged_attn_decode``)
  prefill  packed sequences of different lengths, causal, grouped heads (``attn_prefill_packed``)

With ``own`` false, ``run`` computes them in plain torch operations; with ``own`` true it calls the library.

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
        # one decode step of 128 sequences: the queries and keys of the new tokens
        dict(name="rope step", op="rotary", layout="packed", B=1, S=128, Hq=32, Hk=8, D=128, rot=128, inter=False,
             scaling="none", factor=1.0, dtype="bf16", far=32768),
        # four prompts of a long-context model, head-major, half of each head rotated, far positions
        dict(name="rope prompts", op="rotary", layout="heads", B=4, S=4096, Hq=32, Hk=8, D=128, rot=64, inter=True,
             scaling="ramp", factor=16.0, dtype="f16", far=1 << 20),
        # the same decode step's cache write
        dict(name="write step", op="write", B=128, new="ones", T=128, Hkv=8, D=128, pt=16, rope=True, inter=False,
             far=32768, dtype="bf16", mix=1),
        # the prompts of a batch, written as they are prefilled
        dict(name="write prompts", op="write", B=8, new="ragged", T=16384, Hkv=8, D=128, pt=16, rope=True, inter=True,
             far=4096, dtype="f16", mix=2),
        # contexts fetched for a chunk's prefill
        dict(name="read contexts", op="read", B=16, T=65536, Hkv=8, D=128, pt=16, dtype="bf16", mix=3),
        # the same for three short chats
        dict(name="read short", op="read", B=3, T=1101, Hkv=4, D=64, pt=16, dtype="f16", mix=4),
        # a single user: latency
        dict(name="attend one", op="attend", B=1, T=1500, Hq=32, Hkv=8, D=128, pt=16, dtype="bf16", mix=5),
        # a full server: contexts of 1,024 to 32,768 tokens
        dict(name="attend full", op="attend", B=128, T=2162688, Hq=32, Hkv=8, D=128, pt=16, dtype="f16", mix=6, even=True),
        # one very long document among short chats
        dict(name="attend uneven", op="attend", B=24, T=140000, Hq=64, Hkv=8, D=128, pt=32, dtype="bf16", mix=7, long=131072),
        # two short prompts
        dict(name="prefill short", op="prefill", B=2, T=128, Hq=16, Hkv=4, D=64, causal=True, cap=0.0, past=0, dtype="bf16", mix=8),
        # a batch of prompts
        dict(name="prefill prompts", op="prefill", B=8, T=16384, Hq=32, Hkv=8, D=128, causal=True, cap=0.0, past=0, dtype="bf16", mix=9),
        # chunks of prompts over the contexts before them, with a softcap
        dict(name="prefill chunks", op="prefill", B=6, T=2750, Hq=32, Hkv=8, D=128, causal=True, cap=50.0, past=24000, dtype="f16", mix=10),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "write", "read", "attend", "prefill"])
    mix = rng.randrange(1, 1 << 20)
    Hkv = rng.choice([1, 2, 3, 4, 8])
    g = rng.choice([1, 2, 3, 4, 6, 8, 16])
    if op == "rotary":
        D = rng.choice([64, 80, 96, 128, 256])
        rot = rng.choice([D, D // 2])
        B = rng.randint(1, 6)
        S = _log(rng, 1, 16384 // B)
        return dict(op=op, layout=rng.choice(["packed", "heads"]), B=B, S=S, Hq=Hkv * min(g, 64 // Hkv, 8), Hk=Hkv, D=D, rot=rot,
                    inter=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ntk", "ramp"]), factor=rng.choice([2.0, 4.0, 16.0]),
                    dtype=rng.choice(["bf16", "f16", "f32"]), far=_log(rng, 1 << 10, 1 << 20))
    D, pt = rng.choice([64, 128, 256]), rng.choice([16, 32, 64])
    if op == "write":
        B = _log(rng, 1, 256)
        T = B if rng.random() < 0.4 else max(B, _log(rng, B, 8192))
        return dict(op=op, B=B, new="ones" if T == B else "ragged", T=T, Hkv=Hkv, D=D, pt=pt, rope=rng.random() < 0.6,
                    inter=rng.random() < 0.5, far=_log(rng, 64, 32768), dtype=rng.choice(["bf16", "f16", "f32"]), mix=mix)
    if op == "read":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, T=max(B, _log(rng, B, 32768)), Hkv=Hkv, D=D, pt=pt, dtype=rng.choice(["bf16", "f16", "f32"]), mix=mix)
    if op == "attend":
        B = _log(rng, 1, 200)
        c = dict(op=op, B=B, T=max(B, _log(rng, 4 * B, 400000)), Hq=Hkv * g, Hkv=Hkv, D=D, pt=pt, dtype=rng.choice(["bf16", "f16"]), mix=mix)
        if rng.random() < 0.2:
            c["T"] = max(c["T"], 2 * B + 64)
            c["long"] = c["T"] // 2
        return c
    B = rng.randint(1, 12)
    c = dict(op=op, B=B, T=max(B, _log(rng, B, 12000)), Hq=Hkv * g, Hkv=Hkv, D=rng.choice([64, 128]), causal=rng.random() < 0.8,
             cap=rng.choice([0.0, 0.0, 30.0, 50.0]), past=rng.choice([0, 0, _log(rng, 1, 12000)]), dtype=rng.choice(["bf16", "f16"]), mix=mix)
    while work(c)["flops"] > 3e11 or c["Hq"] * c["B"] * max(_lens(c)[0]) * max(_lens(c)[1]) > 3e9:
        c["T"], c["past"] = max(B, c["T"] * 2 // 3), c["past"] * 2 // 3
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
    if case["op"] == "write":
        new = [1] * B if case["new"] == "ones" else _split(T, B, rng, max(4096, -(-T // B)))
        return new, [n + rng.randrange(0, case["far"]) for n in new]
    if case["op"] == "read":
        n = _split(T, B, rng)
        return n, n
    if case["op"] == "attend":
        if case.get("long"):
            c = [case["long"]] + (_split(T - case["long"], B - 1, rng) if B > 1 else [])
            c[-1] += T - sum(c)
            return [1] * B, c
        if case.get("even"):  # evenly over 1,024 tokens to twice the mean less that, in no order
            c = [1024 + (2 * (T // B) - 2048) * i // (B - 1) for i in range(B)]
            c[0] += T - sum(c)
            rng.shuffle(c)
            return [1] * B, c
        return [1] * B, _split(T, B, rng)
    new = _split(T, B, rng, max(4096, -(-T // B)))
    past = [0] * B if not case["past"] else [int(case["past"] * rng.uniform(0.2, 1.8) / B) for _ in range(B)]
    return new, [n + p for n, p in zip(new, past)]


# ---- rotary angles ---------------------------------------------------------------------------------


def _rope_spec(case):
    if case["op"] == "write":
        return dict(rotary_dim=case["D"], interleaved=case["inter"])
    return dict(rotary_dim=case["rot"], interleaved=case["inter"], scaling=case["scaling"], factor=case["factor"],
                original_len=4096, ramp=(1.0, 32.0), mscale=0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "ramp" else 1.0)


def _inv_freq(rotary_dim, interleaved=False, scaling="none", factor=1.0, original_len=0, ramp=(1.0, 32.0), mscale=1.0):
    """The pairs' angles per position, 64 bits."""
    i = torch.arange(rotary_dim // 2, dtype=torch.float64, device=DEV)
    base = 10000.0
    if scaling == "ntk":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = base ** (-2.0 * i / rotary_dim)
    if scaling == "linear":
        f = f / factor
    if scaling == "ramp":
        turns = original_len * f / (2 * math.pi)
        keep = ((turns - ramp[0]) / (ramp[1] - ramp[0])).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f


def _rotate(x, positions, spec, dtype):
    """x [..., D] in `dtype` rotated at `positions` [...]: angles in 64 bits."""
    rot = spec["rotary_dim"]
    a = positions.double().unsqueeze(-1) * _inv_freq(**spec)
    m = spec.get("mscale", 1.0)
    cos, sin = (a.cos() * m).to(dtype), (a.sin() * m).to(dtype)
    h = rot // 2
    if spec["interleaved"]:
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((u * cos - v * sin, u * sin + v * cos), -1).flatten(-2)
    else:
        u, v = x[..., :h], x[..., h:rot]
        y = torch.cat((u * cos - v * sin, u * sin + v * cos), -1)
    return torch.cat((y, x[..., rot:]), -1)


# ---- FP8 pages ---------------------------------------------------------------------------------------


def _quantise(x):
    """Rows [..., D] (32 or 64 bits) -> (E4M3 codes, E8M0 bytes [...])."""
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)  # amax = m 2^e with m in [0.5, 1): 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), torch.zeros_like(e)).clamp(-127, 127)
    codes = torch.ldexp(x, -e.unsqueeze(-1)).to(torch.float32).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def _codes(pool, pt, D):
    return pool[..., : pt * D].unflatten(-1, (pt, D))


def _scales(pool, pt, D):
    return pool[..., pt * D:]


def _values(pool, pt, D):
    """The views that stand for a pool's values: its E4M3 codes and its E8M0 scales."""
    return _codes(pool, pt, D).view(torch.float8_e4m3fn), _scales(pool, pt, D).view(torch.float8_e8m0fnu)


def _pool(pages, Hkv, pt, D, gen):
    """A pool filled with the quantised rows of an earlier part of the text: mostly normal, of several sizes."""
    pool = torch.empty(pages, Hkv, pt * (D + 1), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 28) // (Hkv * pt * D))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn(n, Hkv, pt, D, generator=gen, device=DEV)
        x *= torch.exp2(torch.randint(-3, 3, (n, Hkv, pt, 1), generator=gen, device=DEV).float())
        c, s = _quantise(x)
        _codes(pool[p:p + n], pt, D).copy_(c.view(torch.uint8))
        _scales(pool[p:p + n], pt, D).copy_(s)
    return pool


def _table(ctx, pt, gen):
    """Pages dealt out in no order, and how many there are (a few more than are used)."""
    need = [-(-c // pt) for c in ctx]
    pages = sum(need) + 5
    perm = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(ctx), max(need)), -1, dtype=torch.int32)
    at = 0
    host = perm.cpu()
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
    gen = torch.Generator(device=DEV).manual_seed(seed * 7919 + 11)
    op, D = case["op"], case["D"]
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=DEV).to(dt)

    s = dict(case=case, op=op)
    if op == "rotary":
        B, S = case["B"], case["S"]
        first = torch.randint(0, case["far"], (B, 1), generator=gen, device=DEV)
        pos = first + torch.arange(S, device=DEV)
        if case["layout"] == "packed":  # views into one projection's output
            qkv = randn(B * S, case["Hq"] + 2 * case["Hk"], D)
            s.update(q=qkv[:, : case["Hq"]], k=qkv[:, case["Hq"]: case["Hq"] + case["Hk"]], positions=pos.reshape(-1))
        else:
            s.update(q=randn(B, case["Hq"], S, D), k=randn(B, case["Hk"], S, D), positions=pos.to(torch.int32))
        s["spec"] = _rope_spec(case)
    else:
        new, ctx = _lens(case)
        Hkv = case["Hkv"]
        s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        s["start"] = _starts(new)
    if op == "write":
        # only the pages that the new tokens touch are in this pool
        pt, T = case["pt"], case["T"]
        table = torch.full((case["B"], -(-max(ctx) // pt)), -1, dtype=torch.int32)
        first = [(c - n) // pt for c, n in zip(ctx, new)]
        count = [-(-c // pt) - f for c, f in zip(ctx, first)]
        pages = sum(count) + 3
        perm = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32).cpu()
        at = 0
        for b in range(case["B"]):
            table[b, first[b]:first[b] + count[b]] = perm[at:at + count[b]]
            at += count[b]
        s.update(k=randn(T, Hkv, D), v=randn(T, Hkv, D), table=table.to(DEV), spec=_rope_spec(case) if case["rope"] else None,
                 k_pool=_pool(pages, Hkv, pt, D, gen), v_pool=_pool(pages, Hkv, pt, D, gen))
        s["out"] = _values(s["k_pool"], pt, D) + _values(s["v_pool"], pt, D)
    if op in ("read", "attend"):
        s["table"], pages = _table(ctx, case["pt"], gen)
        s.update(k_pool=_pool(pages, Hkv, case["pt"], D, gen), v_pool=_pool(pages, Hkv, case["pt"], D, gen), most=max(ctx))
        if op == "attend":
            s["q"] = randn(case["B"], case["Hq"], 1, D)
        else:
            s.update(k_out=torch.zeros(case["T"], Hkv, D, dtype=dt, device=DEV), v_out=torch.zeros(case["T"], Hkv, D, dtype=dt, device=DEV))
    if op == "prefill":
        Tq, Tk = sum(new), sum(ctx)
        s.update(q=randn(Tq + 3, case["Hq"], D), k=randn(Tk + 3, Hkv, D), v=randn(Tk + 3, Hkv, D), k_start=_starts(ctx),
                 y=torch.zeros(Tq + 3, case["Hq"], D, dtype=dt, device=DEV), most_q=max(new), most_k=max(ctx))
    if own:
        import sparse_top_kv_validate_gb300 as sa
        s["sa"] = sa
        if s.get("spec"):  # a program makes its table of angles once
            s["rope"] = sa.rope_table(**s["spec"])
    return s


# ---- run ---------------------------------------------------------------------------------------------


def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_rotary(s):
    return s["sa"].rotary_embed(s["q"], s["k"], s["positions"], s["rope"])


def _own_write(s):
    s["sa"].paged_kv_write(s["k"], s["v"], s["k_pool"], s["v_pool"], s["table"], s["ctx"], s["start"], rope=s.get("rope"))
    return s["out"]


def _own_read(s):
    return s["sa"].paged_kv_read(s["k_pool"], s["v_pool"], s["table"], s["ctx"], s["start"], s["k_out"], s["v_out"])


def _own_attend(s):
    return s["sa"].paged_attn_decode(s["q"], s["k_pool"], s["v_pool"], s["table"], s["ctx"])


def _own_prefill(s):
    c = s["case"]
    return s["sa"].attn_prefill_packed(s["q"], s["k"], s["v"], s["start"], s["k_start"], causal=c["causal"], softcap=c["cap"], y=s["y"])


_own = dict(rotary=_own_rotary, write=_own_write, read=_own_read, attend=_own_attend, prefill=_own_prefill)


def _plain_rotary(s):
    pos = s["positions"]
    at = pos.unsqueeze(1) if pos.dim() == 2 else pos.unsqueeze(-1)  # the same for every head
    return tuple(_rotate(x.float(), at, s["spec"], torch.float32).to(x.dtype) for x in (s["q"], s["k"]))


def _token_places(s, T):
    """(sequence, position) of the packed rows."""
    r = torch.arange(T, device=DEV)
    b = torch.searchsorted(s["start"].long(), r, right=True) - 1
    return b, s["ctx"].long()[b] - (s["start"].long()[b + 1] - r)


def _plain_write(s):
    c = s["case"]
    b, pos = _token_places(s, c["T"])
    page = s["table"].long()[b, pos // c["pt"]]
    k, v = s["k"].float(), s["v"].float()
    if s["spec"]:
        k = _rotate(k, pos.unsqueeze(-1), s["spec"], torch.float32)
    for x, pool in ((k, s["k_pool"]), (v, s["v_pool"])):
        codes, scales = _quantise(x)
        _codes(pool, c["pt"], c["D"])[page, :, pos % c["pt"]] = codes.view(torch.uint8)
        _scales(pool, c["pt"], c["D"])[page, :, pos % c["pt"]] = scales
    return s["out"]


def _dequantised(pool, page, slot, pt, D, dtype=torch.float32):
    """Rows of a pool at (page, slot) [...] -> [..., Hkv, D]."""
    x = _codes(pool, pt, D)[page, :, slot].view(torch.float8_e4m3fn).to(dtype)
    return torch.ldexp(x, _scales(pool, pt, D)[page, :, slot].to(torch.int32).unsqueeze(-1) - 127)


def _plain_read(s):
    c = s["case"]
    r = torch.arange(c["T"], device=DEV)
    b = torch.searchsorted(s["start"].long(), r, right=True) - 1
    pos = r - s["start"].long()[b]
    page = s["table"].long()[b, pos // c["pt"]]
    for pool, out in ((s["k_pool"], s["k_out"]), (s["v_pool"], s["v_out"])):
        out.copy_(_dequantised(pool, page, pos % c["pt"], c["pt"], c["D"]))
    return s["k_out"], s["v_out"]


def _plain_attend(s):
    c = s["case"]
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    t = torch.arange(s["most"], device=DEV)
    seen = t < s["ctx"].unsqueeze(1)
    page = torch.where(seen, s["table"].long()[:, t // c["pt"]], 0)
    q = s["q"].float().view(B, Hkv, c["Hq"] // Hkv, D) / math.sqrt(D)
    k = _dequantised(s["k_pool"], page, t % c["pt"], c["pt"], D)
    x = torch.einsum("bhgd,bthd->bhgt", q, k)
    x = x.masked_fill(~seen[:, None, None], NEG)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    k = _dequantised(s["v_pool"], page, t % c["pt"], c["pt"], D)
    return torch.einsum("bhgt,bthd->bhgd", p, k).reshape(B, c["Hq"], 1, D).to(s["q"].dtype)


def _plain_prefill(s):
    c = s["case"]
    B, Hkv, D, g = c["B"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    qs, ks = s["start"].long(), s["k_start"].long()
    nq, nk = qs[1:] - qs[:-1], ks[1:] - ks[:-1]
    i, j = torch.arange(s["most_q"], device=DEV), torch.arange(s["most_k"], device=DEV)
    in_q, in_k = i < nq[:, None], j < nk[:, None]
    rq, rk = torch.where(in_q, qs[:-1, None] + i, 0), torch.where(in_k, ks[:-1, None] + j, 0)
    q = s["q"][rq].float().view(B, -1, Hkv, g, D) / math.sqrt(D)
    x = torch.einsum("bihgd,bjhd->bhgij", q, s["k"][rk].float())
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    seen = in_k[:, None, :]
    if c["causal"]:
        seen = seen & (j <= i[:, None] + (nk - nq)[:, None, None])
    x = x.masked_fill(~seen[:, None, None], NEG)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top > NEG, top, 0.0))
    total = x.sum(-1, keepdim=True)
    x = x / torch.where(total > 0, total, 1.0)
    y = torch.einsum("bhgij,bjhd->bihgd", x, s["v"][rk].float()).reshape(B, -1, c["Hq"], D)
    s["y"][rq[in_q]] = y[in_q].to(s["y"].dtype)
    return s["y"]


_plain = dict(rotary=_plain_rotary, write=_plain_write, read=_plain_read, attend=_plain_attend, prefill=_plain_prefill)


# ---- work ----------------------------------------------------------------------------------------------


def work(case):
    es = DTYPES[case["dtype"]].itemsize
    op, D = case["op"], case["D"]
    if op == "rotary":
        n = case["B"] * case["S"]
        return dict(bytes=2 * n * (case["Hq"] + case["Hk"]) * D * es + 8 * n, flops=3 * n * (case["Hq"] + case["Hk"]) * case["rot"])
    new, ctx = _lens(case)
    row = 2 * case["Hkv"]  # K and V rows of a token
    if op == "write":
        return dict(bytes=sum(new) * row * (D * es + D + 1), flops=sum(new) * row * D * 3)
    if op == "read":
        return dict(bytes=sum(new) * row * (D * es + D + 1), flops=sum(new) * row * D)
    if op == "attend":
        return dict(bytes=sum(ctx) * row * (D + 1) + 2 * case["B"] * case["Hq"] * D * es, flops=4 * case["Hq"] * D * sum(ctx))
    if case["causal"]:
        pairs = sum(n * (c - n) + n * (n + 1) // 2 for n, c in zip(new, ctx))
    else:
        pairs = sum(n * c for n, c in zip(new, ctx))
    return dict(bytes=(2 * sum(new) * case["Hq"] + sum(ctx) * row) * D * es, flops=4 * case["Hq"] * D * pairs)


# ---- exact ---------------------------------------------------------------------------------------------
# From the definitions in 64 bits, one sequence at a time.


def _exact_rotate(x, positions, spec):
    rot = spec["rotary_dim"]
    f = _inv_freq(**spec)
    m = spec.get("mscale", 1.0)
    y = x.double().clone()
    for i in range(rot // 2):
        a = positions.double() * f[i]
        lo, hi = (2 * i, 2 * i + 1) if spec["interleaved"] else (i, i + rot // 2)
        c, s_ = m * torch.cos(a), m * torch.sin(a)
        u, v = x[..., lo].double(), x[..., hi].double()
        y[..., lo], y[..., hi] = u * c - v * s_, u * s_ + v * c
    return y


def _exact_quantise(x):
    """[n, H, D] 64 bits -> (values of the codes, exponents), by nearest even on E4M3's grid."""
    amax = x.abs().amax(-1)
    e = torch.where(amax > 0, torch.ceil(torch.log2(amax.clamp_min(1e-300) / 448)), 0.0)
    e = torch.where((amax > 0) & (amax > 448 * torch.exp2(e)), e + 1, e)
    e = torch.where((amax > 0) & (amax <= 448 * torch.exp2(e - 1)), e - 1, e).clamp(-127, 127)
    y = x / torch.exp2(e)[..., None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(y / step) * step, e  # torch.round goes to even


def exact(case, seed):
    s = prepare(case, seed)
    op, D = case["op"], case["D"]
    if op == "rotary":
        pos = s["positions"]
        pos = pos[:, None, :] if pos.dim() == 2 else pos[:, None]
        return _exact_rotate(s["q"], pos, s["spec"]), _exact_rotate(s["k"], pos, s["spec"])
    new, ctx = _lens(case)
    if op == "write":
        out = [x.double() for x in s["out"]]
        table = s["table"].cpu()
        at = 0
        pages, slots, places = [], [], []
        for b, n in enumerate(new):
            p = torch.arange(ctx[b] - n, ctx[b])
            pages.append(table[b].long()[p // case["pt"]])
            slots.append(p % case["pt"])
            places.append(p)
            at += n
        pages, slots, places = (torch.cat(x).to(DEV) for x in (pages, slots, places))
        k = _exact_rotate(s["k"], places[:, None], s["spec"]) if s["spec"] else s["k"].double()
        for n, x in ((0, k), (2, s["v"].double())):
            codes, e = _exact_quantise(x)
            out[n][pages, :, slots] = codes
            out[n + 1][pages, :, slots] = torch.exp2(e)
        return tuple(out)
    if op in ("read", "attend"):
        outs, pt, at = ([], []), case["pt"], 0
        for b, n in enumerate(ctx):
            pg = s["table"][b, : -(-n // pt)].long()
            rows = []
            for pool in (s["k_pool"], s["v_pool"]):
                x = pool[pg]
                codes = x[..., : pt * D].reshape(-1, case["Hkv"], pt, D).view(torch.float8_e4m3fn).double()
                x = codes * torch.exp2(x[..., pt * D:].double() - 127)[..., None]
                rows.append(x.transpose(0, 1).reshape(case["Hkv"], -1, D)[:, :n])
            if op == "read":
                for o, x in zip(outs, rows):
                    o.append(x.transpose(0, 1))
            else:
                q = s["q"][b].double().view(case["Hkv"], -1, D)
                p = torch.softmax(q @ rows[0].transpose(1, 2) / math.sqrt(D), -1)
                outs[0].append((p @ rows[1]).reshape(1, case["Hq"], 1, D))
        return (torch.cat(outs[0]), torch.cat(outs[1])) if op == "read" else torch.cat(outs[0])
    y, qa, ka = s["y"].double(), 0, 0
    for n, c in zip(new, ctx):
        q, k, v = s["q"][qa:qa + n], s["k"][ka:ka + c].double(), s["v"][ka:ka + c].double()
        last = torch.arange(n, device=DEV)[:, None] + (c - n)
        hide = (torch.arange(c, device=DEV)[None] > last) if case["causal"] else None
        for h in range(case["Hq"]):
            kv = h // (case["Hq"] // case["Hkv"])
            x = q[:, h].double() @ k[:, kv].T / math.sqrt(D)
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if hide is not None:
                x = x.masked_fill(hide, NEG)
            y[qa:qa + n, h] = torch.softmax(x, -1) @ v[:, kv]
        qa, ka = qa + n, ka + c
    return y
