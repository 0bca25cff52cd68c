"""GPU parity of paged_attn_decode over FP8 pages against 64-bit attention over the
pages' own values.

Tolerance: the codes and q enter the products exactly; an fp32 sum of D products is
off by at most D 2^-22 of the sum of magnitudes (a step of 2^-23 per addition, twice
for truncation), so a score by e_s = D 2^-22 max sum|q||k| scale, and with its
scaling and exp2 (2^-21 of up to 2^7 log2 units) a probability by 2 (e_s + 2^-14) of
itself; the probability times the value's scale is held to 2^-16; the sum and the
division add 2^-18.  An output is off by the total times sum p |v|, plus half a step."""
import math

import pytest
import torch

from oracle import serving as orc
from test_gpu_paged_kv import DT, Layout

pytestmark = pytest.mark.gpu
DEV = "cuda"


def fill(lay, Hkv, D, seed, spread=3):
    """Pools of random codes (NaN codes left out) and scale bytes."""
    g = torch.Generator().manual_seed(seed)
    pools = []
    for _ in range(2):
        p = torch.randint(0, 256, (lay.pages, Hkv, lay.pt * (D + 1)), generator=g, dtype=torch.uint8)
        c = p[..., :lay.pt * D]
        c[(c & 127) == 127] = 64
        p[..., lay.pt * D:] = torch.randint(119 - spread, 119 + spread, (lay.pages, Hkv, lay.pt), generator=g).to(torch.uint8)
        pools.append(p)
    return pools


def values(lay, pool, b, h, D):
    out = torch.empty(lay.ctx[b], D, dtype=torch.float64)
    for pi in range(-(-lay.ctx[b] // lay.pt)):
        page = int(lay.table[b, pi])
        codes = pool[page, h, :lay.pt * D].view(lay.pt, D)
        x = orc.dequantise_rows(codes, pool[page, h, lay.pt * D:])
        n = min(lay.pt, lay.ctx[b] - pi * lay.pt)
        out[pi * lay.pt:pi * lay.pt + n] = x[:n]
    return out


def check(y, q, lay, pools, scale=None, seqs=None):
    y = y.cpu()
    B, Hq, D = q.shape[0], q.shape[1], q.shape[-1]
    Hkv = pools[0].shape[1]
    g = Hq // Hkv
    scale = scale or 1 / math.sqrt(D)
    fi = torch.finfo(y.dtype)
    for b in range(B) if seqs is None else seqs:
        for h in range(Hkv):
            qq = q[b].reshape(Hq, D)[h * g:(h + 1) * g].double().cpu()
            want, mag, most = orc.attend(qq, values(lay, pools[0], b, h, D), values(lay, pools[1], b, h, D), scale)
            got = y[b].reshape(Hq, D)[h * g:(h + 1) * g].double()
            rel = 2 * (D * 2.0 ** -22 * most + 2.0 ** -14) + 2.0 ** -16 + 2.0 ** -18
            tol = rel * mag + (want.abs() + rel * mag) * fi.eps / 2 + fi.smallest_normal * fi.eps
            assert torch.isfinite(got).all()
            off = float(((got - want).abs() - tol).max())
            assert off <= 0, f"seq {b} head {h}: {off:.3e} over the bound"


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("ctx,pt,Hkv,g,D", [
    ([1], 16, 1, 1, 128), ([16], 16, 2, 4, 128), ([17, 1, 300, 15], 16, 2, 4, 128), ([33, 500], 32, 3, 8, 64),
    ([1000, 3, 64, 65], 64, 1, 16, 64), ([700, 90], 16, 2, 16, 128), ([257, 31], 16, 2, 6, 256), ([129], 48, 1, 32, 128),
    ([400, 2], 16, 1, 17, 256), ([5000, 1, 2, 3], 16, 8, 4, 128), ([90] * 33, 16, 1, 2, 64)])
def test_matches_64_bits(cuda_lib, dt, ctx, pt, Hkv, g, D):
    lay = Layout(ctx, ctx, pt, seed=D + len(ctx))
    pools = fill(lay, Hkv, D, 1)
    q = torch.randn(len(ctx), Hkv * g, 1, D, generator=torch.Generator().manual_seed(2)).to(DT[dt])
    table, ctx_t, _ = lay.gpu()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = cuda_lib.paged_attn_decode(q.to(DEV), pools[0].to(DEV), pools[1].to(DEV), table, ctx_t, err_word=err)
    torch.cuda.synchronize()
    assert int(err) == 0 and y.shape == q.shape
    check(y, q, lay, pools)
    y3 = cuda_lib.paged_attn_decode(q[:, :, 0].contiguous().to(DEV), pools[0].to(DEV), pools[1].to(DEV), table, ctx_t)
    assert torch.equal(y3, y[:, :, 0])                     # and the same again, bit for bit


def test_a_long_context_split_over_the_machine(cuda_lib):
    lay = Layout([70000, 5, 20000], [1, 1, 1], 16, seed=3)
    pools = fill(lay, 2, 128, 4)
    q = torch.randn(3, 8, 1, 128, generator=torch.Generator().manual_seed(5)).bfloat16()
    table, ctx_t, _ = lay.gpu()
    y = cuda_lib.paged_attn_decode(q.to(DEV), pools[0].to(DEV), pools[1].to(DEV), table, ctx_t, scale=0.05)
    check(y, q, lay, pools, scale=0.05)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_every_code_and_far_scales(cuda_lib, dt):
    """All 254 finite codes (subnormal ones among them) as K and as V; scales from 2^-60 to
    2^40 between the tokens of one sequence."""
    D, n = 128, 64
    lay = Layout([n], [n], 16)
    codes = torch.tensor([c for c in range(256) if c & 127 != 127], dtype=torch.uint8)
    pools = []
    for s in range(2):
        rows = codes[(torch.arange(n * D) * (7 if s else 1)) % 254].view(n, D)
        e = torch.tensor([127 - 60, 127, 127 + (40 if s else 0), 120], dtype=torch.uint8)[torch.arange(n) % 4]
        p = torch.zeros(lay.pages, 1, 16 * (D + 1), dtype=torch.uint8)
        for i in range(n):
            page, slot = lay.place(0, i)
            orc.write_row(p, page, 0, slot, 16, D, rows[i], e[i])
        pools.append(p)
    table, ctx_t, _ = lay.gpu()
    if dt == "f16":                                        # the output has to hold the result
        for i in range(n):
            page, slot = lay.place(0, i)
            b = pools[1][page, 0, 16 * D + slot]
            pools[1][page, 0, 16 * D + slot] = min(int(b), 120)
    for size in (1.0, 2.0 ** -13, 100.0):
        q = (torch.randn(1, 4, 1, D, generator=torch.Generator().manual_seed(1)) * size / 64).to(DT[dt])
        y = cuda_lib.paged_attn_decode(q.to(DEV), pools[0].to(DEV), pools[1].to(DEV), table, ctx_t, scale=2.0 ** -7 / size)
        check(y, q, lay, pools, scale=2.0 ** -7 / size)


def test_what_lies_behind_the_context_never_counts(cuda_lib):
    """NaN codes and NaN scales in the slots past the context, in its page and in others."""
    lay = Layout([37, 16, 1], [1] * 3, 32)
    pools = fill(lay, 2, 128, 7)
    clean = [p.clone() for p in pools]
    for p in pools:
        used = torch.zeros(lay.pages, 32, dtype=torch.bool)
        for b, c in enumerate(lay.ctx):
            for i in range(c):
                used[lay.place(b, i)] = True
        for page in range(lay.pages):
            for slot in range(32):
                if not used[page, slot]:
                    p[page, :, slot * 128:(slot + 1) * 128] = 0xFF
                    p[page, :, 32 * 128 + slot] = 255
    q = torch.randn(3, 8, 1, 128, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    table, ctx_t, _ = lay.gpu()
    a = cuda_lib.paged_attn_decode(q, pools[0].to(DEV), pools[1].to(DEV), table, ctx_t)
    b = cuda_lib.paged_attn_decode(q, clean[0].to(DEV), clean[1].to(DEV), table, ctx_t)
    assert torch.isfinite(a.float()).all() and torch.equal(a, b)


def test_nan_rows_and_nan_queries_come_out_as_nan(cuda_lib):
    lay = Layout([9000, 50], [1, 1], 16)
    table, ctx_t, _ = lay.gpu()
    q = torch.randn(2, 4, 1, 64, generator=torch.Generator().manual_seed(1)).half().to(DEV)
    for which in (0, 1):
        pools = fill(lay, 1, 64, 7)
        page, slot = lay.place(0, 4000)
        pools[which][page, 0, 16 * 64 + slot] = 255
        y = cuda_lib.paged_attn_decode(q, pools[0].to(DEV), pools[1].to(DEV), table, ctx_t)
        assert torch.isnan(y[0]).all() and torch.isfinite(y[1]).all()
    q[0, 2] = float("nan")
    pools = fill(lay, 1, 64, 7)
    y = cuda_lib.paged_attn_decode(q, pools[0].to(DEV), pools[1].to(DEV), table, ctx_t)
    assert torch.isnan(y[0, 2]).all() and torch.isfinite(y[0, [0, 1, 3]]).all() and torch.isfinite(y[1]).all()


def test_new_token_is_quantised_into_its_page_first(cuda_lib):
    sa = cuda_lib
    lay = Layout([33, 16, 1, 700], [1] * 4, 16)
    pools = fill(lay, 2, 128, 3)
    g = torch.Generator().manual_seed(4)
    q = torch.randn(4, 8, 1, 128, generator=g).bfloat16().to(DEV)
    kn, vn = (torch.randn(4, 2, 128, generator=g).bfloat16().to(DEV) for _ in range(2))
    table, ctx_t, _ = lay.gpu()
    a, b = [p.to(DEV) for p in pools], [p.to(DEV) for p in pools]
    y = sa.paged_attn_decode(q, *a, table, ctx_t, k_new=kn, v_new=vn)
    sa.paged_kv_write(kn, vn, *b, table, ctx_t)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(y, sa.paged_attn_decode(q, *b, table, ctx_t))
    check(y, q, lay, [p.cpu() for p in b])


def test_bad_contexts_and_table_entries(cuda_lib):
    sa = cuda_lib
    lay = Layout([40, 40, 40], [1] * 3, 16)
    pools = fill(lay, 2, 64, 3)
    q = torch.randn(3, 4, 1, 64, generator=torch.Generator().manual_seed(1)).half().to(DEV)
    table, ctx_t, _ = lay.gpu()
    for what in ("table", "long", "none"):
        t, c = table.clone(), ctx_t.clone()
        if what == "table":
            t[1, 0] = -3
        else:
            c[1] = 10 ** 6 if what == "long" else 0
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        y = sa.paged_attn_decode(q, *[p.to(DEV) for p in pools], t, c, err_word=err)
        assert int(err) == sa.ERRBIT_PAGE
        assert torch.isfinite(y.float()).all()
        # the other sequences are right; not bit for bit what they were: the tiles that one
        # sequence no longer has move where the others' contexts are cut, and so the order of
        # their sums, which the bound of check() allows for
        check(y, q, lay, pools, seqs=(0, 2))
        if what != "table":
            assert not y[1].any()                          # no context: zeros


def test_two_streams_and_two_graphs_at_once(cuda_lib):
    """Calls in flight together have scratch of their own: kept per stream, and a graph's own."""
    sa = cuda_lib
    lay = Layout([20000, 3000], [1, 1], 16, seed=8)
    pools = [p.to(DEV) for p in fill(lay, 2, 128, 5)]
    table, ctx_t, _ = lay.gpu()
    qs = [torch.randn(2, 8, 1, 128, generator=torch.Generator().manual_seed(i)).bfloat16().to(DEV) for i in range(2)]
    want = [sa.paged_attn_decode(q, *pools, table, ctx_t) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(sa.paged_attn_decode(qs[i], *pools, table, ctx_t, stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sa.paged_attn_decode(qs[i], *pools, table, ctx_t))
        graphs.append(g)
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(outs[i], want[i]) for i in range(2))


def test_a_workspace_of_the_callers(cuda_lib):
    sa = cuda_lib
    lay = Layout([20000], [1], 16)
    pools = [p.to(DEV) for p in fill(lay, 1, 64, 5)]
    table, ctx_t, _ = lay.gpu()
    q = torch.randn(1, 2, 1, 64).half().to(DEV)
    need = sa.paged_attn_decode_workspace(q, *pools, table, ctx_t)
    ws = sa.new_workspace(need, DEV).fill_(0xFF)
    y = sa.paged_attn_decode(q, *pools, table, ctx_t, workspace=ws)
    assert torch.equal(y, sa.paged_attn_decode(q, *pools, table, ctx_t))
    with pytest.raises(sa.SAError):
        sa.paged_attn_decode(q, *pools, table, ctx_t, workspace=sa.new_workspace(need - 1, DEV))


def test_refusals(cuda_lib):
    sa = cuda_lib
    lay = Layout([40], [1], 16)
    table, ctx_t, _ = lay.gpu()
    pools = [sa.new_fp8_pool(lay.pages, 2, 16, 128) for _ in range(2)]
    q = torch.zeros(1, 8, 1, 128, dtype=torch.float16, device=DEV)
    for kw in (dict(q=q.float()), dict(options=sa.OPT_ROW_COPIES)):
        with pytest.raises(sa.SAError):
            sa.paged_attn_decode(**dict(dict(q=q, k_pool=pools[0], v_pool=pools[1], block_table=table, ctx_len=ctx_t), **kw))
    kn = torch.zeros(1, 2, 128, dtype=torch.float16, device=DEV)
    for kw in (dict(q=q[..., :64].contiguous()), dict(v_pool=pools[1][:-1]), dict(k_new=kn.float(), v_new=kn.float()),
               dict(k_new=kn[..., :64].contiguous(), v_new=kn), dict(y=q.float()), dict(q=q.expand(1, 8, 2, 128).contiguous()),
               dict(ctx_len=ctx_t.expand(2).contiguous())):
        with pytest.raises(ValueError):
            sa.paged_attn_decode(**dict(dict(q=q, k_pool=pools[0], v_pool=pools[1], block_table=table, ctx_len=ctx_t), **kw))
    with pytest.raises(sa.SAError):
        sa.paged_attn_decode(q, *pools, table, ctx_t, k_new=kn)
    with pytest.raises(sa.SAError):
        sa.paged_attn_decode(q, pools[0], pools[0], table, ctx_t)


def bound_check(y, q, k, v, weight, scale, what):
    """One sequence's heads of one KV head against 64 bits.  Besides check()'s steps a value
    weight p 2^ev is held to 2^-25 of a unit in which the largest weight that counts (after
    the maximum's rises) is at least 2^6: 2^-31 of the largest, per token, times its code."""
    want, mag, most = orc.attend(q, k, v, scale)
    fi = torch.finfo(y.dtype)
    rel = 2 * (q.shape[-1] * 2.0 ** -22 * most + 2.0 ** -14) + 2.0 ** -16 + 2.0 ** -18
    p = torch.softmax(q.double() @ k.T * scale, -1)
    near = rel * mag + 2.0 ** -31 * (p * weight).amax(-1, keepdim=True) * (v / weight[:, None]).abs().sum(0)
    tol = near + (want.abs() + near) * fi.eps / 2 + fi.smallest_normal * fi.eps
    got = y.double().cpu()
    assert torch.isfinite(got).all(), what
    off = float(((got - want).abs() - tol).max())
    assert off <= 0, f"{what}: {off:.3e} over the bound, largest output {float(want.abs().max()):.3e}"


def shared_context(n, pt, Hkv, D, k, v, B):
    """FP8 pools with the rows k, v [n, Hkv, D] (quantised) as one context, and a table in
    which B sequences share its pages, so that a warp's range holds many tiles."""
    lay = Layout([n], [n], pt)
    pools, vals, weight = [], [], None
    for x in (k, v):
        codes, scales = orc.quantise_rows(x.reshape(-1, D))
        codes, scales = codes.view(n, Hkv, D), scales.view(n, Hkv)
        p = torch.zeros(lay.pages, Hkv, pt * (D + 1), dtype=torch.uint8)
        for i in range(n):
            page, slot = lay.place(0, i)
            for h in range(Hkv):
                orc.write_row(p, page, h, slot, pt, D, codes[i, h], scales[i, h])
        pools.append(p.to(DEV))
        vals.append(orc.dequantise_rows(codes, scales))
        weight = 2.0 ** (scales.double() - 127)
    table = lay.table.expand(B, -1).contiguous().to(DEV)
    return pools, table, torch.full((B,), n, dtype=torch.int32, device=DEV), vals, weight


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("drop,rise,how", [(16, 30, "step"), (20, 30, "step"), (26, 60, "step"), (30, 90, "step"),
                                           (16, 30, "ramp"), (24, 40, "ramp"), (30, 60, "ramp"), (28, 200, "ramp")])
def test_value_scales_fall_while_the_scores_rise(cuda_lib, dt, drop, rise, how):
    """Rows of large values that the running maximum soon scales away: the later rows'
    weights count in full."""
    n, Hkv, g, D, B = 192, 4, 4, 128, 240
    gen = torch.Generator().manual_seed(drop)
    q = (torch.rand(B, Hkv * g, 1, D, generator=gen) + 0.5).to(DT[dt])
    t = torch.arange(n).double() / (n - 1)
    t = (t > 0.2).double() if how == "step" else t
    scale = 1 / math.sqrt(D)
    up = rise * math.log(2) / (D * scale)                  # mean q is 1: `rise` log2 units of score
    k = 0.05 * torch.randn(n, Hkv, D, generator=gen).double() + (t * up)[:, None, None]
    v = torch.randn(n, Hkv, D, generator=gen).double() * torch.exp2(drop * (0.3 - t).round(decimals=3))[:, None, None]
    pools, table, ctx, vals, weight = shared_context(n, 16, Hkv, D, k, v, B)
    y = cuda_lib.paged_attn_decode(q.to(DEV), *pools, table, ctx)
    for b in (0, 1, 7, 100, 101, 102, 103, 239):
        for h in range(Hkv):
            bound_check(y[b, h * g:(h + 1) * g, 0], q[b, h * g:(h + 1) * g, 0].double(), vals[0][:, h], vals[1][:, h],
                        weight[:, h], scale, f"{dt} drop {drop} rise {rise} {how}: {b} {h}")


@pytest.mark.parametrize("dt,size", [("bf16", 2.0 ** -6), ("f16", 2.0 ** -6), ("bf16", 2.0 ** -26), ("bf16", 2.0 ** -60)])
@pytest.mark.parametrize("where", [(0,), (5, 700), (1990,), tuple(range(0, 2000, 3))])
def test_value_rows_of_zeros_say_nothing_about_the_others(cuda_lib, dt, size, where):
    """A row of zeros is stored with a scale of 1, whatever the size of the rows around it;
    here the zero rows have nearly all of the probability."""
    n, Hkv, g, D, B = 2000, 2, 4, 64, 200
    gen = torch.Generator().manual_seed(len(where))
    q = (torch.rand(B, Hkv * g, 1, D, generator=gen) + 0.5).to(DT[dt])
    k = 0.05 * torch.randn(n, Hkv, D, generator=gen).double()
    v = size * torch.randn(n, Hkv, D, generator=gen).double()
    k[list(where)] += 16 * math.log(2) / math.sqrt(D)      # 2^16 times the others' probability
    v[list(where)] = 0
    pools, table, ctx, vals, weight = shared_context(n, 16, Hkv, D, k, v, B)
    weight[list(where)] = weight.min()                     # (they hold nothing)
    y = cuda_lib.paged_attn_decode(q.to(DEV), *pools, table, ctx)
    for b in (0, 1, 66, 199):
        for h in range(Hkv):
            bound_check(y[b, h * g:(h + 1) * g, 0], q[b, h * g:(h + 1) * g, 0].double(), vals[0][:, h], vals[1][:, h],
                        weight[:, h], 1 / math.sqrt(D), f"{dt} {size} {where[:3]}: {b} {h}")


def test_a_nan_row_of_zero_codes_is_still_nan(cuda_lib):
    """What paged_kv_write stores for a row with a NaN: codes 0, scale byte 255."""
    n, D = 40, 64
    k = torch.randn(n, 1, D, generator=torch.Generator().manual_seed(1)).double()
    for at in (0, 17, 39):
        pools, table, ctx, _, _ = shared_context(n, 16, 1, D, k, k, 3)
        lay = Layout([n], [n], 16)
        page, slot = lay.place(0, at)
        pools[1][page, 0, slot * D:(slot + 1) * D] = 0
        pools[1][page, 0, 16 * D + slot] = 255
        y = cuda_lib.paged_attn_decode(torch.ones(3, 4, 1, D, device=DEV, dtype=torch.bfloat16), *pools, table, ctx)
        assert torch.isnan(y).all()


def test_two_threads_on_one_stream(cuda_lib):
    """Their calls' launches may alternate on the stream: each thread has scratch of its own."""
    import threading
    sa = cuda_lib
    lay = Layout([20000, 3000], [1, 1], 16, seed=8)
    pools = [p.to(DEV) for p in fill(lay, 2, 128, 5)]
    table, ctx_t, _ = lay.gpu()
    qs = [torch.randn(2, 8, 1, 128, generator=torch.Generator().manual_seed(i)).bfloat16().to(DEV) for i in range(4)]
    want = [sa.paged_attn_decode(q, *pools, table, ctx_t) for q in qs]
    torch.cuda.synchronize()
    got, barrier = [None] * 4, threading.Barrier(4)

    def work(i):
        barrier.wait()
        got[i] = [sa.paged_attn_decode(qs[i], *pools, table, ctx_t) for _ in range(100)]

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(4) for y in got[i])


@pytest.mark.parametrize("D,g", [(64, 16), (128, 16), (256, 8), (256, 16), (128, 3)])
@pytest.mark.parametrize("zeros", [False, True])
def test_the_same_for_every_form_of_the_kernel(cuda_lib, D, g, zeros):
    """Falling value scales under rising scores, or rows of zeros with most of the probability,
    for both numbers of MMA columns and every head size."""
    n, Hkv, B, dt = 192, 2, 300, "bf16"
    gen = torch.Generator().manual_seed(D + g)
    q = (torch.rand(B, Hkv * g, 1, D, generator=gen) + 0.5).to(DT[dt])
    t = (torch.arange(n) > n // 5).double()
    rise, drop = (12, 20) if zeros else (40, 26)
    k = 0.05 * torch.randn(n, Hkv, D, generator=gen).double() + (t * rise * math.log(2) / math.sqrt(D))[:, None, None]
    v = torch.randn(n, Hkv, D, generator=gen).double() * (2.0 ** -drop if zeros else torch.exp2(-drop * t)[:, None, None])
    if zeros:
        v[n // 2:] = 0
    pools, table, ctx, vals, weight = shared_context(n, 16, Hkv, D, k, v, B)
    if zeros:
        weight[n // 2:] = weight.min()
    y = cuda_lib.paged_attn_decode(q.to(DEV), *pools, table, ctx)
    for b in (0, 1, 150, 299):
        for h in range(Hkv):
            bound_check(y[b, h * g:(h + 1) * g, 0], q[b, h * g:(h + 1) * g, 0].double(), vals[0][:, h], vals[1][:, h],
                        weight[:, h], 1 / math.sqrt(D), f"D {D} group {g} zeros {zeros}: {b} {h}")
