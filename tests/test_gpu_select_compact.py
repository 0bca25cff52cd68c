"""GPU parity of paged_kv_select and paged_kv_compact with their plain forms: both are exact.
After them, the operators that keep a cache within a budget in a run."""
import math
import random

import pytest
import torch

import test_gpu_packed as packed
import test_gpu_paged_fp8 as fp8
import test_gpu_weights as wt
from oracle import eviction as ev
from test_gpu_paged_kv import DT, Layout

pytestmark = pytest.mark.gpu
DEV = "cuda"


def weights_like(lay, Hkv, kind, seed):
    g = torch.Generator().manual_seed(seed)
    shape = (lay.pages, Hkv, lay.pt)
    if kind == "spread":
        return torch.exp(3 * torch.randn(shape, generator=g))
    if kind == "ties":
        return torch.randint(0, 5, shape, generator=g).float()
    if kind == "zeros":
        return torch.where(torch.rand(shape, generator=g) < 0.02, 1.0, 0.0)
    if kind == "close":                                     # keys that differ in their last bits
        return 1 + torch.randint(0, 60, shape, generator=g).float() * 2.0 ** -23
    x = torch.randn(shape, generator=g)                     # "odd"
    x[torch.rand(shape, generator=g) < 0.1] = math.nan
    x[torch.rand(shape, generator=g) < 0.1] = -math.inf
    x[torch.rand(shape, generator=g) < 0.1] = math.inf
    x[torch.rand(shape, generator=g) < 0.2] = -0.0
    x[torch.rand(shape, generator=g) < 0.2] = 0.0
    x[torch.rand(shape, generator=g) < 0.1] = 1e-42
    return x


def selected(sa, lay, w, budget, sink, recent, Hkv):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    keep, n = sa.paged_kv_select(w.to(DEV), lay.table.to(DEV), lay.ctx_t.to(DEV), budget, sink=sink, recent=recent, err_word=err)
    assert int(err) == 0 and tuple(keep.shape) == (len(lay.ctx), Hkv, budget)
    keep = keep.cpu()
    assert n.tolist() == [min(c, budget) for c in lay.ctx]
    for b, c in enumerate(lay.ctx):
        page, slot = ev.token_places(lay.table[b], c, lay.pt)
        for h in range(Hkv):
            want = ev.select_row(w[page, h, slot].tolist(), budget, sink, recent)
            assert keep[b, h].tolist() == want + [-1] * (budget - len(want)), (b, h)
    return keep


@pytest.mark.parametrize("kind", ["spread", "ties", "zeros", "close", "odd"])
@pytest.mark.parametrize("ctx,pt,Hkv,budget,sink,recent", [
    ([1], 16, 1, 1, 0, 0), ([2, 1, 0], 16, 1, 1, 0, 0), ([40, 5, 300, 41], 16, 2, 40, 4, 8), ([100, 64, 65], 5, 3, 64, 0, 63),
    ([300] * 3, 1, 1, 16, 16, 0), ([513, 2047, 2049, 8191, 8192, 8193], 16, 1, 512, 3, 100), ([20000, 100], 64, 2, 777, 0, 256),
    ([70001], 32, 1, 5000, 4, 1000), ([9000, 17], 7, 2, 8999, 1, 2), ([150000], 16, 1, 300, 1, 1)])
def test_selection(cuda_lib, kind, ctx, pt, Hkv, budget, sink, recent):
    lay = Layout(ctx, [0] * len(ctx), pt, seed=pt)
    selected(cuda_lib, lay, weights_like(lay, Hkv, kind, budget), budget, sink, recent, Hkv)


def test_selection_in_a_table_far_wider_than_the_contexts(cuda_lib):
    lay = Layout([300, 40, 2000], [0] * 3, 16, seed=1, cols=20000)
    selected(cuda_lib, lay, weights_like(lay, 2, "spread", 2), 128, 4, 32, 2)


def test_selection_over_part_of_a_pool_off_16_bytes(cuda_lib):
    sa, lay = cuda_lib, Layout([500, 90], [0, 0], 16, seed=3)
    w = weights_like(lay, 2, "spread", 3)
    raw = torch.zeros(w.numel() + 1, device=DEV)
    odd = raw[1:].view(w.shape)
    odd.copy_(w)
    a = sa.paged_kv_select(odd, lay.table.to(DEV), lay.ctx_t.to(DEV), 64, sink=2, recent=8)
    b = sa.paged_kv_select(w.to(DEV), lay.table.to(DEV), lay.ctx_t.to(DEV), 64, sink=2, recent=8)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("B,Hkv", [(256, 3), (257, 3), (100, 8), (96, 9)])
def test_selection_of_many_contexts_whose_longest_go_first(cuda_lib, B, Hkv):
    rng = random.Random(B)
    ctx = [rng.choice([0, 1, 30, 31, 200, 200, rng.randint(32, 700)]) for _ in range(B)]
    ctx[0], ctx[-1] = 0, 700
    lay = Layout(ctx, [0] * B, 16, seed=B)
    selected(cuda_lib, lay, weights_like(lay, Hkv, "spread", B), 30, 2, 5, Hkv)


def test_selection_of_many_contexts_with_lengths_that_are_none(cuda_lib):
    sa, B, Hkv = cuda_lib, 200, 4
    lay = Layout([50] * B, [0] * B, 16, seed=6)
    w = weights_like(lay, Hkv, "spread", 6)
    ctx = lay.ctx_t.clone()
    bad = torch.arange(0, B, 3)
    ctx[bad] = torch.tensor([-1, -2147483648, 2147483647, 4096])[torch.arange(len(bad)) % 4].to(torch.int32)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    keep, n = sa.paged_kv_select(w.to(DEV), lay.table.to(DEV), ctx.to(DEV), 20, recent=4, err_word=err)
    keep = keep.cpu()
    assert int(err) == sa.ERRBIT_PAGE and n.tolist() == [0 if b % 3 == 0 else 20 for b in range(B)]
    for b in range(B):
        page, slot = ev.token_places(lay.table[b], 50, 16)
        for h in range(Hkv):
            want = [-1] * 20 if b % 3 == 0 else ev.select_row(w[page, h, slot].tolist(), 20, 0, 4)
            assert keep[b, h].tolist() == want, (b, h)


def test_selection_reports_bad_contexts_and_pages(cuda_lib):
    sa, lay = cuda_lib, Layout([100, 100, 100], [0] * 3, 16, seed=4)
    w = weights_like(lay, 1, "spread", 4) + 1
    lay.table[1, 2] = lay.pages
    ctx = torch.tensor([-1, 100, 1 << 30], dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    keep, n = sa.paged_kv_select(w.to(DEV), lay.table.to(DEV), ctx, 90, err_word=err)
    assert int(err) == sa.ERRBIT_PAGE and n.tolist() == [0, 90, 0]
    assert (keep[0] == -1).all() and (keep[2] == -1).all()
    page, slot = ev.token_places(torch.where(lay.table[1] < lay.pages, lay.table[1], 0), 100, 16)
    line = w[page, 0, slot]
    line[32:48] = -math.inf                                 # the bad page's tokens
    assert keep[1, 0].tolist() == ev.select_row(line.tolist(), 90, 0, 0)


def test_selection_is_what_the_selected_token_decode_takes(cuda_lib):
    """keep rows validate, and give the attention over the kept tokens."""
    sa, Hkv, D, T = cuda_lib, 2, 64, 300
    lay = Layout([T], [0], 16, seed=5)
    lay.table[0, :19] = torch.arange(19)
    w = weights_like(lay, Hkv, "spread", 5)
    keep, _ = sa.paged_kv_select(w.to(DEV), lay.table.to(DEV), lay.ctx_t.to(DEV), 100, sink=4, recent=16)
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(1, H, S, D, generator=g).bfloat16().to(DEV) for H, S in ((8, 1), (Hkv, T), (Hkv, T)))
    idx = keep[:, :, None]                                  # [B, I = Hkv, Sq = 1, K]
    status, err = sa.validate_indices(idx.contiguous(), bound=T)
    assert int(err) == 0 and int(status.sum()) == 0
    y = sa.sparse_attn_decode(q, k, v, idx.contiguous())
    for h in range(8):
        at = keep[0, h // 4].long()
        p = torch.softmax(q[0, h].double() @ k[0, h // 4, at].double().T / math.sqrt(D), -1)
        assert (y[0, h].double() - p @ v[0, h // 4, at].double()).abs().max() < 0.05


def test_selection_refusals(cuda_lib):
    sa = cuda_lib
    w, t = sa.new_weight_pool(4, 2, 16), torch.zeros(1, 4, dtype=torch.int32, device=DEV)
    c = torch.ones(1, dtype=torch.int32, device=DEV)
    for bad in (dict(weights=w.double()), dict(block_table=t.long()), dict(ctx_len=c.long()), dict(weights=w.cpu())):
        with pytest.raises(TypeError):
            sa.paged_kv_select(**{**dict(weights=w, block_table=t, ctx_len=c, budget=4), **bad})
    for bad in (dict(weights=w[0]), dict(block_table=t[0]), dict(keep=torch.zeros(7, dtype=torch.int32, device=DEV)),
                dict(new_len=torch.zeros(2, dtype=torch.int32, device=DEV))):
        with pytest.raises(ValueError):
            sa.paged_kv_select(**{**dict(weights=w, block_table=t, ctx_len=c, budget=4), **bad})
    for bad in (dict(budget=0), dict(sink=5), dict(sink=2, recent=3), dict(recent=-1), dict(new_len=c)):
        with pytest.raises(sa.SAError):
            sa.paged_kv_select(**{**dict(weights=w, block_table=t, ctx_len=c, budget=4), **bad})


# ---- compaction --------------------------------------------------------------------------------


def lists(lay, Hkv, width, seed, most=None):
    rng = random.Random(seed)
    keep = torch.full((len(lay.ctx), Hkv, width), -1, dtype=torch.int32)
    for b, n in enumerate(lay.ctx):
        for h in range(Hkv):
            m = rng.randint(0, min(n, width)) if most is None else min(n, width, most)
            rows = sorted(rng.sample(range(n), m))
            if h == 0 and m > 3:
                rows[:3] = [0, 1, 2] if rows[3] > 2 else rows[:3]
            keep[b, h, :m] = torch.tensor(rows, dtype=torch.int32)
    return keep


def planes(pool, lay, D):
    if pool.dtype != torch.uint8:
        return [pool]
    return [pool[..., :lay.pt * D].unflatten(-1, (lay.pt, D)), pool[..., lay.pt * D:]]


def compacted(sa, lay, pools, w, keep, D, **kw):
    want = [p.clone() for p in pools] + ([] if w is None else [w.clone()])
    for x in sum((planes(p, lay, D) for p in want), []) if w is None else \
            sum((planes(p, lay, D) for p in want[:2]), []) + [want[2]]:
        for b in range(len(lay.ctx)):
            for h in range(keep.shape[1]):
                ev.compact_row(x, lay.table[b], lay.pt, h, [i for i in keep[b, h].tolist() if i >= 0])
    got = [p.to(DEV) for p in pools]
    gw = None if w is None else w.to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sa.paged_kv_compact(*got, lay.table.to(DEV), lay.ctx_t.to(DEV), keep.to(DEV), weights=gw, err_word=err, **kw)
    assert int(err) == 0
    for x, y in zip(got + ([] if w is None else [gw]), want):
        assert torch.equal(x.cpu().view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("ctx,pt,Hkv,D,width", [
    ([1], 16, 1, 64, 1), ([40, 5, 300, 0], 16, 2, 128, 40), ([513, 2047], 32, 3, 64, 600), ([5000, 100], 16, 1, 256, 2500),
    ([900] * 40, 48, 2, 128, 512), ([30000], 16, 2, 128, 20000), ([200, 200], 16, 1, 64, 5000)])
def test_compaction_of_quantised_pages(cuda_lib, ctx, pt, Hkv, D, width):
    lay = Layout(ctx, [0] * len(ctx), pt, seed=D)
    g = torch.Generator().manual_seed(1)                    # any bytes: NaN codes and scales among them
    pools = [torch.randint(0, 256, (lay.pages, Hkv, pt * (D + 1)), generator=g, dtype=torch.uint8) for _ in range(2)]
    for most in (None, width):
        compacted(cuda_lib, lay, pools, weights_like(lay, Hkv, "odd", 2), lists(lay, Hkv, width, width, most), D)
    compacted(cuda_lib, lay, pools, None, lists(lay, Hkv, width, 3), D, head_dim=D)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("ctx,pt,Hkv,D,width", [
    ([1], 16, 1, 64, 1), ([40, 5, 300, 0], 5, 2, 128, 40), ([513, 2047], 1, 3, 80, 600), ([700, 100], 16, 1, 1, 500),
    ([700, 100], 16, 2, 3, 500), ([60, 90], 7, 1, 1023, 50), ([60, 90], 7, 1, 1024, 50), ([20000], 16, 2, 128, 15000)])
def test_compaction_of_pages_of_elements(cuda_lib, dt, ctx, pt, Hkv, D, width):
    lay = Layout(ctx, [0] * len(ctx), pt, seed=D)
    pools = wt.elements(lay, Hkv, D, dt, 3)
    for most in (None, width):
        compacted(cuda_lib, lay, pools, weights_like(lay, Hkv, "spread", 4), lists(lay, Hkv, width, D, most), D)
    compacted(cuda_lib, lay, pools, None, lists(lay, Hkv, width, 3), D)


def test_compaction_again_and_again(cuda_lib):
    """Rows moved by ones, by whole chunks and not at all: shifts of every kind."""
    lay = Layout([4000], [0], 16, seed=6)
    g = torch.Generator().manual_seed(6)
    pools = [torch.randint(0, 256, (lay.pages, 1, 16 * 65), generator=g, dtype=torch.uint8) for _ in range(2)]
    w = weights_like(lay, 1, "spread", 6)
    for rows in (range(4000), range(1, 4000), range(0, 4000, 2), list(range(2000)) + list(range(2001, 4000)),
                 range(3000, 4000), [3999], [0, 3999]):
        keep = torch.tensor(list(rows), dtype=torch.int32).view(1, 1, -1)
        compacted(cuda_lib, lay, pools, w, keep, 64)


def test_compaction_leaves_rows_whose_list_is_no_list(cuda_lib):
    sa, lay = cuda_lib, Layout([100] * 7, [0] * 7, 16, seed=7)
    pools = wt.elements(lay, 1, 64, "bf16", 7)
    keep = torch.full((7, 1, 8), -1, dtype=torch.int32)
    bad = [[3, -1, 5], [3, 2], [3, 3], [3, 100], [-2, 3], [99, 2 ** 31 - 1], [5, 9]]
    codes = [sa.IDX_AFTER_PADDING, sa.IDX_NOT_INCREASING, sa.IDX_DUPLICATE, sa.IDX_OUT_OF_RANGE, sa.IDX_BELOW_SENTINEL,
             sa.IDX_OUT_OF_RANGE, 0]
    for b, r in enumerate(bad):
        keep[b, 0, :len(r)] = torch.tensor(r, dtype=torch.int32)
        assert ev.row_code(keep[b, 0].tolist(), 100)[1] == codes[b]
    got, err = [p.to(DEV) for p in pools], torch.zeros(1, dtype=torch.int32, device=DEV)
    sa.paged_kv_compact(*got, lay.table.to(DEV), lay.ctx_t.to(DEV), keep.to(DEV), err_word=err)
    assert int(err) == sum(set(codes))
    for x, p in zip(got, pools):
        want = p.clone()
        ev.compact_row(want, lay.table[6], 16, 0, [5, 9])
        assert torch.equal(x.cpu(), want)


def test_compaction_reports_bad_contexts_and_pages(cuda_lib):
    sa, lay = cuda_lib, Layout([100] * 3, [0] * 3, 16, seed=8)
    pools = wt.elements(lay, 1, 64, "bf16", 8)
    lay.table[0, 3] = -1
    lay.table[0, 0] = 0                                     # (the page that the rows go to)
    keep = torch.tensor([[[40, 50, 60]], [[1, 2, 3]], [[1, 2, 3]]], dtype=torch.int32)
    ctx = torch.tensor([100, -5, 1 << 29], dtype=torch.int32, device=DEV)
    got, err = [p.to(DEV) for p in pools], torch.zeros(1, dtype=torch.int32, device=DEV)
    sa.paged_kv_compact(*got, lay.table.to(DEV), ctx, keep.to(DEV), err_word=err)
    assert int(err) == sa.ERRBIT_PAGE
    for x, p in zip(got, pools):  # token 50 lies on the page that does not exist: its row stays
        want = p.clone()
        page = lay.table[0].long()
        want[0, 0, 0] = p[page[2], 0, 8]
        assert torch.equal(x.cpu(), want)


def test_compaction_past_2_31_bytes(cuda_lib):
    sa, D, pt, pages = cuda_lib, 128, 16, 140000
    pools = [torch.empty((pages, 8, pt, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    w = torch.empty((pages, 8, pt), device=DEV)
    table = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32, device=DEV)
    ctx = torch.tensor([40], dtype=torch.int32, device=DEV)
    for p in pools + [w]:
        p[pages - 3:] = torch.randn(3, *p.shape[1:]).to(p.dtype).to(DEV)
    near = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    small = [p[pages - 3:].clone() for p in pools + [w]]
    keep = torch.tensor([1, 5, 17, 18, 33, 39], dtype=torch.int32, device=DEV).expand(1, 8, 6).contiguous()
    sa.paged_kv_compact(*pools, table, ctx, keep, weights=w)
    sa.paged_kv_compact(*small[:2], near, ctx, keep, weights=small[2])
    for p, x in zip(pools + [w], small):
        assert torch.equal(p[pages - 3:], x)
    sel = [sa.paged_kv_select(x, t, ctx, 9, sink=1, recent=3)[0] for x, t in ((w, table), (small[2], near))]
    assert torch.equal(*sel)


def test_compaction_refusals(cuda_lib):
    sa = cuda_lib
    e = [torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    f = [sa.new_fp8_pool(4, 2, 16, 64) for _ in range(2)]
    t, c = torch.zeros(1, 4, dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    keep = torch.zeros(1, 2, 4, dtype=torch.int32, device=DEV)
    for bad in (dict(keep=keep.long()), dict(ctx_len=c.long()), dict(k_pool=e[0].cpu()), dict(weights=torch.zeros(4, 2, 16, device=DEV).half())):
        with pytest.raises((TypeError, ValueError)):
            sa.paged_kv_compact(**{**dict(k_pool=e[0], v_pool=e[1], block_table=t, ctx_len=c, keep=keep), **bad})
    for bad in (dict(keep=keep[:, :1]), dict(keep=keep[0]), dict(v_pool=e[1][:3]), dict(head_dim=32), dict(k_pool=f[0], v_pool=f[1]),
                dict(k_pool=f[0], v_pool=f[1], head_dim=100), dict(weights=sa.new_weight_pool(4, 2, 32)),
                dict(k_pool=f[0], v_pool=f[1], weights=sa.new_weight_pool(4, 2, 4000))):
        with pytest.raises(ValueError):
            sa.paged_kv_compact(**{**dict(k_pool=e[0], v_pool=e[1], block_table=t, ctx_len=c, keep=keep), **bad})
    with pytest.raises(sa.SAError, match="overlap"):
        sa.paged_kv_compact(e[0], e[0], t, c, keep)


# ---- in a run -------------------------------------------------------------------------------------


@pytest.mark.parametrize("quantised", [True, False])
def test_a_cache_kept_within_its_budget(cuda_lib, quantised):
    """Prompts prefilled, counted and cut to a budget; decode steps that count on, over the
    compacted pages; cut again.  Each stage against its plain form on the stage's own inputs."""
    sa, Hq, Hkv, D, pt, budget, sink, recent = cuda_lib, 8, 2, 64, 16, 64, 4, 16
    n, steps = [150, 40, 90], 20
    room = [max(a, budget) + steps for a in n]
    B, g = len(n), Hq // Hkv
    lay = Layout(room, room, pt, seed=12)
    table = lay.table.to(DEV)
    gen = torch.Generator().manual_seed(12)
    pools = [sa.new_fp8_pool(lay.pages, Hkv, pt, D) if quantised else
             torch.zeros(lay.pages, Hkv, pt, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    w = torch.full((lay.pages, Hkv, pt), 7.0, device=DEV)   # pages that others have used
    rope, err = sa.rope_table(D), torch.zeros(1, dtype=torch.int32, device=DEV)
    qs, ks, vs = ([torch.randn(a, H, D, generator=gen).bfloat16() for a in n] for H in (Hq, Hkv, Hkv))
    q, k, v = (torch.cat(x).to(DEV) for x in (qs, ks, vs))
    s = [0]
    for a in n:
        s.append(s[-1] + a)
    pos = torch.cat([torch.arange(a) for a in n]).to(DEV)
    ctx = torch.tensor(n, dtype=torch.int32, device=DEV)
    q, k = sa.rotary_embed(q, k, pos, rope)
    sa.paged_kv_write(k, v, *pools, table, ctx, packed.starts(s), err_word=err)
    y = sa.attn_prefill_packed(q, k, v, packed.starts(s), err_word=err)
    packed.check(y, q.cpu(), k.cpu(), v.cpu(), s, s)
    before = w.cpu()
    sa.attn_weights_packed(q, k, w, table, packed.starts(s), err_word=err)
    lay.ctx, lay.ctx_t = n, ctx.cpu()
    wt.check(w, before, lay, ev.weights_packed(q.cpu(), k.cpu(), s, s), n, D, [a * g for a in n])

    def cut():
        lay.ctx, lay.ctx_t = ctx.tolist(), ctx.cpu()
        before = [p.cpu() for p in pools], w.cpu()
        keep = selected(sa, lay, before[1], budget, sink, recent, Hkv)
        _, new = sa.paged_kv_select(w, table, ctx, budget, sink=sink, recent=recent, err_word=err)
        sa.paged_kv_compact(*pools, table, ctx, keep.to(DEV), weights=w, err_word=err)
        for b in range(B):
            for h in range(Hkv):
                rows = [i for i in keep[b, h].tolist() if i >= 0]
                for p in before[0]:
                    for x in planes(p, lay, D):
                        ev.compact_row(x, lay.table[b], pt, h, rows)
                ev.compact_row(before[1], lay.table[b], pt, h, rows)
        assert all(torch.equal(p.cpu(), x) for p, x in zip(pools, before[0])) and torch.equal(w.cpu(), before[1])
        ctx.copy_(new)

    cut()
    assert ctx.tolist() == [64, 40, 64]
    place = torch.tensor(n, device=DEV)                     # the true positions go on
    for _ in range(steps):
        q1, k1, v1 = (torch.randn(B, H, D, generator=gen).bfloat16().to(DEV) for H in (Hq, Hkv, Hkv))
        ctx += 1
        q1, k1 = sa.rotary_embed(q1, k1, place, rope)
        place += 1
        sa.paged_kv_write(k1, v1, *pools, table, ctx, err_word=err)
        before = w.cpu()
        y = sa.paged_attn_decode(q1, *pools, table, ctx, weights=w, err_word=err)
        lay.ctx, lay.ctx_t = ctx.tolist(), ctx.cpu()
        kc = pools[0].cpu()
        wt.check(w, before, lay, [ev.weights_decode(q1[b].cpu(), wt.keys_of(lay, kc, b, D), D ** -0.5) for b in range(B)],
                 [1] * B, D, [g] * B)
    if quantised:
        fp8.check(y[:, :, None], q1[:, :, None], lay, [p.cpu() for p in pools])
    cut()
    assert ctx.tolist() == [64, 60, 64] and int(err) == 0


@pytest.mark.parametrize("quantised", [True, False])
def test_a_captured_step_that_keeps_its_budget(cuda_lib, quantised):
    """A token written and attended to, the tokens to keep selected, their rows moved, the
    lengths set back: one graph, replayed with new tokens, against the calls one by one."""
    sa, Hq, Hkv, D, pt, budget, sink, recent = cuda_lib, 8, 2, 64, 16, 40, 2, 8
    n = [39, 40, 7]
    lay = Layout([budget + 1] * 3, [1] * 3, pt, seed=15)
    table = lay.table.to(DEV)
    pools = [p.to(DEV) for p in (fp8.fill(lay, Hkv, D, 15) if quantised else wt.elements(lay, Hkv, D, "bf16", 15))]
    w, ctx = wt.pool_of(lay, Hkv, 15).to(DEV), torch.tensor(n, dtype=torch.int32, device=DEV)
    q, k, v = (torch.zeros(3, H, D, dtype=torch.bfloat16, device=DEV) for H in (Hq, Hkv, Hkv))
    err, gen = torch.zeros(1, dtype=torch.int32, device=DEV), torch.Generator().manual_seed(15)

    def step(pools, w, ctx):
        ctx += 1
        y = sa.paged_attn_decode(q, *pools, table, ctx, k_new=k, v_new=v, weights=w, err_word=err)
        seen = w.clone()
        keep, left = sa.paged_kv_select(w, table, ctx, budget, sink=sink, recent=recent, err_word=err)
        sa.paged_kv_compact(*pools, table, ctx, keep, weights=w, head_dim=D, err_word=err)
        ctx.copy_(left)
        return y, seen, keep

    step([p.clone() for p in pools], w.clone(), ctx.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(pools, w, ctx)
    for _ in range(6):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=gen).bfloat16())
        lens = [c + 1 for c in ctx.tolist()]
        own = [p.clone() for p in pools], w.clone(), ctx.clone()
        graph.replay()
        want = step(*own)
        for a, b in zip((*out, *pools, w, ctx), (*want, *own[0], own[1], own[2])):
            assert torch.equal(a, b)
        for b, c in enumerate(lens):
            page, slot = ev.token_places(lay.table[b], c, pt)
            for h in range(Hkv):
                rows = ev.select_row(out[1].cpu()[page, h, slot].tolist(), budget, sink, recent)
                assert out[2][b, h].tolist() == rows + [-1] * (budget - len(rows))
    assert ctx.tolist() == [40, 40, 13] and int(err) == 0
