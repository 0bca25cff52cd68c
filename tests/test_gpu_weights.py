"""GPU parity of attn_weights_packed and of paged_attn_decode's weights against 64 bits.

Tolerance: an fp32 sum of D products is off by at most D 2^-22 of the sum of magnitudes (a
step of 2^-23 per addition, twice for truncation), so a score by e = D 2^-22 max sum|q||k|
scale.  In log2 units, of up to U = 1.45 max sum|q||k| scale, the scaling, the row's
logarithm and their difference add roundings of 2^-24 each of at most 2 U + 32, the row's
sum and exp2 2^-20: a probability is off by 2 (e + 2^-22 (4 U + 64)) + 2^-19 of itself, once
for the score and once for the row.  A weight adds those up, in sums of at most 64 + n / 32
additions of 2^-24 each for n queries times heads."""
import math

import pytest
import torch

import test_gpu_packed as packed
import test_gpu_paged_fp8 as fp8
from oracle import eviction as ev
from test_gpu_paged_kv import DT, Layout

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rel_bound(D, most, n):
    u = 1.45 * most
    return 2 * (D * 2.0 ** -22 * most + 2.0 ** -22 * (4 * u + 64)) + 2.0 ** -19 + (64 + n / 32) * 2.0 ** -24


def pool_of(lay, Hkv, seed=0):
    return torch.rand(lay.pages, Hkv, lay.pt, generator=torch.Generator().manual_seed(seed)) * 4


def check(got, before, lay, ws, fresh, D, rows):
    """The pool against `ws` [(w, most)] put into `before`: the tokens within their bound, the
    rest of the pool bit for bit."""
    got = got.cpu()
    touched = torch.zeros(got.shape, dtype=torch.bool)
    for b, (w, most) in enumerate(ws):
        n = w.shape[1]
        if n == 0 or rows[b] == 0:
            continue
        page, slot = ev.token_places(lay.table[b], n, lay.pt)
        touched[page, :, slot] = True
        old = before[page, :, slot].double()
        old[n - min(fresh[b], n):] = 0
        want = old + w.T
        have = got[page, :, slot].double()
        tol = w.T * rel_bound(D, most, rows[b]) + want.abs() * 2.0 ** -24 + 1e-30
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(have), nan)
        off = ((have - want).abs() - tol)[~nan]
        assert off.numel() == 0 or float(off.max()) <= 0, f"sequence {b}: {float(off.max()):.3e} over the bound"
    assert torch.equal(got[~touched], before[~touched])


def run(sa, dt, nq, nk, Hq, Hkv, D, pt=16, accumulate=True, scale=0.0, seed=0, pad=2):
    q, k, _, qs, ks = packed.make(dt, nq, nk, Hq, Hkv, D, seed, pad)
    lay = Layout(nk, nq, pt, seed=seed)
    before = pool_of(lay, Hkv, seed)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = sa.attn_weights_packed(q.to(DEV), k.to(DEV), before.to(DEV), lay.table.to(DEV), packed.starts(qs),
                                 packed.starts(ks), scale=scale, accumulate=accumulate, err_word=err)
    ws = ev.weights_packed(q, k, qs, ks, scale)
    g = Hq // Hkv
    check(got, before, lay, ws, nq if accumulate else nk, D, [n * g for n in nq])
    assert int(err) == 0
    return got


# ---- packed queries ---------------------------------------------------------------------------


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("nq,nk,Hq,Hkv,D", [
    ([1], [1], 1, 1, 64), ([1], [300], 4, 1, 128), ([5, 1, 0, 130], [5, 700, 9, 130], 8, 2, 64),
    ([128, 256], [128, 256], 4, 4, 128), ([127, 129, 33], [127, 400, 33], 6, 2, 128), ([300], [300], 5, 1, 64),
    ([700], [1500], 16, 1, 128), ([40] * 9, [41] * 9, 12, 4, 64), ([70], [70], 32, 1, 64), ([9], [520], 128, 1, 64)])
def test_matches_64_bits(cuda_lib, dt, nq, nk, Hq, Hkv, D):
    run(cuda_lib, dt, nq, nk, Hq, Hkv, D, seed=D + Hq)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_more_queries_than_keys(cuda_lib, dt):
    """The queries before the first key see nothing; a sequence without keys has nothing to set."""
    run(cuda_lib, dt, [300, 5, 40, 1], [20, 4, 0, 1], 8, 2, 64, seed=3)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("accumulate", [True, False])
def test_pages_of_any_size_set_and_added(cuda_lib, dt, accumulate):
    for pt in (1, 5, 16, 128, 1000):
        run(cuda_lib, dt, [33, 2, 64], [260, 2, 70], 4, 2, 64, pt=pt, accumulate=accumulate, seed=pt)


@pytest.mark.parametrize("D,dt", [(4, "f32"), (80, "bf16"), (96, "f16"), (256, "bf16"), (256, "f32"), (36, "f32")])
def test_other_head_sizes(cuda_lib, D, dt):
    run(cuda_lib, dt, [65, 3], [65, 210], 6, 3, D, seed=D)


def test_scales(cuda_lib):
    run(cuda_lib, "bf16", [50], [90], 4, 2, 64, scale=0.5)
    run(cuda_lib, "bf16", [50], [90], 4, 2, 64, scale=-0.25)  # (the fp32 pipes)


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (3, 1), (10, 2)])
def test_what_is_nobodys_never_counts(cuda_lib, Hq, Hkv):
    """NaN in rows of no sequence, in a neighbour's keys and in keys that no query sees leaves the
    bits of the others."""
    sa, D = cuda_lib, 64
    nq, nk = [70, 41, 5], [70, 200, 133]
    q, k, _, qs, ks = packed.make("bf16", nq, nk, Hq, Hkv, D, seed=5, pad=130)
    lay = Layout(nk, nq, 16, seed=5)
    args = (lay.table.to(DEV), packed.starts(qs), packed.starts(ks))
    clean = sa.attn_weights_packed(q.to(DEV), k.to(DEV), pool_of(lay, Hkv).to(DEV), *args)
    q[qs[-1]:], k[ks[-1]:] = math.nan, math.inf
    q[qs[1]:qs[2]], k[ks[1]:ks[2]] = math.nan, math.nan
    got = sa.attn_weights_packed(q.to(DEV), k.to(DEV), pool_of(lay, Hkv).to(DEV), *args)
    for b in (0, 2):
        page, slot = ev.token_places(lay.table[b], nk[b], 16)
        assert torch.equal(got.cpu()[page, :, slot], clean.cpu()[page, :, slot])
    page, slot = ev.token_places(lay.table[1], nk[1], 16)
    assert torch.isnan(got.cpu()[page, :, slot]).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_nan_query_and_keys_that_are_not_finite(cuda_lib, dt):
    """A row with a NaN score gives NaN to every key that it sees, to no other; a key of -inf
    scores receives nothing."""
    sa, D, n = cuda_lib, 64, 200
    q, k, _, qs, ks = packed.make(dt, [n], [n], 2, 1, D, seed=6, pad=0)
    q = q.abs() + 0.1
    q[150, 1, 3] = math.nan
    k[20, 0, 5] = -math.inf
    lay = Layout([n], [n], 16, seed=6)
    got = sa.attn_weights_packed(q.to(DEV), k.to(DEV), pool_of(lay, 1).to(DEV), lay.table.to(DEV), packed.starts(qs))
    page, slot = ev.token_places(lay.table[0], n, 16)
    w = got.cpu()[page, 0, slot]
    assert torch.isnan(w[:151]).all() and torch.isfinite(w[151:]).all()
    q[150, 1, 3] = 1.0
    got = sa.attn_weights_packed(q.to(DEV), k.to(DEV), pool_of(lay, 1).to(DEV), lay.table.to(DEV), packed.starts(qs))
    w = got.cpu()[page, 0, slot]
    assert torch.isfinite(w).all() and w[20] == 0 and (w[:20] > 0).all()


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("f16", 128), ("f32", 64)])
@pytest.mark.parametrize("g", [1, 3, 4, 5, 6, 7, 10, 12, 33, 65, 127])
def test_keys_of_infinite_scores_in_groups_of_any_size(cuda_lib, dt, D, g):
    """Keys whose score is -inf for every query receive 0, the others what the definition gives:
    also where the heads of a group leave rows of a query tile unfilled."""
    sa, nq, nk = cuda_lib, [260, 40], [260, 500]
    q, k, _, qs, ks = packed.make(dt, nq, nk, 2 * g, 2, D, seed=g, pad=3)
    q[:, :, 5] = q[:, :, 5].abs() + 0.1
    for b in range(2):
        k[ks[b] + 20, 0, 5] = -math.inf
        k[ks[b] + 77, :, 5] = -math.inf
    lay = Layout(nk, nq, 16, seed=g)
    before = pool_of(lay, 2, g)
    got = sa.attn_weights_packed(q.to(DEV), k.to(DEV), before.to(DEV), lay.table.to(DEV), packed.starts(qs), packed.starts(ks))
    check(got, before, lay, ev.weights_packed(q, k, qs, ks), nq, D, [n * g for n in nq])


def test_strided_views(cuda_lib):
    sa, D, n = cuda_lib, 128, 150
    g = torch.Generator().manual_seed(7)
    qkv = torch.randn(n, 8 + 4, D, generator=g).bfloat16().to(DEV)
    q, k = qkv[:, :8], qkv[:, 8:10]
    lay = Layout([n], [n], 16, seed=7)
    t = lay.table.to(DEV)
    a = sa.attn_weights_packed(q, k, pool_of(lay, 2).to(DEV), t, packed.starts([0, n]))
    b = sa.attn_weights_packed(q.contiguous(), k.contiguous(), pool_of(lay, 2).to(DEV), t, packed.starts([0, n]))
    assert torch.equal(a, b)
    shared = k[:, :1].expand(-1, 2, -1)                       # stride 0: the fp32 pipes
    c = sa.attn_weights_packed(q, shared, pool_of(lay, 2).to(DEV), t, packed.starts([0, n]))
    check(c, pool_of(lay, 2), lay, ev.weights_packed(q.cpu(), shared.cpu(), [0, n], [0, n]), [n], D, [4 * n])
    odd = torch.randn(n, 2 * D + 1, generator=g).bfloat16().to(DEV)[:, 1:].view(n, 2, D)  # off by two bytes
    d = sa.attn_weights_packed(odd, odd[:, :1], pool_of(lay, 1).to(DEV), t, packed.starts([0, n]))
    check(d, pool_of(lay, 1), lay, ev.weights_packed(odd.cpu(), odd[:, :1].cpu(), [0, n], [0, n]), [n], D, [2 * n])


@pytest.mark.parametrize("D,gap", [(36, 0), (36, 1), (128, 3), (20, 4)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_that_four_elements_do_not_divide(cuda_lib, dt, D, gap):
    """On the fp32 pipes: q's tokens `gap` elements apart, k's rows whole, and the other way round."""
    sa, n = cuda_lib, 140
    g = torch.Generator().manual_seed(D + gap)
    wide = torch.randn(n, 4 * D + gap, generator=g).to(DT[dt]).to(DEV)[:, :4 * D].unflatten(1, (4, D))
    whole = torch.randn(n, 4, D, generator=g).to(DT[dt]).to(DEV)
    lay = Layout([n], [n], 16, seed=D)
    for q, k in ((wide, whole[:, :2]), (whole, wide[:, 1:3])):
        got = sa.attn_weights_packed(q, k, pool_of(lay, 2).to(DEV), lay.table.to(DEV), packed.starts([0, n]), scale=-0.2)
        check(got, pool_of(lay, 2), lay, ev.weights_packed(q.cpu(), k.cpu(), [0, n], [0, n], -0.2), [n], D, [2 * n])


@pytest.mark.parametrize("nq,nk,Hq,Hkv", [([4000], [4000], 2, 1), ([3000, 10], [3000, 9000], 16, 1), ([1], [30000], 8, 1)])
def test_items_cut_between_multiprocessors_and_the_same_every_time(cuda_lib, nq, nk, Hq, Hkv):
    a = run(cuda_lib, "bf16", nq, nk, Hq, Hkv, 64, pad=0)
    b = run(cuda_lib, "bf16", nq, nk, Hq, Hkv, 64, pad=0)
    assert torch.equal(a, b)


def test_many_sequences(cuda_lib):
    g = torch.Generator().manual_seed(8)
    nq = torch.randint(0, 4, (2300,), generator=g).tolist()
    nk = [n + int(x) for n, x in zip(nq, torch.randint(0, 40, (2300,), generator=g))]
    run(cuda_lib, "f16", nq, nk, 4, 2, 64, seed=8)


def test_bad_pages_are_reported_and_skipped(cuda_lib):
    sa = cuda_lib
    for dt in ("bf16", "f32"):
        q, k, _, qs, ks = packed.make(dt, [40, 9], [64, 30], 4, 2, 64, seed=9)
        lay = Layout([64, 30], [40, 9], 16, seed=9)
        before = pool_of(lay, 2)
        lost = lay.table[0, 1].item()
        lay.table[0, 1], lay.table[1, 0] = lay.pages, -1
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = sa.attn_weights_packed(q.to(DEV), k.to(DEV), before.to(DEV), lay.table.to(DEV), packed.starts(qs),
                                     packed.starts(ks), err_word=err).cpu()
        assert int(err) == sa.ERRBIT_PAGE
        assert torch.equal(got[lost], before[lost])
        want = before.double()
        good = Layout([64, 30], [40, 9], 16, seed=9)
        for b, (w, _) in enumerate(ev.weights_packed(q, k, qs, ks)):
            ev.put_weights(want, good.table[b], w, [40, 9][b])
        kept = [int(lay.table[0, i]) for i in (0, 2, 3)] + [int(lay.table[1, 1])]
        assert torch.allclose(got[kept].double(), want[kept], rtol=1e-3)
        # a table shorter than the context
        err.zero_()
        sa.attn_weights_packed(q.to(DEV), k.to(DEV), before.to(DEV), good.table[:, :3].contiguous().to(DEV),
                               packed.starts(qs), packed.starts(ks), err_word=err)
        assert int(err) == sa.ERRBIT_PAGE


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_prefix_that_sequences_share(cuda_lib, dt):
    """Weights added to the tokens of a page of two sequences come from both; weights that are
    set there are those of either."""
    sa, D, Hkv, g, pt = cuda_lib, 64, 2, 3, 16
    nq, nk, common = [20, 130], [52, 162], 32
    q, k, _, qs, ks = packed.make(dt, nq, nk, Hkv * g, Hkv, D, seed=14, pad=0)
    k[ks[1]:ks[1] + common] = k[:common]
    lay = Layout(nk, nq, pt, seed=14)
    lay.table[1, :common // pt] = lay.table[0, :common // pt]
    ws = ev.weights_packed(q, k, qs, ks)
    before = pool_of(lay, Hkv, 14)
    page, slot = ev.token_places(lay.table[0], common, pt)
    for accumulate in (True, False):
        got = sa.attn_weights_packed(q.to(DEV), k.to(DEV), before.to(DEV), lay.table.to(DEV), packed.starts(qs),
                                     packed.starts(ks), accumulate=accumulate).cpu()
        have = got[page, :, slot].double()
        parts = [w[:, :common].T for w, _ in ws]
        rel = [rel_bound(D, m, n * g) for (_, m), n in zip(ws, nq)]
        if accumulate:                                      # (two additions, in either order)
            want = before[page, :, slot].double() + parts[0] + parts[1]
            tol = parts[0] * rel[0] + parts[1] * rel[1] + want.abs() * 2.0 ** -23
            assert ((have - want).abs() <= tol).all()
        else:
            near = [(have - w).abs() <= w * (r + 2.0 ** -24) + 1e-30 for w, r in zip(parts, rel)]
            assert (near[0] | near[1]).all()
        for b in range(2):                                  # their own tokens
            p, s = ev.token_places(lay.table[b], nk[b], pt)
            w = ws[b][0][:, common:].T
            have = got[p, :, s][common:].double()
            old = before[p, :, s][common:].double() if accumulate else torch.zeros_like(w)
            old[len(old) - nq[b]:] = 0
            assert ((have - old - w).abs() <= w * rel[b] + (old + w) * 2.0 ** -24 + 1e-30).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_malformed_starts_write_nothing(cuda_lib, dt):
    sa = cuda_lib
    q, k, _, qs, ks = packed.make(dt, [40, 9], [64, 30], 4, 2, 64, seed=9, pad=0)
    lay = Layout([64, 30], [40, 9], 16, seed=9)
    for bad_q, bad_k in (([0, 50, 49], ks), (qs, [0, 64, 95]), ([-1, 40, 49], ks), (qs, [5, 2, 94])):
        before = pool_of(lay, 2).to(DEV)
        got, err = before.clone(), torch.zeros(1, dtype=torch.int32, device=DEV)
        sa.attn_weights_packed(q.to(DEV), k.to(DEV), got, lay.table.to(DEV), packed.starts(bad_q), packed.starts(bad_k),
                               err_word=err)
        assert int(err) == sa.ERRBIT_SEQ and torch.equal(got, before)


@pytest.mark.parametrize("accumulate", [True, False])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_malformed_starts_of_many_sequences_write_nothing(cuda_lib, dt, accumulate):
    """A bad start anywhere among more sequences than a launch takes: none of them is written."""
    sa, B = cuda_lib, 2600
    nq, nk = [1, 2] * (B // 2), [3, 2] * (B // 2)
    q, k, _, qs, ks = packed.make(dt, nq, nk, 4, 2, 64, seed=13, pad=0)
    lay = Layout(nk, nq, 16, seed=13)
    t, before = lay.table.to(DEV), pool_of(lay, 2).to(DEV)
    q, k, ws = q.to(DEV), k.to(DEV), ev.weights_packed(q, k, qs, ks)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for at, by in ((B, 1), (1500, 50), (3, -40), (2047, 20)):
        for which in (0, 1):
            bad = [list(qs), list(ks)]
            bad[which][at] += by
            got = before.clone()
            err.zero_()
            sa.attn_weights_packed(q, k, got, t, packed.starts(bad[0]), packed.starts(bad[1]), accumulate=accumulate, err_word=err)
            assert int(err) == sa.ERRBIT_SEQ and torch.equal(got, before), (at, by, which)
    got = before.clone()
    err.zero_()
    sa.attn_weights_packed(q, k, got, t, packed.starts(qs), packed.starts(ks), accumulate=accumulate, err_word=err)
    assert int(err) == 0
    check(got, before.cpu(), lay, ws, nq if accumulate else nk, 64, [2 * n for n in nq])


def test_captured_and_on_two_streams(cuda_lib):
    sa, nq, nk = cuda_lib, [300, 64], [500, 640]
    q, k, _, qs, ks = packed.make("bf16", nq, nk, 8, 2, 128, seed=10)
    lay = Layout(nk, nq, 16, seed=10)
    q, k, t, qs, ks = q.to(DEV), k.to(DEV), lay.table.to(DEV), packed.starts(qs), packed.starts(ks)
    want = sa.attn_weights_packed(q, k, pool_of(lay, 2).to(DEV), t, qs, ks, accumulate=False)
    pools, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        pools.append(pool_of(lay, 2).to(DEV))
        s.wait_stream(torch.cuda.current_stream())
        sa.attn_weights_packed(q, k, pools[-1], t, qs, ks, accumulate=False, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(p, want) for p in pools)
    for p in pools:
        p.zero_()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            sa.attn_weights_packed(q, k, p, t, qs, ks, accumulate=False)
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    page, slot = ev.token_places(lay.table[0], nk[0], 16)
    for p in pools:
        assert torch.equal(p.cpu()[page, :, slot], want.cpu()[page, :, slot])


def test_workspace_of_the_callers_and_nothing_to_do(cuda_lib):
    sa = cuda_lib
    q, k, _, qs, ks = packed.make("bf16", [40], [64], 4, 2, 64, pad=0)
    lay = Layout([64], [40], 16)
    p, t = pool_of(lay, 2).to(DEV), lay.table.to(DEV)
    small = torch.empty(256, dtype=torch.uint8, device=DEV)
    with pytest.raises(sa.SAError, match="workspace"):
        sa.attn_weights_packed(q.to(DEV), k.to(DEV), p, t, packed.starts(qs), packed.starts(ks), workspace=small)
    big = torch.full((8 << 20,), 255, dtype=torch.uint8, device=DEV)
    a = sa.attn_weights_packed(q.to(DEV), k.to(DEV), p.clone(), t, packed.starts(qs), packed.starts(ks), workspace=big)
    assert torch.equal(a, sa.attn_weights_packed(q.to(DEV), k.to(DEV), p.clone(), t, packed.starts(qs), packed.starts(ks)))
    b = sa.attn_weights_packed(q[:0].to(DEV), k.to(DEV), p.clone(), t, packed.starts([0, 0]), packed.starts(ks))
    assert torch.equal(b, p)


def test_refusals(cuda_lib):
    sa = cuda_lib
    q, k = torch.randn(40, 4, 64).bfloat16().to(DEV), torch.randn(40, 2, 64).bfloat16().to(DEV)
    p, t, s = sa.new_weight_pool(6, 2, 16), torch.zeros(1, 4, dtype=torch.int32, device=DEV), packed.starts([0, 40])
    for bad in (dict(q=q.float()), dict(weights=p.half()), dict(block_table=t.long()), dict(q_start=s.long()),
                dict(q=q.cpu())):
        with pytest.raises(TypeError):
            sa.attn_weights_packed(**{**dict(q=q, k=k, weights=p, block_table=t, q_start=s), **bad})
    for bad in (dict(weights=sa.new_weight_pool(6, 3, 16)), dict(weights=p[0]), dict(block_table=t[0]), dict(k=k[:39]),
                dict(q=q.transpose(1, 2)), dict(k=k[..., :32]), dict(block_table=t.expand(2, 4).contiguous())):
        with pytest.raises(ValueError):
            sa.attn_weights_packed(**{**dict(q=q, k=k, weights=p, block_table=t, q_start=s), **bad})
    for bad in (dict(scale=math.nan), dict(q=q[:, :3])):
        with pytest.raises(sa.SAError):
            sa.attn_weights_packed(**{**dict(q=q, k=k, weights=p, block_table=t, q_start=s), **bad})


# ---- a decode step -----------------------------------------------------------------------------


def elements(lay, Hkv, D, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(lay.pages, Hkv, lay.pt, D, generator=g).to(DT[dt]) for _ in range(2)]


def keys_of(lay, pool, b, D):
    """[Hkv, n, D] of a sequence, 64 bits."""
    n = lay.ctx[b]
    if pool.dtype == torch.uint8:
        return torch.stack([fp8.values(lay, pool, b, h, D) for h in range(pool.shape[1])])
    page, slot = ev.token_places(lay.table[b], n, lay.pt)
    return pool[page, :, slot].transpose(0, 1).double()


def decode_case(sa, ctx, pt, Hkv, g, D, dt, quantised, seed=1, scale=0.0):
    lay = Layout(ctx, [1] * len(ctx), pt, seed=seed)
    pools = fp8.fill(lay, Hkv, D, seed) if quantised else elements(lay, Hkv, D, dt, seed)
    q = torch.randn(len(ctx), Hkv * g, D, generator=torch.Generator().manual_seed(seed + 1)).to(DT[dt])
    table, ctx_t, _ = lay.gpu()
    before = pool_of(lay, Hkv, seed)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    w = before.to(DEV)
    kp, vp = (p.to(DEV) for p in pools)
    y = sa.paged_attn_decode(q.to(DEV), kp, vp, table, ctx_t, weights=w, scale=scale, err_word=err)
    assert int(err) == 0
    assert torch.equal(y, sa.paged_attn_decode(q.to(DEV), kp, vp, table, ctx_t, scale=scale))
    s = scale or 1 / math.sqrt(D)
    ws = [ev.weights_decode(q[b], keys_of(lay, pools[0], b, D), s) for b in range(len(ctx))]
    check(w, before, lay, ws, [1] * len(ctx), D, [g] * len(ctx))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("ctx,pt,Hkv,g,D", [
    ([1], 16, 1, 1, 128), ([16], 16, 2, 4, 128), ([17, 1, 300, 15], 16, 2, 4, 128), ([33, 500], 32, 3, 8, 64),
    ([1000, 3, 64, 65], 64, 1, 16, 64), ([700, 90], 16, 2, 16, 128), ([257, 31], 16, 2, 6, 256), ([129], 48, 1, 32, 128),
    ([400, 2], 16, 1, 17, 256), ([5000, 1, 2, 3], 16, 8, 4, 128), ([90] * 33, 16, 1, 2, 64)])
def test_decode_over_quantised_pages(cuda_lib, dt, ctx, pt, Hkv, g, D):
    decode_case(cuda_lib, ctx, pt, Hkv, g, D, dt, True)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("ctx,pt,Hkv,g,D", [
    ([1], 16, 1, 1, 128), ([17, 1, 300, 15], 16, 2, 4, 128), ([33, 500], 5, 3, 8, 64), ([700, 90], 16, 2, 16, 128),
    ([257, 31], 1, 2, 6, 256), ([129, 5], 48, 1, 32, 80), ([5000, 1, 2, 3], 16, 8, 4, 128), ([90] * 33, 16, 1, 2, 64)])
def test_decode_over_pages_of_elements(cuda_lib, dt, ctx, pt, Hkv, g, D):
    decode_case(cuda_lib, ctx, pt, Hkv, g, D, dt, False)


def test_decode_long_contexts(cuda_lib):
    decode_case(cuda_lib, [30000, 40], 16, 2, 4, 128, "bf16", True, seed=4)
    decode_case(cuda_lib, [30000, 40], 16, 1, 4, 64, "f16", False, seed=4)
    decode_case(cuda_lib, [9000, 40], 16, 2, 2, 64, "bf16", True, seed=5, scale=0.9)


@pytest.mark.parametrize("quantised", [True, False])
def test_decode_steps_captured(cuda_lib, quantised):
    """New tokens written and counted step by step: one graph, replayed."""
    sa, Hkv, g, D, pt = cuda_lib, 2, 4, 64, 16
    total = [40, 7]
    lay = Layout(total, [1, 1], pt, seed=6)
    lay.ctx = [36, 3]
    pools = [p.to(DEV) for p in (fp8.fill(lay, Hkv, D, 6) if quantised else elements(lay, Hkv, D, "bf16", 6))]
    table, ctx = lay.table.to(DEV), torch.tensor(lay.ctx, dtype=torch.int32, device=DEV)
    w = pool_of(lay, Hkv, 6).to(DEV)
    q, k, v = (torch.zeros(2, H, D, dtype=torch.bfloat16, device=DEV) for H in (Hkv * g, Hkv, Hkv))
    gen = torch.Generator().manual_seed(7)

    def step():
        return sa.paged_attn_decode(q, *pools, table, ctx, k_new=k, v_new=v, weights=w)

    ctx += 1
    keep = w.clone(), [p.clone() for p in pools]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    w.copy_(keep[0])
    for p, o in zip(pools, keep[1]):
        p.copy_(o)
    ctx -= 1
    for _ in range(4):
        ctx += 1
        lay.ctx = ctx.tolist()
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=gen).bfloat16())
        before = w.cpu()
        graph.replay()
        torch.cuda.synchronize()
        kc = pools[0].cpu()
        ws = [ev.weights_decode(q[b].cpu(), keys_of(lay, kc, b, D), 1 / math.sqrt(D)) for b in range(2)]
        check(w, before, lay, ws, [1, 1], D, [g, g])


def test_decode_of_bad_contexts_and_pages(cuda_lib):
    sa, Hkv, D, pt = cuda_lib, 2, 64, 16
    for quantised in (True, False):
        lay = Layout([40, 40, 40, 40], [1] * 4, pt, seed=9)
        pools = [p.to(DEV) for p in (fp8.fill(lay, Hkv, D, 9) if quantised else elements(lay, Hkv, D, "bf16", 9))]
        q = torch.randn(4, 4, D, generator=torch.Generator().manual_seed(9)).bfloat16()
        lay.table[3, 1] = lay.pages + 5
        ctx = torch.tensor([0, 40, 1 << 20, 40], dtype=torch.int32, device=DEV)
        before = pool_of(lay, Hkv, 9)
        w, err = before.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
        sa.paged_attn_decode(q.to(DEV), *pools, lay.table.to(DEV), ctx, weights=w, err_word=err)
        assert int(err) == sa.ERRBIT_PAGE
        got = w.cpu()
        kc = keys_of(lay, pools[0].cpu(), 1, D)
        want = before.double()
        ev.put_weights(want, lay.table[1], ev.weights_decode(q[1], kc, D ** -0.5)[0], 1)
        at = lay.table[1, :3].long()
        assert torch.allclose(got[at].double(), want[at], rtol=1e-4)
        for b in (0, 2):
            at = lay.table[b, :3].long()
            assert torch.equal(got[at], before[at])
        # sequence 3: the softmax over the tokens of its good pages
        place = [int(lay.table[3, 0])] * 16 + [int(lay.table[3, 2])] * 8
        two = Layout([24], [1], pt)
        two.table = torch.tensor([[place[0], place[16]]], dtype=torch.int32)
        two.pages = lay.pages
        want = before.double()
        wq = ev.weights_decode(q[3], keys_of(two, pools[0].cpu(), 0, D), D ** -0.5)[0]
        ev.put_weights(want, two.table[0], wq, 1)
        assert torch.allclose(got[two.table[0].long()].double(), want[two.table[0].long()], rtol=1e-4)


def test_decode_nan_and_shared_pages(cuda_lib):
    sa, D, pt = cuda_lib, 64, 16
    for quantised in (True, False):
        lay = Layout([20, 20], [1, 1], pt, seed=11)
        lay.table[1] = lay.table[0]                         # one context of both: added twice, set by one
        pools = [p.to(DEV) for p in (fp8.fill(lay, 1, D, 9) if quantised else elements(lay, 1, D, "bf16", 9))]
        q = torch.randn(2, 4, D, generator=torch.Generator().manual_seed(3)).bfloat16()
        w = torch.zeros(lay.pages, 1, pt, device=DEV)
        sa.paged_attn_decode(q.to(DEV), *pools, lay.table.to(DEV), lay.ctx_t.to(DEV), weights=w)
        page, slot = ev.token_places(lay.table[0], 20, pt)
        both = sum(ev.weights_decode(q[b], keys_of(lay, pools[0].cpu(), 0, D), D ** -0.5)[0][0] for b in range(2))
        assert torch.allclose(w.cpu()[page, 0, slot][:19].double(), both[:19], rtol=1e-4)
        q[0, 2, 5] = math.nan
        w.zero_()
        one = Layout([20], [1], pt)
        one.table = lay.table[:1]
        sa.paged_attn_decode(q[:1].to(DEV), *pools, one.table.to(DEV), one.ctx_t.to(DEV), weights=w)
        assert torch.isnan(w.cpu()[page, 0, slot]).all()


# contexts of one partial, of a few and of many (16 tokens to a warp where there are few)
@pytest.mark.parametrize("n", [9, 20, 100, 127, 150, 1200, 9000])
@pytest.mark.parametrize("dt,D", [("bf16", 64), ("f16", 128), ("f32", 64), ("f32", 72)])
def test_a_nan_reaches_y_and_the_weights_alike(cuda_lib, dt, D, n):
    """A query with a NaN, and a key with one: the output and the weights of what sees it are
    NaN and the others' are not, however many parts a context was split into."""
    sa, Hkv, g = cuda_lib, 2, 3
    lay = Layout([n, 40], [1, 1], 16, seed=n)
    kp, vp = elements(lay, Hkv, D, dt, n)
    q = torch.randn(2, Hkv * g, D, generator=torch.Generator().manual_seed(n)).to(DT[dt])
    table, ctx, _ = lay.gpu()
    page, slot = ev.token_places(lay.table[0], n, 16)
    before = pool_of(lay, Hkv, n)

    def both(q, kp):
        w = before.to(DEV)
        y = sa.paged_attn_decode(q.to(DEV), kp.to(DEV), vp.to(DEV), table, ctx, weights=w)
        plain = sa.paged_attn_decode(q.to(DEV), kp.to(DEV), vp.to(DEV), table, ctx)
        assert torch.equal(torch.isnan(y), torch.isnan(plain)) and torch.equal(torch.nan_to_num(y), torch.nan_to_num(plain))
        return torch.isnan(y.cpu()), torch.isnan(w.cpu())

    bad = q.clone()
    bad[0, 1, 7] = math.nan                                 # a head of KV head 0
    ny, nw = both(bad, kp)
    assert ny[0, 1].all() and ny.sum() == D
    assert nw[page, 0, slot].all() and nw.sum() == n
    for t in sorted({0, n // 2, n - 1}):                    # a key of KV head 1
        kb = kp.clone()
        kb[page[t], 1, slot[t], 3] = math.nan
        ny, nw = both(q, kb)
        assert ny[0, g:].all() and ny.sum() == g * D, t
        assert nw[page, 1, slot].all() and nw.sum() == n, t
    kb = kp.clone()                                         # a run of keys
    kb[page[n // 3:2 * n // 3 + 1], 1, slot[n // 3:2 * n // 3 + 1], 3] = math.nan
    ny, nw = both(q, kb)
    assert ny[0, g:].all() and ny.sum() == g * D
    assert nw[page, 1, slot].all() and nw.sum() == n


def y_of(q, k, v, scale):
    """A decode's y [Hq, D] of one sequence in 64 bits, and sum p |v|: q [Hq, D], k and v [Hkv, n, D]."""
    qq = q.double().view(k.shape[0], -1, q.shape[-1])
    p = ev._softmax(qq @ k.double().transpose(1, 2) * scale)
    return (p @ v.double()).view(q.shape), (p @ v.double().abs()).view(q.shape)


@pytest.mark.parametrize("n", [9, 100, 1200])
@pytest.mark.parametrize("dt,D", [("bf16", 64), ("f16", 80), ("f32", 64), ("f32", 256)])
def test_a_decode_of_keys_with_infinite_scores(cuda_lib, dt, D, n):
    """Keys whose score is -inf, the first of every thread's among them, have no part in y and
    receive 0.  Off by a probability's bound (its rounding to 16 bits added) times sum p |v|,
    and half a step of y."""
    sa, Hkv, g = cuda_lib, 2, 2
    lay = Layout([n, 5], [1, 1], 16, seed=n)
    kp, vp = elements(lay, Hkv, D, dt, n)
    q = torch.randn(2, Hkv * g, D, generator=torch.Generator().manual_seed(n)).to(DT[dt])
    q[:, :, 2] = q[:, :, 2].abs() + 0.1
    page, slot = ev.token_places(lay.table[0], n, 16)
    for t in (0, 1, 2, 3, 5, n // 2, n - 1):
        kp[page[t], :, slot[t], 2] = -math.inf
    before = pool_of(lay, Hkv, n)
    w = before.to(DEV)
    table, ctx, _ = lay.gpu()
    y = sa.paged_attn_decode(q.to(DEV), kp.to(DEV), vp.to(DEV), table, ctx, weights=w).cpu()
    ws, s = [], 1 / math.sqrt(D)
    for b in range(2):
        k, v = keys_of(lay, kp, b, D), keys_of(lay, vp, b, D)
        low = torch.nan_to_num(k, neginf=0.0)               # (of finite magnitudes, the bound's)
        ws.append((ev.weights_decode(q[b], k, s)[0], ev.weights_decode(q[b], low, s)[1]))
        want, mag = y_of(q[b], k, v, s)
        fi = torch.finfo(y.dtype)
        rel = rel_bound(D, ws[b][1], 1) + lay.ctx[b] * 2.0 ** -22 + (0 if dt == "f32" else fi.eps / 2)
        assert ((y[b].double() - want).abs() <= rel * mag + (want.abs() + rel * mag) * fi.eps / 2 + 1e-30).all()
    check(w, before, lay, ws, [1, 1], D, [g, g])


def test_decode_refusals(cuda_lib):
    sa, D = cuda_lib, 64
    kp, vp = sa.new_fp8_pool(4, 2, 16, D), sa.new_fp8_pool(4, 2, 16, D)
    q, t = torch.zeros(1, 4, D, dtype=torch.bfloat16, device=DEV), torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    c, w = torch.ones(1, dtype=torch.int32, device=DEV), sa.new_weight_pool(4, 2, 16)
    with pytest.raises(TypeError):
        sa.paged_attn_decode(q, kp, vp, t, c, weights=w.half())
    for bad in (sa.new_weight_pool(5, 2, 16), sa.new_weight_pool(4, 1, 16), sa.new_weight_pool(4, 2, 32)):
        with pytest.raises(ValueError):
            sa.paged_attn_decode(q, kp, vp, t, c, weights=bad)
    small = torch.empty(512, dtype=torch.uint8, device=DEV)
    with pytest.raises(sa.SAError, match="workspace"):
        sa.paged_attn_decode(q, kp, vp, t, c, weights=w, workspace=small)
    need = sa.paged_attn_decode_weights_workspace(q, kp, vp, t, c)
    assert need > sa.paged_attn_decode_workspace(q, kp, vp, t, c)
    ws = sa.new_workspace(need, DEV)
    sa.paged_attn_decode(q, kp, vp, t, c, weights=w, workspace=ws)
    e = torch.zeros(4, 2, 16, D, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(sa.SAError):
        sa.paged_attn_decode(q, e, torch.zeros_like(e), t, c, weights=w, options=sa.OPT_ROW_COPIES)
