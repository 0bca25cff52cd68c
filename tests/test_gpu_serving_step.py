"""The serving-step operators in a run, as a server uses them: rotary positions, the
page write, packed prefill of prompts and of chunks over read-back contexts, and a
captured decode step over FP8 pages.  Every stage is compared with its 64-bit form on
the stage's own inputs, with that operator's tolerance (in its own test file); a
quantised key is off by half a step of its code (2^-4 of it, or 2^-10 of the row's
power of two, which is below 1/224 of its largest element) besides the rotation.

After it, what only a large cache reaches: offsets past 2^31, more sequences than a
launch takes."""
import pytest
import torch

import test_gpu_packed as packed
import test_gpu_paged_fp8 as decode
import test_gpu_rope as rope_test
from oracle import serving as orc
from test_gpu_paged_kv import Layout

pytestmark = pytest.mark.gpu
DEV = "cuda"


def near_quantised(got, want, mag):
    turn = mag * 2.0 ** -21
    top = (want.abs() + turn).amax(-1, keepdim=True)
    step = torch.maximum((want.abs() + turn) * 2.0 ** -4, top * (2.0 ** -10 / 224))
    assert ((got - want).abs() <= turn + step).all()


@pytest.mark.parametrize("Hq,Hkv,D,spec", [(8, 2, 128, dict(interleaved=True)),
                                           (6, 2, 64, dict(scaling="ramp", factor=16.0, original_len=4096, mscale=1.27))])
def test_prompts_chunks_and_decode_steps(cuda_lib, Hq, Hkv, D, spec):
    sa = cuda_lib
    first, more, steps, pt = [70, 5, 130], [30, 64, 1], 3, 16
    total = [a + b + steps for a, b in zip(first, more)]
    B = len(total)
    lay = Layout(total, total, pt, seed=D)
    table = lay.table.to(DEV)
    pools = [sa.new_fp8_pool(lay.pages, Hkv, pt, D) for _ in range(2)]
    g = torch.Generator().manual_seed(Hq)
    qs, ks, vs = ([torch.randn(n, H, D, generator=g).bfloat16() for n in total] for H in (Hq, Hkv, Hkv))
    rope = sa.rope_table(D, **spec)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def stage(at, n):
        """Rows at .. at + n of every sequence: rotated, written, and the pools compared."""
        q, k, v = (torch.cat([x[b][at[b]:at[b] + n[b]] for b in range(B)]).to(DEV) for x in (qs, ks, vs))
        pos = torch.cat([torch.arange(at[b], at[b] + n[b]) for b in range(B)])
        yq, yk = sa.rotary_embed(q, k, pos.to(DEV), rope)
        for x, y in ((q, yq), (k, yk)):
            want, mag = rope_test.oracle(x, pos[:, None], D, spec)
            rope_test.check(y, want, mag)
        lay.ctx = [a + c for a, c in zip(at, n)]
        starts = [0]
        for c in n:
            starts.append(starts[-1] + c)
        ctx = torch.tensor(lay.ctx, dtype=torch.int32, device=DEV)
        sa.paged_kv_write(k, v, *pools, table, ctx, packed.starts(starts), rope=rope, err_word=err)
        for b in range(B):
            want, mag = rope_test.oracle(ks[b][:lay.ctx[b]], torch.arange(lay.ctx[b])[:, None], D, spec)
            for h in range(Hkv):
                near_quantised(decode.values(lay, pools[0].cpu(), b, h, D), want[:, h], mag[:, h])
                x = vs[b][:lay.ctx[b], h].double()
                near_quantised(decode.values(lay, pools[1].cpu(), b, h, D), x, torch.zeros_like(x))
        return yq, yk, v, starts, ctx

    # prompts: attention over the rows themselves
    yq, yk, v, s, _ = stage([0] * B, first)
    y = sa.attn_prefill_packed(yq, yk, v, packed.starts(s), err_word=err)
    packed.check(y, yq.cpu(), yk.cpu(), v.cpu(), s, s, what="prompts")

    # chunks: attention over the contexts read back from their pages
    yq, _, _, s, ctx = stage(first, more)
    c = [0]
    for n in lay.ctx:
        c.append(c[-1] + n)
    kc, vc = sa.paged_kv_read(*pools, table, ctx, packed.starts(c), total=c[-1], head_dim=D, err_word=err)
    for b in range(B):
        for h in range(Hkv):
            for got, pool in ((kc, pools[0]), (vc, pools[1])):
                assert torch.equal(got[c[b]:c[b + 1], h].cpu(), decode.values(lay, pool.cpu(), b, h, D).bfloat16())
    y = sa.attn_prefill_packed(yq, kc, vc, packed.starts(s), packed.starts(c), err_word=err)
    packed.check(y, yq.cpu(), kc.cpu(), vc.cpu(), s, c, what="chunks")

    # decode steps: one graph, replayed with the next tokens and longer contexts
    q1, k1, v1 = (torch.zeros(B, H, D, dtype=torch.bfloat16, device=DEV) for H in (Hq, Hkv, Hkv))

    def step():
        yq, _ = sa.rotary_embed(q1, None, ctx - 1, rope)
        sa.paged_kv_write(k1, v1, *pools, table, ctx, rope=rope, err_word=err)
        return yq, sa.paged_attn_decode(yq, *pools, table, ctx, err_word=err)

    graph = None
    for i in range(steps):
        at = list(lay.ctx)
        lay.ctx = [n + 1 for n in at]
        ctx.copy_(torch.tensor(lay.ctx, dtype=torch.int32))
        for buf, x in ((q1, qs), (k1, ks), (v1, vs)):
            buf.copy_(torch.stack([x[b][at[b]] for b in range(B)]))
        eager = step()
        torch.cuda.synchronize()
        if graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], eager[0]) and torch.equal(out[1], eager[1])
        decode.check(out[1][:, :, None], out[0][:, :, None], lay, [p.cpu() for p in pools])
    assert int(err) == 0


def test_more_sequences_than_a_launch_takes(cuda_lib):
    g = torch.Generator().manual_seed(1)
    n = torch.randint(0, 4, (2300,), generator=g).tolist()
    q, k, v, qs, _ = packed.make("bf16", n, n, 2, 1, 64, seed=2)
    y = torch.full(q.shape, 9.0, dtype=q.dtype, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    cuda_lib.attn_prefill_packed(q.to(DEV), k.to(DEV), v.to(DEV), packed.starts(qs), y=y, err_word=err)
    packed.check(y, q, k, v, qs, qs)
    assert int(err) == 0 and (y[qs[-1]:] == 9.0).all()
    lay = Layout([1 + c % 40 for c in range(2300)], [1] * 2300, 16, seed=3)
    pools = decode.fill(lay, 1, 64, 4)
    q = torch.randn(2300, 4, 1, 64, generator=g).half()
    table, ctx, _ = lay.gpu()
    y = cuda_lib.paged_attn_decode(q.to(DEV), pools[0].to(DEV), pools[1].to(DEV), table, ctx, err_word=err)
    decode.check(y, q, lay, pools, seqs=range(0, 2300, 37))
    assert int(err) == 0


def test_heads_that_share_one_row(cuda_lib):
    """K and V of one head, expanded: stride 0."""
    q, k, v, qs, ks = packed.make("bf16", [40, 3], [90, 3], 4, 1, 64, pad=0)
    x = cuda_lib.attn_prefill_packed(q.to(DEV), k.to(DEV).expand(-1, 4, -1), v.to(DEV).expand(-1, 4, -1),
                                     packed.starts(qs), packed.starts(ks))
    packed.check(x, q, k.expand(-1, 4, -1), v.expand(-1, 4, -1), qs, ks)


def test_rows_further_apart_than_32_bits_reach(cuda_lib):
    sa, g = cuda_lib, torch.Generator().manual_seed(6)
    far = [torch.empty((1 << 31) + 4096, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    k, v = (f.as_strided((3, 2, 64), (1 << 30, 64, 1)) for f in far)
    for x in (k, v):
        x.copy_(torch.randn(3, 2, 64, generator=g).bfloat16())
    q = torch.randn(3, 4, 64, generator=g).bfloat16()
    s = packed.starts([0, 3])
    packed.check(sa.attn_prefill_packed(q.to(DEV), k, v, s), q, k.cpu(), v.cpu(), [0, 3], [0, 3])
    pool = [sa.new_fp8_pool(2, 2, 16, 64) for _ in range(2)]
    near = [sa.new_fp8_pool(2, 2, 16, 64) for _ in range(2)]
    table, ctx = torch.tensor([[1]], dtype=torch.int32, device=DEV), torch.tensor([3], dtype=torch.int32, device=DEV)
    sa.paged_kv_write(k, v, *pool, table, ctx, s)
    sa.paged_kv_write(k.contiguous(), v.contiguous(), *near, table, ctx, s)
    assert torch.equal(pool[0], near[0]) and torch.equal(pool[1], near[1])
    want = v.clone()
    rope = sa.rope_table(64)
    pos = torch.arange(3, device=DEV)
    a, b = sa.rotary_embed(k.contiguous(), v.contiguous(), pos, rope)
    sa.rotary_embed(k, v, pos, rope, q_out=k, k_out=v)
    assert torch.equal(k, a) and torch.equal(v, b)
    sa.paged_kv_read(*pool, table, ctx, s, k=k, v=v)
    near_k, near_v = sa.paged_kv_read(*pool, table, ctx, s, total=3, head_dim=64)
    assert torch.equal(k, near_k) and torch.equal(v, near_v)
    near_quantised(v.cpu().double(), want.cpu().double(), torch.zeros(3, 2, 64, dtype=torch.float64))


@pytest.mark.parametrize("fp8", [True, False])
def test_pages_past_2_31_bytes(cuda_lib, fp8):
    sa, Hkv, D, pt, n, pages = cuda_lib, 8, 128, 16, 40, 140000
    shape = (pages, Hkv, pt * (D + 1)) if fp8 else (pages, Hkv, pt, D)
    pools = [torch.empty(shape, dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV) for _ in range(2)]
    table = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32, device=DEV)
    near = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    ctx, s = torch.tensor([n], dtype=torch.int32, device=DEV), packed.starts([0, n])
    g = torch.Generator().manual_seed(8)
    k, v = (torch.randn(n, Hkv, D, generator=g).bfloat16().to(DEV) for _ in range(2))
    for p in pools:
        p[pages - 3:] = 0
    small = [torch.zeros_like(p[:3]) for p in pools]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sa.paged_kv_write(k, v, *pools, table, ctx, s, err_word=err)
    sa.paged_kv_write(k, v, *small, near, ctx, s)
    assert all(torch.equal(p[pages - 3:], x) for p, x in zip(pools, small))
    got = sa.paged_kv_read(*pools, table, ctx, s, total=n, head_dim=D, err_word=err)
    want = sa.paged_kv_read(*small, near, ctx, s, total=n, head_dim=D)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    q = torch.randn(1, 32, 1, D, generator=g).bfloat16().to(DEV)
    assert torch.equal(sa.paged_attn_decode(q, *pools, table, ctx, err_word=err), sa.paged_attn_decode(q, *small, near, ctx))
    assert int(err) == 0


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("B", [32, 33, 300])
def test_many_sequences_of_very_different_lengths(cuda_lib, B, causal):
    """Chunks of 0 to 400 tokens after contexts of up to 1,500: the two ways in which the items
    are put in order."""
    g = torch.Generator().manual_seed(B)
    nq = (2.0 ** (8.7 * torch.rand(B, generator=g)) - 1).int().tolist()
    past = (2.0 ** (10.6 * torch.rand(B, generator=g)) - 1).int().tolist()
    nk = [a + b for a, b in zip(nq, past)]
    nk[3] = 0                                              # queries without a key
    q, k, v, qs, ks = packed.make("f16", nq, nk, 3, 1, 64, seed=B)
    y = torch.full(q.shape, 9.0, dtype=q.dtype, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    cuda_lib.attn_prefill_packed(q.to(DEV), k.to(DEV), v.to(DEV), packed.starts(qs), packed.starts(ks), causal=causal,
                                 y=y, err_word=err)
    assert int(err) == 0 and (y[qs[-1]:] == 9.0).all()
    packed.check(y, q, k, v, qs, ks, causal=causal)
