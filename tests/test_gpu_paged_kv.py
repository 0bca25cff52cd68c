"""GPU parity of paged_kv_write and paged_kv_read: without a rotation every byte
of the pools is the 64-bit quantiser's (x / 2^e is exact, so a code depends on x
alone), and reading back is exact up to the output's one rounding."""
import pytest
import torch

from oracle import serving as orc

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


class Layout:
    """Sequences with contexts `ctx` over shuffled pages, and the rows `new` at their ends."""

    def __init__(self, ctx, new, pt, seed=0, extra=3, cols=1):
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.new, self.pt = ctx, new, pt
        need = [-(-c // pt) for c in ctx]
        self.pages = sum(need) + extra
        perm = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((len(ctx), max(max(need), 1) + cols), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        s = [0]
        for n in new:
            s.append(s[-1] + n)
        self.start = torch.tensor(s, dtype=torch.int32)
        self.ctx_t = torch.tensor(ctx, dtype=torch.int32)

    def gpu(self):
        return self.table.to(DEV), self.ctx_t.to(DEV), self.start.to(DEV)

    def place(self, b, pos):
        return int(self.table[b, pos // self.pt]), pos % self.pt

    def write_rows(self):
        """(row, sequence, position) of the rows that a write places."""
        for b, n in enumerate(self.new):
            for i in range(n):
                yield int(self.start[b]) + i, b, self.ctx[b] - n + i


def rows(shape, dt, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g, dtype=torch.float64)
    x *= torch.exp2(torch.randint(-12, 9, shape[:-1], generator=g).double())[..., None]
    if x.shape[0] > 2:
        x[1] = 0                                   # a row of zeros
        x[2, :, ::3] = 0
    return x.to(DT[dt])


CASES = [  # (contexts, new rows, page tokens, Hkv, D)
    ([1], [1], 16, 1, 64), ([40, 5, 300], [40, 5, 300], 16, 2, 128), ([17, 33, 1, 64], [3, 0, 1, 64], 32, 3, 64),
    ([100, 1000], [70, 513], 64, 4, 256), ([16] * 40, [1] * 40, 16, 8, 128), ([0, 20], [0, 20], 16, 1, 128)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("ctx,new,pt,Hkv,D", CASES)
def test_quantised_bytes(cuda_lib, dt, ctx, new, pt, Hkv, D):
    lay = Layout(ctx, new, pt)
    T = sum(new)
    k, v = rows((T + 2, Hkv, D), dt, 1), rows((T + 2, Hkv, D), dt, 2)
    g = torch.Generator().manual_seed(9)
    pools = [torch.randint(0, 256, (lay.pages, Hkv, pt * (D + 1)), generator=g, dtype=torch.uint8) for _ in range(2)]
    want = [p.clone() for p in pools]
    for x, p in ((k, want[0]), (v, want[1])):
        codes, scales = orc.quantise_rows(x.reshape(-1, D))
        codes, scales = codes.view(T + 2, Hkv, D), scales.view(T + 2, Hkv)
        for r, b, pos in lay.write_rows():
            page, slot = lay.place(b, pos)
            for h in range(Hkv):
                orc.write_row(p, page, h, slot, pt, D, codes[r, h], scales[r, h])
    table, ctx_t, start = lay.gpu()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = [p.to(DEV) for p in pools]
    cuda_lib.paged_kv_write(k.to(DEV), v.to(DEV), *got, table, ctx_t, start, err_word=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    for a, b in zip(got, want):
        assert torch.equal(a.cpu(), b)             # the other bytes stay as they are

    # read the contexts back
    first = Layout(ctx, ctx, pt)
    n = sum(ctx)
    for out in ("bf16", "f16", "f32"):
        ko = torch.full((n + 2, Hkv, D), 7.0, dtype=DT[out], device=DEV)
        vo = ko.clone()
        err.zero_()
        cuda_lib.paged_kv_read(*got, table, ctx_t, first.start.to(DEV), ko, vo, err_word=err)
        torch.cuda.synchronize()
        assert int(err) == 0
        for o, p in ((ko.cpu(), want[0]), (vo.cpu(), want[1])):
            exp = torch.full((n + 2, Hkv, D), 7.0, dtype=torch.float64)
            for b, c in enumerate(ctx):
                for i in range(c):
                    page, slot = lay.place(b, i)
                    for h in range(Hkv):
                        exp[int(first.start[b]) + i, h] = orc.dequantise_rows(*orc.read_row(p, page, h, slot, pt, D))
            exp = exp.to(DT[out])                  # the values are doubles exactly: one rounding
            assert torch.equal(torch.isnan(o), torch.isnan(exp))
            assert torch.equal(o[~torch.isnan(exp)], exp[~torch.isnan(exp)])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,Hkv,pt", [(128, 2, 16), (72, 3, 5), (20, 1, 16), (576, 1, 16), (16, 2, 1)])
def test_plain_pages_are_exact_copies(cuda_lib, dt, D, Hkv, pt):
    ctx, new = [30, 7, 64], [12, 7, 50]
    lay = Layout(ctx, new, pt, seed=2)
    T = sum(new)
    k, v = rows((T, Hkv, D), dt, 3), rows((T, Hkv, D), dt, 4)
    kp = torch.full((lay.pages, Hkv, pt, D), 3.0, dtype=DT[dt], device=DEV)
    vp = kp.clone()
    want = [kp.cpu().clone(), vp.cpu().clone()]
    for x, p in ((k, want[0]), (v, want[1])):
        for r, b, pos in lay.write_rows():
            page, slot = lay.place(b, pos)
            p[page, :, slot] = x[r]
    table, ctx_t, start = lay.gpu()
    cuda_lib.paged_kv_write(k.to(DEV), v.to(DEV), kp, vp, table, ctx_t, start)
    assert torch.equal(kp.cpu(), want[0]) and torch.equal(vp.cpu(), want[1])
    ko, vo = cuda_lib.paged_kv_read(kp, vp, table, ctx_t, Layout(ctx, ctx, pt, seed=2).start.to(DEV),
                                    total=sum(ctx), head_dim=D, dtype=DT[dt])
    at = 0
    for b, c in enumerate(ctx):
        for i in range(c):
            page, slot = lay.place(b, i)
            assert torch.equal(ko[at].cpu(), want[0][page, :, slot])
            assert torch.equal(vo[at].cpu(), want[1][page, :, slot])
            at += 1


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("dt,D,R,inter", [("bf16", 128, 128, False), ("f16", 128, 64, True), ("f32", 64, 64, False),
                                          ("bf16", 256, 32, False), ("f16", 64, 20, True), ("bf16", 128, 100, False)])
def test_rotated_keys(cuda_lib, fp8, dt, D, R, inter):
    """K is rotated at its position, then rounded: an element is off by half a step of
    its format (E4M3: 2^-4 of the value, or half its smallest step in the row's scale)
    and 2^-21 (|u| + |v|) of the rotation; V has no rotation."""
    ctx, new, Hkv, pt = [5000, 77, 4096], [60, 77, 1], 2, 16
    lay = Layout(ctx, new, pt, seed=5)
    T = sum(new)
    k, v = rows((T, Hkv, D), dt, 6), rows((T, Hkv, D), dt, 7)
    pos = torch.zeros(T, dtype=torch.int64)
    for r, b, p in lay.write_rows():
        pos[r] = p
    want, mag = orc.rotate(k, pos[:, None], orc.rope_freqs(R), inter)
    rope = cuda_lib.rope_table(R, interleaved=inter)
    table, ctx_t, start = lay.gpu()
    if fp8:
        pools = [cuda_lib.new_fp8_pool(lay.pages, Hkv, pt, D) for _ in range(2)]
    else:
        pools = [torch.zeros(lay.pages, Hkv, pt, D, dtype=DT[dt], device=DEV) for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    cuda_lib.paged_kv_write(k.to(DEV), v.to(DEV), *pools, table, ctx_t, start, rope=rope, err_word=err)
    assert int(err) == 0
    pools = [p.cpu() for p in pools]
    vc, vs = orc.quantise_rows(v.reshape(-1, D))
    for r, b, p in lay.write_rows():
        page, slot = lay.place(b, p)
        for h in range(Hkv):
            x, m = want[r, h], mag[r, h] * 2.0 ** -21
            if fp8:
                codes, scale = orc.read_row(pools[0], page, h, slot, pt, D)
                e = int(scale) - 127
                top, slack = float(x.abs().max()), float(m.max())
                assert top - slack <= 448 * 2.0 ** e and (top == 0 or top + slack > 224 * 2.0 ** e)
                got = orc.dequantise_rows(codes[None], scale[None])[0]
                half = torch.maximum((x.abs() + m) * 2.0 ** -4, torch.tensor(2.0 ** (e - 10)))
                assert torch.equal(orc.read_row(pools[1], page, h, slot, pt, D)[0], vc.view(T, Hkv, D)[r, h])
            else:
                got = pools[0][page, h, slot].double()
                fi = torch.finfo(DT[dt])
                half = (x.abs() + m) * fi.eps / 2 + fi.smallest_normal * fi.eps
                assert torch.equal(pools[1][page, h, slot], v[r, h])
            assert float(((got - x).abs() - half - m).max()) <= 0


def test_strided_and_misaligned_rows(cuda_lib):
    """K and V as views of a projection's output, and rows that start off 16 bytes."""
    lay = Layout([50, 20], [50, 20], 16)
    table, ctx_t, start = lay.gpu()
    buf = rows((70, 8, 128), "bf16", 8).to(DEV)
    odd = rows((70, 2, 131), "bf16", 8).to(DEV)
    for k, v in ((buf[:, 4:6], buf[:, 6:8]), (odd[:, :, 3:], odd[:, :, 1:129])):
        a = [cuda_lib.new_fp8_pool(lay.pages, 2, 16, 128) for _ in range(2)]
        b = [cuda_lib.new_fp8_pool(lay.pages, 2, 16, 128) for _ in range(2)]
        cuda_lib.paged_kv_write(k, v, *a, table, ctx_t, start)
        cuda_lib.paged_kv_write(k.contiguous(), v.contiguous(), *b, table, ctx_t, start)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        out = torch.zeros(70, 8, 128, dtype=torch.bfloat16, device=DEV)
        cuda_lib.paged_kv_read(*a, table, ctx_t, start, out[:, 1:3], out[:, 5:7])
        ko, vo = cuda_lib.paged_kv_read(*a, table, ctx_t, start, total=70, head_dim=128)
        assert torch.equal(out[:, 1:3], ko) and torch.equal(out[:, 5:7], vo)
        assert not out[:, 3:5].any() and not out[:, 0].any() and not out[:, 7].any()


def test_rows_with_nan_or_infinity_read_as_nan(cuda_lib):
    lay = Layout([4], [4], 16)
    table, ctx_t, start = lay.gpu()
    k = torch.ones(4, 1, 64, dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    k[1, 0, 7], v[2, 0, 63] = float("nan"), float("-inf")
    pools = [cuda_lib.new_fp8_pool(lay.pages, 1, 16, 64) for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    cuda_lib.paged_kv_write(k, v, *pools, table, ctx_t, start, err_word=err)
    assert int(err) == cuda_lib.ERRBIT_NONFINITE
    ko, vo = cuda_lib.paged_kv_read(*pools, table, ctx_t, start, total=4, head_dim=64)
    for x, bad in ((ko, 1), (vo, 2)):
        assert torch.isnan(x[bad]).all()
        assert torch.equal(x[[i for i in range(4) if i != bad]], k[[0, 3, 3]])


@pytest.mark.parametrize("fp8", [True, False])
def test_bad_tables_contexts_and_starts_are_skipped_and_reported(cuda_lib, fp8):
    sa = cuda_lib
    lay = Layout([40, 40, 40, 40], [40, 40, 40, 40], 16)
    k = rows((160, 1, 64), "bf16", 1).to(DEV)
    for what in ("table", "context", "negative", "starts", "short"):
        pools = [sa.new_fp8_pool(lay.pages, 1, 16, 64) if fp8 else
                 torch.zeros(lay.pages, 1, 16, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        table, ctx_t, start = (t.clone() for t in lay.gpu())
        bit = sa.ERRBIT_PAGE
        if what == "table":
            table[1, 1] = 10 ** 9
        elif what == "context":
            ctx_t[1] = 10 ** 6
        elif what == "negative":
            ctx_t[1] = -5
        elif what == "short":
            ctx_t[1] = 39                      # fewer tokens than rows
        else:
            start[2], bit = 2 ** 30, sa.ERRBIT_SEQ
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        sa.paged_kv_write(k, k, *pools, table, ctx_t, start, err_word=err)
        assert int(err) & bit, what
        err.zero_()
        ko, vo = sa.paged_kv_read(*pools, table, ctx_t, start, total=160, head_dim=64, err_word=err)
        assert int(err) & bit, what
        if what != "starts":                   # the other sequences are there
            keep = torch.cat((torch.arange(40), torch.arange(80, 160)))
            want = k if not fp8 else None
            if want is not None:
                assert torch.equal(ko[keep], k[keep]) and torch.equal(vo[keep], k[keep])
            else:
                assert float((ko[keep].double() - k[keep].double()).abs().max()) <= float(k.double().abs().max()) * 2 ** -4


def test_one_row_per_sequence_without_starts(cuda_lib):
    lay = Layout([1, 16, 17, 90], [1, 1, 1, 1], 16)
    table, ctx_t, start = lay.gpu()
    k, v = rows((4, 2, 128), "f16", 1).to(DEV), rows((4, 2, 128), "f16", 2).to(DEV)
    a, b = ([cuda_lib.new_fp8_pool(lay.pages, 2, 16, 128) for _ in range(2)] for _ in range(2))
    cuda_lib.paged_kv_write(k, v, *a, table, ctx_t)
    cuda_lib.paged_kv_write(k, v, *b, table, ctx_t, start)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert a[0].any()


def test_many_sequences_and_empty_ones(cuda_lib):
    """3,001 sequences, most of them empty: the owner of every row is found."""
    new = [0] * 3001
    for b in (0, 1, 31, 32, 33, 1024, 1500, 2999, 3000):
        new[b] = 2
    lay = Layout([max(n, 1) for n in new], new, 16)
    T = sum(new)
    k = rows((T, 1, 64), "bf16", 1).to(DEV)
    pools = [torch.zeros(lay.pages, 1, 16, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    table, ctx_t, start = lay.gpu()
    cuda_lib.paged_kv_write(k, k, *pools, table, ctx_t, start)
    for r, b, pos in lay.write_rows():
        page, slot = lay.place(b, pos)
        assert torch.equal(pools[1][page, 0, slot], k[r, 0])
    ko, _ = cuda_lib.paged_kv_read(*pools, table, ctx_t, start, total=T, head_dim=64)
    assert torch.equal(ko, k)


def test_captured_and_on_another_stream(cuda_lib):
    lay = Layout([70], [70], 16)
    table, ctx_t, start = lay.gpu()
    k = rows((70, 2, 128), "bf16", 1).to(DEV)
    rope = cuda_lib.rope_table(128)
    a, b = ([cuda_lib.new_fp8_pool(lay.pages, 2, 16, 128) for _ in range(2)] for _ in range(2))
    cuda_lib.paged_kv_write(k, k, *a, table, ctx_t, start, rope=rope)
    want = cuda_lib.paged_kv_read(*a, table, ctx_t, start, total=70, head_dim=128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cuda_lib.paged_kv_write(k, k, *b, table, ctx_t, start, rope=rope, stream=s)
    got = cuda_lib.paged_kv_read(*b, table, ctx_t, start, total=70, head_dim=128, stream=s)
    s.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cuda_lib.paged_kv_write(k, k, *b, table, ctx_t, start, rope=rope)
        out = cuda_lib.paged_kv_read(*b, table, ctx_t, start, total=70, head_dim=128)
    k.mul_(-1)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[1], -want[1])


def test_refusals(cuda_lib):
    sa = cuda_lib
    lay = Layout([40], [40], 16)
    table, ctx_t, start = lay.gpu()
    k = torch.zeros(40, 2, 128, dtype=torch.bfloat16, device=DEV)
    pools = [sa.new_fp8_pool(lay.pages, 2, 16, 128) for _ in range(2)]
    w = lambda **kw: sa.paged_kv_write(**dict(dict(k=k, v=k, k_pool=pools[0], v_pool=pools[1], block_table=table,  # noqa: E731
                                                  ctx_len=ctx_t, seq_start=start), **kw))
    for kw in (dict(ctx_len=ctx_t.long()), dict(block_table=table.long()), dict(seq_start=start.long()), dict(v=k.half()),
               dict(rope=3), dict(k=k.double(), v=k.double())):
        with pytest.raises(TypeError):
            w(**kw)
    for kw in (dict(seq_start=None), dict(seq_start=start[:1]), dict(v=k[:, :1]), dict(k_pool=pools[0][..., :-1].contiguous()),
               dict(k=k[:, :1], v=k[:, :1]), dict(k=k.transpose(1, 2), v=k.transpose(1, 2)), dict(block_table=table.expand(2, -1).contiguous())):
        with pytest.raises(ValueError):
            w(**kw)
    for kw in (dict(v_pool=pools[0]), dict(rope=sa.rope_table(256))):
        with pytest.raises(sa.SAError):
            w(**kw)
    with pytest.raises(sa.SAError):            # a page of 8 tokens
        p = [sa.new_fp8_pool(5, 2, 8, 128) for _ in range(2)]
        w(k_pool=p[0], v_pool=p[1])
    with pytest.raises(sa.SAError):            # rows of 96 codes
        x = torch.zeros(40, 2, 96, dtype=torch.bfloat16, device=DEV)
        p = [sa.new_fp8_pool(5, 2, 16, 96) for _ in range(2)]
        w(k=x, v=x, k_pool=p[0], v_pool=p[1])
    with pytest.raises(ValueError):
        sa.paged_kv_read(*pools, table, ctx_t, start)
    with pytest.raises(ValueError):
        sa.paged_kv_read(*pools, table, ctx_t, None, total=40, head_dim=128)
    with pytest.raises(sa.SAError):            # one output for both
        sa.paged_kv_read(*pools, table, ctx_t, start, k, k)


def test_places_past_2_to_the_31_bytes_of_a_page(cuda_lib):
    """Rows behind the first 2^31 bytes of one page, through the kernel for any rotary_dim
    (a rotation by no angle) and through the other one."""
    D, pt, n = 256, (1 << 23) + 64, 5
    k, v = rows((n, 1, D), "f32", 1), rows((n, 1, D), "f32", 2)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    ctx = torch.tensor([pt - 3], dtype=torch.int32, device=DEV)
    start = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    first = pt - 3 - n
    for rope in (cuda_lib.rope_table(20, inv_freq=[0.0] * 10), None):
        pools = [cuda_lib.new_fp8_pool(1, 1, pt, D) for _ in range(2)]
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        cuda_lib.paged_kv_write(k.to(DEV), v.to(DEV), *pools, table, ctx, start, rope=rope, err_word=err)
        torch.cuda.synchronize()
        assert int(err) == 0
        for x, p in ((k, pools[0]), (v, pools[1])):
            codes, scales = orc.quantise_rows(x[:, 0])
            page = p[0, 0]
            assert torch.equal(page[first * D:(first + n) * D].cpu().view(n, D), codes)
            assert torch.equal(page[pt * D + first:pt * D + first + n].cpu(), scales)
            assert int((page[:first * D].view(torch.int64) != 0).sum()) == 0
        del pools, page, p
