"""GPU parity of attn_prefill_packed against 64-bit attention, sequence by sequence.

Tolerance: a score is off by e_s = D 2^-22 max sum|q||k| scale (fp32 sums), with a
softcap c by 2^-20 c more (tanh), and its exp2 by 2^-16; 16-bit types round the
probability once before the product (half a step), the sums add D 2^-22 and 2^-16.
An output is off by that total times sum p |v|, plus half a step of its type."""
import math

import pytest
import torch

from oracle import serving as orc

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def make(dt, nq, nk, Hq, Hkv, D, seed=0, pad=2):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(sum(nq) + pad, Hq, D, generator=g).to(DT[dt])
    k, v = (torch.randn(sum(nk) + pad, Hkv, D, generator=g).to(DT[dt]) for _ in range(2))
    qs, ks = [0], [0]
    for a, b in zip(nq, nk):
        qs.append(qs[-1] + a)
        ks.append(ks[-1] + b)
    return q, k, v, qs, ks


def starts(s):
    return torch.tensor(s, dtype=torch.int32, device=DEV)


def check(y, q, k, v, qs, ks, causal=True, softcap=0.0, scale=0.0, what=""):
    want, mag, most = orc.prefill_packed(q, k, v, qs, ks, causal, scale, softcap)
    y = y.cpu()
    fi = torch.finfo(y.dtype)
    D = q.shape[2]
    rel = 2 * (D * 2.0 ** -22 * most + 2.0 ** -20 * softcap + 2.0 ** -16) + D * 2.0 ** -22 + 2.0 ** -16
    if y.dtype != torch.float32:
        rel += fi.eps / 2
    own = ~torch.isnan(want)
    tol = rel * mag + (want.abs() + rel * mag) * fi.eps / 2 + fi.smallest_normal * fi.eps
    assert torch.isfinite(y[own].double()).all(), what
    off = float(((y.double() - want).abs() - tol)[own].max()) if own.any() else 0.0
    assert off <= 0, f"{what}: {off:.3e} over the bound"


SHAPES = [  # (queries, keys, Hq, Hkv, D)
    ([1], [1], 1, 1, 64), ([5, 1, 40], [5, 1, 40], 4, 2, 64), ([130, 7, 0, 64], [130, 7, 0, 64], 8, 2, 128),
    ([1, 1, 3], [300, 17, 129], 8, 1, 128), ([33, 128], [161, 128], 6, 2, 64), ([257], [257], 3, 1, 128),
    ([20, 9], [0, 4], 4, 4, 64), ([100, 50], [30, 600], 5, 5, 128), ([260], [515], 16, 1, 128), ([3] * 50, [40] * 50, 2, 1, 64),
    ([11], [150], 32, 1, 128), ([64, 65], [64, 65], 7, 1, 64)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("causal,cap", [(True, 0.0), (False, 0.0), (True, 30.0), (False, 2.0), (True, 200.0)])
@pytest.mark.parametrize("nq,nk,Hq,Hkv,D", SHAPES)
def test_matches_64_bits(cuda_lib, dt, causal, cap, nq, nk, Hq, Hkv, D):
    q, k, v, qs, ks = make(dt, nq, nk, Hq, Hkv, D, seed=len(nq) + D)
    # what belongs to no sequence may be anything, and is left alone in y
    k[ks[-1]:], v[ks[-1]:] = float("nan"), float("inf")
    y = torch.full(q.shape, 9.0, dtype=DT[dt], device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = cuda_lib.attn_prefill_packed(q.to(DEV), k.to(DEV), v.to(DEV), starts(qs), starts(ks), causal=causal, softcap=cap,
                                       y=y, err_word=err)
    torch.cuda.synchronize()
    assert int(err) == 0 and out.data_ptr() == y.data_ptr()
    check(y, q, k, v, qs, ks, causal, cap, what=f"{dt} {causal} {cap}")
    assert (y[qs[-1]:] == 9.0).all()


@pytest.mark.parametrize("D,dt", [(96, "bf16"), (256, "f16"), (72, "f32"), (4, "f16"), (256, "f32"), (128, "bf16")])
def test_other_head_sizes_scales_and_same_starts(cuda_lib, D, dt):
    q, k, v, qs, _ = make(dt, [30, 90], [30, 90], 4, 2, D, seed=D)
    scale = 0.3 if D != 128 else -0.1                     # a negative scale as well
    y = cuda_lib.attn_prefill_packed(q.to(DEV), k.to(DEV), v.to(DEV), starts(qs), scale=scale)
    check(y, q, k, v, qs, qs, scale=scale)


def test_neighbours_and_hidden_keys_never_leak(cuda_lib):
    """NaN and infinities in the keys and values of the next sequence, and in keys that a
    query does not see, leave its row as it is."""
    for D, dt in ((128, "bf16"), (64, "f16"), (128, "f32")):
        q, k, v, qs, ks = make(dt, [70, 70, 10], [100, 70, 10], 4, 2, D)
        clean = cuda_lib.attn_prefill_packed(q.to(DEV), k.to(DEV), v.to(DEV), starts(qs), starts(ks))
        k2, v2 = k.clone(), v.clone()
        k2[100:170], v2[100:170] = float("nan"), float("inf")      # the whole second sequence
        v2[175:], k2[178] = float("-inf"), float("nan")            # the third's last keys
        y = cuda_lib.attn_prefill_packed(q.to(DEV), k2.to(DEV), v2.to(DEV), starts(qs), starts(ks))
        assert torch.equal(y[:70], clean[:70])
        assert torch.equal(y[140:145], clean[140:145])             # queries 0 .. 4 see keys 0 .. 4
        assert not torch.isfinite(y[145:150].float()).any()
        assert not torch.isfinite(y[70:140].float()).any()


def test_strided_views(cuda_lib):
    """q, k and v as heads of one projection, y as heads of a wider buffer."""
    g = torch.Generator().manual_seed(3)
    buf = torch.randn(150, 8 + 2 + 2, 128, generator=g).bfloat16().to(DEV)
    q, k, v = buf[:, :8], buf[:, 8:10], buf[:, 10:]
    s = starts([0, 50, 150])
    want = cuda_lib.attn_prefill_packed(q.contiguous(), k.contiguous(), v.contiguous(), s)
    wide = torch.zeros(150, 12, 128, dtype=torch.bfloat16, device=DEV)
    got = cuda_lib.attn_prefill_packed(q, k, v, s, y=wide[:, 2:10])
    assert torch.equal(got, want) and not wide[:, :2].any() and not wide[:, 10:].any()
    check(want, q.cpu(), k.cpu(), v.cpu(), [0, 50, 150], [0, 50, 150])
    odd = torch.randn(150, 3, 67, generator=g).half().to(DEV)      # rows off 16 bytes
    x = odd[:, :, 1:65]
    check(cuda_lib.attn_prefill_packed(x, x, x, s), x.cpu(), x.cpu(), x.cpu(), [0, 50, 150], [0, 50, 150])


def test_longer_prompts_sampled(cuda_lib):
    nq, nk = [1000, 37, 2049], [1000, 1500, 2049]
    q, k, v, qs, ks = make("bf16", nq, nk, 8, 2, 128, seed=5)
    y = cuda_lib.attn_prefill_packed(q.to(DEV), k.to(DEV), v.to(DEV), starts(qs), starts(ks)).cpu()
    for h in (0, 5):
        kv = h // 4
        check(y[:, h:h + 1], q[:, h:h + 1], k[:, kv:kv + 1], v[:, kv:kv + 1], qs, ks)


def test_large_scores_and_equal_rows(cuda_lib):
    """Scores of hundreds (the running maximum rises in every tile) and rows of equal keys."""
    q, k, v, qs, ks = make("f16", [300], [300], 2, 1, 64, seed=7)
    k *= torch.linspace(0.1, 12, 302)[:, None, None].half()
    y = cuda_lib.attn_prefill_packed(q.to(DEV), k.to(DEV), v.to(DEV), starts(qs), starts(ks), scale=1.0)
    check(y, q, k, v, qs, ks, scale=1.0)
    k[:] = k[0]
    y = cuda_lib.attn_prefill_packed(q.to(DEV), k.to(DEV), v.to(DEV), starts(qs), starts(ks))
    check(y, q, k, v, qs, ks)


def test_nothing_to_do(cuda_lib):
    z = torch.empty(0, 4, 64, dtype=torch.float16, device=DEV)
    assert cuda_lib.attn_prefill_packed(z, z, z, starts([0, 0])).shape == (0, 4, 64)
    q = torch.randn(9, 4, 64, device=DEV, dtype=torch.float16)
    y = cuda_lib.attn_prefill_packed(q, z, z, starts([0, 4, 9]), starts([0, 0, 0]))
    assert not y.any()


def test_malformed_starts_are_reported(cuda_lib):
    sa = cuda_lib
    for dt, D in (("bf16", 128), ("f32", 64)):
        q, k, v, _, _ = make(dt, [200], [200], 4, 2, D, pad=0)
        for s in ([0, 150, 100, 200], [0, 50, 10 ** 8, 200], [-50, 50, 100, 200], [0, 200, 0, 200]):
            err = torch.zeros(1, dtype=torch.int32, device=DEV)
            sa.attn_prefill_packed(q.to(DEV), k.to(DEV), v.to(DEV), starts(s), err_word=err)
            torch.cuda.synchronize()
            assert int(err) == sa.ERRBIT_SEQ, s


def test_captured_and_on_another_stream(cuda_lib):
    q, k, v, qs, ks = make("bf16", [64, 300], [64, 300], 4, 2, 128, pad=0)
    q, k, v = q.to(DEV), k.to(DEV), v.to(DEV)
    a, b = starts(qs), starts(ks)
    want = cuda_lib.attn_prefill_packed(q, k, v, a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = cuda_lib.attn_prefill_packed(q, k, v, a, b, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = cuda_lib.attn_prefill_packed(q, k, v, a, b)
    a.copy_(starts([0, 100, 364]))
    b.copy_(a)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, cuda_lib.attn_prefill_packed(q, k, v, a, b)) and not torch.equal(out, want)


def test_refusals(cuda_lib):
    sa = cuda_lib
    q = torch.zeros(10, 4, 64, dtype=torch.float16, device=DEV)
    k = torch.zeros(10, 2, 64, dtype=torch.float16, device=DEV)
    s = starts([0, 10])
    for args in ((q, k, k.float(), s), (q, k.float(), k.float(), s), (q, k, k, s.long()), (q, k, k, s, s.long())):
        with pytest.raises(TypeError):
            sa.attn_prefill_packed(*args)
    for args in ((q, k[:9], k[:9], s), (q, k, k[:9], s, s), (q, k[..., :32].contiguous(), k[..., :32].contiguous(), s),
                 (q, k, k, s, starts([0, 5, 10])), (q.transpose(1, 2), k, k, s)):
        with pytest.raises(ValueError):
            sa.attn_prefill_packed(*args)
    with pytest.raises(sa.SAError):                       # 3 KV heads for 4 query heads
        sa.attn_prefill_packed(q, torch.zeros(10, 3, 64, dtype=torch.float16, device=DEV),
                               torch.zeros(10, 3, 64, dtype=torch.float16, device=DEV), s)
    for kw in (dict(softcap=-1.0), dict(scale=float("nan")), dict(y=q)):
        with pytest.raises(sa.SAError):
            sa.attn_prefill_packed(q, k, k, s, **kw)
    with pytest.raises(sa.SAError):
        x = torch.zeros(10, 2, 258, dtype=torch.float16, device=DEV)
        sa.attn_prefill_packed(x, x, x, s)


def leaning(dt, nq, nk, Hq, Hkv, D, lean, seed):
    """Queries and keys whose scores (scale 1 / sqrt(D)) lie around `lean`, or around both
    signs of it ("mixed": a sign per key)."""
    q, k, v, qs, ks = make(dt, nq, nk, Hq, Hkv, D, seed=seed)
    mean, size = (24.0, 24.0) if lean == "mixed" else (lean, abs(lean))
    side = math.sqrt(size / math.sqrt(D))
    sign = torch.where(torch.rand(k.shape[:2], generator=torch.Generator().manual_seed(seed)) < 0.5, -1.0, 1.0)[..., None] \
        if lean == "mixed" else math.copysign(1.0, mean)
    return (side + 0.3 * q.float()).to(DT[dt]), (sign * side + 0.3 * k.float()).to(DT[dt]), v, qs, ks


def check_tail(y, q, k, v, qs, ks, causal, cap, what, tanh=2.0 ** -20):
    """check()'s bound (`tanh`: of the softcap's tanh), and for f16 what its subnormal probabilities lose: a probability
    held against an offset of at most the row's maximum is off by half of 2^-24 at the
    most, and the row's sum is at least 1."""
    want, mag, most = orc.prefill_packed(q, k, v, qs, ks, causal, 0.0, cap)
    y = y.cpu()
    fi = torch.finfo(y.dtype)
    D, g = q.shape[2], q.shape[1] // k.shape[1]
    rel = 2 * (D * 2.0 ** -22 * most + tanh * cap + 2.0 ** -16) + D * 2.0 ** -22 + 2.0 ** -16 + fi.eps / 2
    lost = torch.zeros_like(want)
    if y.dtype == torch.float16:
        for b in range(len(qs) - 1):
            s = v[ks[b]:ks[b + 1]].double().abs().sum(0) * 2.0 ** -25
            lost[qs[b]:qs[b + 1]] = s.repeat_interleave(g, 0)[None]
    own = ~torch.isnan(want)
    near = rel * mag + lost
    tol = near + (want.abs() + near) * fi.eps / 2 + fi.smallest_normal * fi.eps
    assert torch.isfinite(y[own].double()).all(), what
    off = float(((y.double() - want).abs() - tol)[own].max())
    assert off <= 0, f"{what}: {off:.3e} over the bound"


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("cap", [9.7, 9.8, 30.0, 50.0, 67.0, 68.0])
@pytest.mark.parametrize("lean", [24.0, -24.0, 100.0, -100.0, "mixed"])
def test_scores_that_reach_the_softcap(cuda_lib, dt, cap, lean):
    """Logits around +-20 and at the cap itself: what 2^logit is without an offset is far
    outside f16 there, on either side."""
    for D, Hq, Hkv in ((128, 4, 2), (64, 3, 1)):
        q, k, v, qs, ks = leaning(dt, [200, 70], [512, 70], Hq, Hkv, D, lean, seed=int(cap))
        y = cuda_lib.attn_prefill_packed(q.to(DEV), k.to(DEV), v.to(DEV), starts(qs), starts(ks), softcap=cap)
        check_tail(y, q, k, v, qs, ks, True, cap, f"{dt} cap {cap} lean {lean} D {D}")


@pytest.mark.parametrize("dt,D,cap", [("bf16", 128, 30.0), ("bf16", 64, 200.0), ("f16", 128, 30.0), ("f16", 64, 9.0)])
def test_with_a_softcap_too_neighbours_and_hidden_keys_leave_the_bits(cuda_lib, dt, D, cap):
    """Keys that none of a warp's rows sees and other sequences' queries and keys do not choose
    the form in which its logits are computed."""
    q, k, v, qs, ks = make(dt, [70, 70, 64], [100, 70, 64], 4, 2, D)
    run = lambda *a: cuda_lib.attn_prefill_packed(*(t.to(DEV) for t in a), starts(qs), starts(ks), softcap=cap)  # noqa: E731
    clean = run(q, k, v)
    for x in (float("nan"), 300.0):
        k2, q2 = k.clone(), q.clone()
        k2[100:170], q2[70:140] = x, x                             # the whole second sequence
        k2[218:] = x                                               # the third's keys 48 to 63
        y = run(q2, k2, v)
        assert torch.equal(y[:70], clean[:70])
        assert torch.equal(y[140:188], clean[140:188])             # its queries 0 .. 47: three warps


@pytest.mark.parametrize("g", [3, 5])
@pytest.mark.parametrize("cap", [30.0, 200.0])
def test_rows_of_a_tile_without_a_head_do_not_count(cuda_lib, g, cap):
    """Heads that do not divide 128, several query tiles per CTA: large outputs of other
    sequences, which pass through the query tiles' memory, leave a row's bits alone."""
    n = [50] * 120
    q, k, v, qs, _ = make("bf16", n, n, 4 * g, 4, 64, seed=g)
    run = lambda v: cuda_lib.attn_prefill_packed(q.to(DEV), k.to(DEV), v.to(DEV), starts(qs), softcap=cap)  # noqa: E731
    clean = run(v)
    for period in (2, 4, 8, 16, 32):                               # whichever items share a CTA's buffer
        v2 = v.clone()
        for b in range(120):
            if b % period < period // 2:
                v2[qs[b]:qs[b + 1]] *= 1e4
        y = run(v2)
        for b in range(120):
            if b % period >= period // 2:
                assert torch.equal(y[qs[b]:qs[b + 1]], clean[qs[b]:qs[b + 1]]), (period, b)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("cap", [100.0, 1e3, 1e4, 1e6, 1e8, 1e12])
def test_a_softcap_far_above_the_scores(cuda_lib, dt, cap):
    """The logits' error goes by the logits, not by the cap: scores of up to 12 in magnitude,
    each off by 2^-18 of itself at the most, in tiles with hidden keys and in others."""
    for D, nq, nk in ((128, [70, 1, 300], [70, 200, 700]), (64, [257], [257])):
        q, k, v, qs, ks = make(dt, nq, nk, 4, 2, D, seed=int(math.log10(cap)))
        y = cuda_lib.attn_prefill_packed(q.to(DEV), k.to(DEV), v.to(DEV), starts(qs), starts(ks), softcap=cap)
        check_tail(y, q, k, v, qs, ks, True, cap, f"{dt} cap {cap} D {D}", tanh=2.0 ** -18 * 12 / cap)


@pytest.mark.parametrize("dt,scale", [("bf16", 0.1), ("f16", 0.1), ("f32", 0.1), ("f32", -0.1)])
def test_the_largest_softcap_is_none(cuda_lib, dt, scale):
    q, k, v, qs, _ = make(dt, [70, 200], [70, 200], 4, 2, 64)
    run = lambda cap: cuda_lib.attn_prefill_packed(q.to(DEV), k.to(DEV), v.to(DEV), starts(qs), scale=scale, softcap=cap)  # noqa: E731
    y = run(3.4e38)
    assert torch.equal(y[:270], run(0.0)[:270]) and torch.isfinite(y[:270].float()).all()
