"""GPU parity of rotary_embed against the 64-bit rotation.

Tolerance of an element of pair (u, v): the angle reaches sincospi as a fraction
of a turn cut at 2^-32 and rounded to fp32 (2^-24 of at most pi), sincospi is
within 2 ulp, cos * mscale, the two products and their sum round 4 times: all
below 2^-21 (|u| + |v|) |mscale|; then half a step of the output type."""
import math

import pytest
import torch

from oracle import serving as orc

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def bound(want, mag, dtype):
    fi = torch.finfo(dtype)
    return mag * 2.0 ** -21 + (want.abs() + mag * 2.0 ** -21) * fi.eps / 2 + fi.smallest_normal * fi.eps


def check(got, want, mag, what=""):
    got = got.cpu()
    off = (got.double() - want).abs() - bound(want, mag, got.dtype)
    assert torch.isfinite(got.double()).all(), what
    assert float(off.max()) <= 0, f"{what}: {float(off.max()):.3e} over the bound"


SPECS = [dict(), dict(interleaved=True), dict(scaling="linear", factor=4.0),
         dict(scaling="ntk", factor=8.0, interleaved=True),
         dict(scaling="ramp", factor=16.0, original_len=4096, mscale=1.27)]


def freqs(R, spec):
    kw = {k: v for k, v in spec.items() if k not in ("interleaved", "mscale")}
    return orc.rope_freqs(R, **kw)


def oracle(x, pos, R, spec):
    return orc.rotate(x.cpu(), pos.cpu(), freqs(R, spec), spec.get("interleaved", False),
                      spec.get("mscale", 1.0))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("spec", SPECS, ids=lambda s: s.get("scaling", "none") + str(int(s.get("interleaved", 0))))
@pytest.mark.parametrize("T,Hq,Hk,D,R", [(1, 4, 1, 64, 64), (37, 8, 2, 128, 64), (700, 3, 1, 80, 40),
                                         (5, 16, 16, 256, 256), (130, 5, 5, 96, 96), (9, 2, 1, 64, 6)])
def test_packed_rows(cuda_lib, dt, spec, T, Hq, Hk, D, R):
    g = torch.Generator().manual_seed(T * 131 + D)
    q, k = (torch.randn(T, H, D, generator=g).to(DT[dt]).to(DEV) for H in (Hq, Hk))
    pos = torch.randint(0, 1 << 21, (T,), generator=g)
    pos[0] = 0
    rope = cuda_lib.rope_table(R, **spec)
    for p in (pos, pos.to(torch.int32)):
        yq, yk = cuda_lib.rotary_embed(q, k, p.to(DEV), rope)
        torch.cuda.synchronize()
        for x, y in ((q, yq), (k, yk)):
            want, mag = oracle(x, pos[:, None], R, spec)
            check(y, want, mag, f"{dt} {spec}")
            assert torch.equal(y[..., R:], x[..., R:])   # the dims past the rotated ones, exactly


@pytest.mark.parametrize("shared", [True, False])
def test_head_major_tensors_and_positions_of_every_batch(cuda_lib, shared):
    g = torch.Generator().manual_seed(3)
    q = torch.randn(3, 6, 41, 64, generator=g).half().to(DEV)
    k = torch.randn(3, 2, 41, 64, generator=g).half().to(DEV)
    pos = torch.randint(0, 100000, (41,) if shared else (3, 41), generator=g)
    rope = cuda_lib.rope_table(32, interleaved=True)
    yq, yk = cuda_lib.rotary_embed(q, k, pos.to(DEV), rope)
    at = pos.expand(3, 41)[:, None]
    for x, y in ((q, yq), (k, yk)):
        assert y.is_contiguous()
        want, mag = oracle(x, at, 32, dict(interleaved=True))
        check(y, want, mag)


@pytest.mark.parametrize("R", [128, 48, 6])
def test_views_of_one_projection_in_place(cuda_lib, R):
    """q and k are heads of one buffer: rotated where they stand, v untouched."""
    g = torch.Generator().manual_seed(4)
    buf = torch.randn(333, 8 + 2 + 2, 128, generator=g).bfloat16().to(DEV)
    old = buf.clone()
    pos = torch.arange(1000, 1333, device=DEV)
    rope = cuda_lib.rope_table(R)
    q, k = buf[:, :8], buf[:, 8:10]
    yq, yk = cuda_lib.rotary_embed(q, k, pos, rope, q_out=q, k_out=k)
    assert yq.data_ptr() == buf.data_ptr()
    for a, b in ((0, 8), (8, 10)):
        want, mag = oracle(old[:, a:b], pos[:, None], R, {})
        check(buf[:, a:b], want, mag)
    assert torch.equal(buf[:, 10:], old[:, 10:])


def test_odd_strides_and_a_misaligned_view(cuda_lib):
    g = torch.Generator().manual_seed(5)
    base = torch.randn(50, 4, 67, generator=g).bfloat16().to(DEV)
    q = base[:, :, 3:67]                 # rows of 64, 6 bytes off, stride 67
    pos = torch.arange(50, device=DEV)
    y, none = cuda_lib.rotary_embed(q, None, pos, cuda_lib.rope_table(64))
    assert none is None
    want, mag = oracle(q, pos[:, None], 64, {})
    check(y, want, mag)


def test_far_and_negative_positions(cuda_lib):
    """Exact angle reduction at positions whose fp32 product has no fraction left."""
    pos = torch.tensor([2 ** 24 + 1, 2 ** 31 - 1, -1, -12345, 2 ** 26 + 3])
    q = torch.randn(5, 2, 128, generator=torch.Generator().manual_seed(6)).to(DEV)
    y, _ = cuda_lib.rotary_embed(q, None, pos.to(DEV), cuda_lib.rope_table(128))
    want, mag = oracle(q, pos[:, None], 128, {})
    # the oracle's own angle: a double product of up to 2^31 rad is 2^-22 off at most, in
    # the same pairs; positions here keep it below 2^31 * 2^-53
    off = (y.cpu().double() - want).abs() - bound(want, mag, y.dtype) - mag * 2.0 ** -21
    assert float(off.max()) <= 0


def test_no_tokens_is_a_call_that_does_nothing(cuda_lib):
    q = torch.empty(0, 4, 64, device=DEV)
    y, _ = cuda_lib.rotary_embed(q, None, torch.empty(0, dtype=torch.int64, device=DEV),
                                 cuda_lib.rope_table(64))
    assert y.shape == (0, 4, 64)


def test_captured_replayed_and_on_another_stream(cuda_lib):
    q = torch.randn(64, 8, 128, device=DEV, dtype=torch.float16)
    k = torch.randn(64, 2, 128, device=DEV, dtype=torch.float16)
    pos = torch.arange(64, device=DEV)
    rope = cuda_lib.rope_table(128)
    want = cuda_lib.rotary_embed(q, k, pos, rope)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = cuda_lib.rotary_embed(q, k, pos, rope, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = cuda_lib.rotary_embed(q, k, pos, rope)
    pos += 100
    g.replay()
    want = cuda_lib.rotary_embed(q, k, pos, rope)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals(cuda_lib):
    sa = cuda_lib
    q = torch.zeros(8, 4, 64, device=DEV)
    pos = torch.arange(8, device=DEV)
    rope = sa.rope_table(64)
    with pytest.raises(TypeError):
        sa.rotary_embed(q, None, pos.float(), rope)
    with pytest.raises(TypeError):
        sa.rotary_embed(q, q.half(), pos, rope)
    with pytest.raises(TypeError):
        sa.rotary_embed(q, None, pos, object())
    with pytest.raises(ValueError):
        sa.rotary_embed(q, None, pos[:7], rope)
    with pytest.raises(ValueError):
        sa.rotary_embed(q.transpose(1, 2), None, pos, rope)
    with pytest.raises(sa.SAError):                       # rotary_dim beyond the head
        sa.rotary_embed(q[..., :32].contiguous(), None, pos, rope)
    with pytest.raises(sa.SAError):                       # an output one row further on
        buf = torch.zeros(9, 4, 64, device=DEV)
        sa.rotary_embed(buf[:8], None, pos, rope, q_out=buf[1:])
    with pytest.raises(sa.SAError):                       # an output that repeats its rows
        sa.rotary_embed(q, None, pos, rope, q_out=torch.zeros(1, 4, 64, device=DEV).expand(8, 4, 64))
    with pytest.raises(sa.SAError):
        sa.rotary_embed(q, q[:, :2], pos, rope, q_out=None, k_out=q[:, 2:])


@pytest.mark.parametrize("order", ["head-major", "token-major"])
def test_views_of_one_projection_of_several_batches_in_place(cuda_lib, order):
    """q and k as heads of one [B, Hq + 2 Hk, S, D] (or [B, S, Hq + 2 Hk, D]) buffer."""
    sa = cuda_lib
    B, S, Hq, Hk, D = 3, 50, 8, 2, 128
    g = torch.Generator().manual_seed(1)
    if order == "head-major":
        buf = torch.randn(B, Hq + 2 * Hk, S, D, generator=g).bfloat16().to(DEV)
        q, k, v = buf[:, :Hq], buf[:, Hq:Hq + Hk], buf[:, Hq + Hk:]
    else:
        buf = torch.randn(B, S, Hq + 2 * Hk, D, generator=g).bfloat16().to(DEV)
        q, k, v = (x.transpose(1, 2) for x in (buf[:, :, :Hq], buf[:, :, Hq:Hq + Hk], buf[:, :, Hq + Hk:]))
    pos = torch.randint(0, 5000, (B, S), generator=g).to(DEV)
    rope = sa.rope_table(D)
    want = sa.rotary_embed(q.contiguous(), k.contiguous(), pos, rope)
    before = v.clone()
    a, b = sa.rotary_embed(q, k, pos, rope, q_out=q, k_out=k)
    assert a.data_ptr() == q.data_ptr() and b.data_ptr() == k.data_ptr()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, before)
    with pytest.raises(sa.SAError):                       # keys that begin inside the queries
        x = (buf[:, Hq - 1:Hq - 1 + Hk] if order == "head-major" else buf[:, :, Hq - 1:Hq - 1 + Hk].transpose(1, 2))
        sa.rotary_embed(q, x, pos, rope, q_out=q, k_out=x)


def test_keys_without_queries_are_refused(cuda_lib):
    """Queries of no heads beside keys of some: not a call that returns keys never written."""
    sa = cuda_lib
    rope, pos = sa.rope_table(64), torch.arange(5, device=DEV)
    k = torch.ones(5, 2, 64, device=DEV, dtype=torch.bfloat16)
    with pytest.raises(sa.SAError):
        sa.rotary_embed(k[:, :0], k, pos, rope)
    with pytest.raises(sa.SAError):
        sa.rotary_embed(k[None].transpose(1, 2)[:, :0], k[None].transpose(1, 2), pos, rope)
    q, none = sa.rotary_embed(k[:, :0], None, pos, rope)
    assert q.shape == (5, 0, 64) and none is None
    q, x = sa.rotary_embed(k[:0], k[:0], pos[:0], rope)
    assert q.shape == x.shape == (0, 2, 64)
