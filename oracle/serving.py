"""Plain 64-bit forms of the serving-step operators (rotary positions, FP8 pages,
decode over them, packed prefill), written from their definitions in
include/sa.h and sharing no code with the library.  CPU tensors in, float64 out;
what a bound needs (sums of magnitudes) comes beside the values."""
from __future__ import annotations

import math

import torch

__all__ = ["rope_freqs", "rotate", "e4m3_values", "quantise_rows", "dequantise_rows", "read_row",
           "write_row", "attend", "prefill_packed"]


def rope_freqs(rotary_dim, base=10000.0, scaling="none", factor=1.0, original_len=0,
               ramp=(1.0, 32.0)):
    """f_i of the rotary pairs, as Python floats."""
    out = []
    for i in range(rotary_dim // 2):
        b = base * factor ** (rotary_dim / (rotary_dim - 2)) if scaling == "ntk" else base
        f = b ** (-2.0 * i / rotary_dim)
        if scaling == "linear":
            f /= factor
        if scaling == "ramp":
            g = (original_len * f / (2 * math.pi) - ramp[0]) / (ramp[1] - ramp[0])
            g = min(1.0, max(0.0, g))
            f = f * g + f / factor * (1 - g)
        out.append(f)
    return out


def rotate(x, positions, freqs, interleaved=False, mscale=1.0):
    """``x [..., D]`` at ``positions [...]`` (broadcast): (rotated, |u| + |v| of each element's
    pair times |mscale|, 0 past the rotated dims)."""
    x = x.double()
    y, mag = x.clone(), torch.zeros_like(x)
    R = 2 * len(freqs)
    for i, f in enumerate(freqs):
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        a = torch.remainder(positions.double() * f, 2 * math.pi)
        c, s = torch.cos(a) * mscale, torch.sin(a) * mscale
        u, v = x[..., lo], x[..., hi]
        y[..., lo], y[..., hi] = u * c - v * s, u * s + v * c
        mag[..., lo] = mag[..., hi] = (u.abs() + v.abs()) * abs(mscale)
    return y, mag


def e4m3_values():
    """The values of the 256 E4M3FN codes (OCP: bias 7, S.1111.111 is NaN)."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.nan if (e, m) == (15, 7) else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(-x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64)


def quantise_rows(x):
    """Rows ``[n, D]`` -> (codes uint8 [n, D], scale bytes uint8 [n]): the nearest code, ties to
    the even one, by comparing with every value of the grid."""
    x = x.double()
    grid = e4m3_values()[:127]  # 0 .. 448, ascending: index = code
    codes = torch.zeros(x.shape, dtype=torch.uint8)
    scales = torch.zeros(x.shape[0], dtype=torch.uint8)
    for r, row in enumerate(x):
        if not torch.isfinite(row).all():
            scales[r] = 255
            continue
        top = float(row.abs().max())
        e = -127
        if top == 0:
            e = 0
        else:
            while top > 448 * 2.0 ** e:
                e += 1
        y = row / 2.0 ** e
        d = (y.abs()[:, None] - grid[None]).abs()
        best = d.min(1).values
        near = d == best[:, None]
        c = torch.argmax(near.int(), 1)                    # the lower of two equally near
        two = near.sum(1) > 1
        c = torch.where(two & (c % 2 == 1), c + 1, c)      # the even one
        codes[r] = (c + 128 * (torch.signbit(row)).long()).to(torch.uint8)
        scales[r] = e + 127
    return codes, scales


def dequantise_rows(codes, scales):
    s = torch.where(scales == 255, math.nan, 2.0 ** (scales.double() - 127))
    return e4m3_values()[codes.long()] * s[..., None]


def read_row(pool, page, head, slot, page_tokens, D):
    """(codes, scale byte) of one row of an FP8 pool."""
    p = pool[page, head]
    return p[slot * D:(slot + 1) * D], p[page_tokens * D + slot]


def write_row(pool, page, head, slot, page_tokens, D, codes, scale):
    pool[page, head, slot * D:(slot + 1) * D] = codes
    pool[page, head, page_tokens * D + slot] = scale


def _softmax_rows(s):
    """Softmax of the last axis; a row of nothing but -inf gives zeros."""
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    z = p.sum(-1, keepdim=True)
    return torch.where(z > 0, p / z, torch.zeros_like(p))


def attend(q, k, v, scale):
    """One sequence, one KV head: ``q [G, D]``, ``k, v [n, D]`` -> (y, sum p |v|, the largest
    sum |q||k| scale)."""
    q, k, v = q.double(), k.double(), v.double()
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.zeros_like(q), 0.0
    p = _softmax_rows(q @ k.T * scale)
    return p @ v, p @ v.abs(), float((q.abs() @ k.abs().T).max()) * abs(scale)


def prefill_packed(q, k, v, q_start, k_start, causal=True, scale=0.0, softcap=0.0):
    """Packed ``q [Tq, Hq, D]``, ``k, v [Tk, Hkv, D]`` with lists of starts -> (y, sum p |v|, the
    largest score magnitude sum); rows of no sequence are NaN."""
    D, g = q.shape[2], q.shape[1] // k.shape[1]
    scale = scale or 1 / math.sqrt(D)
    y = torch.full(q.shape, math.nan, dtype=torch.float64)
    mag = torch.zeros(q.shape, dtype=torch.float64)
    most = 0.0
    for b in range(len(q_start) - 1):
        qa, qe, ka, ke = q_start[b], q_start[b + 1], k_start[b], k_start[b + 1]
        n, m = qe - qa, ke - ka
        hide = torch.arange(m)[None] > torch.arange(n)[:, None] + (m - n)
        for h in range(q.shape[1]):
            qq, kk, vv = (t.double() for t in (q[qa:qe, h], k[ka:ke, h // g], v[ka:ke, h // g]))
            if n == 0:
                continue
            if m == 0:
                y[qa:qe, h] = 0
                continue
            s = qq @ kk.T * scale
            most = max(most, float((qq.abs() @ torch.nan_to_num(kk).abs().T).max()) * abs(scale))
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            if causal:
                s = s.masked_fill(hide, -math.inf)
            p = _softmax_rows(s)
            # a hidden key's value never counts, whatever it holds
            vis = (~hide if causal else torch.ones_like(hide))
            for c in range(n):
                keep = vis[c]
                y[qa + c, h] = p[c, keep] @ vv[keep]
                mag[qa + c, h] = p[c, keep] @ vv[keep].abs()
    return y, mag, most
