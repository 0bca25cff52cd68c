"""Plain 64-bit forms of the operators that keep a paged cache within a budget of tokens
(attention weights, selection, compaction), written from their definitions in include/sa.h
and sharing no code with the library.  CPU tensors in."""
from __future__ import annotations

import math

import torch

__all__ = ["weights_packed", "weights_decode", "token_places", "put_weights", "select_row",
           "row_code", "compact_row"]


def _softmax(s):
    """Softmax of the last axis in 64 bits; a row of nothing but -inf gives zeros."""
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    z = p.sum(-1, keepdim=True)
    return torch.where(z == 0, torch.zeros_like(p), p / z)


def weights_packed(q, k, q_start, k_start, scale=0.0):
    """Per sequence: (w [Hkv, nk], the largest sum |q||k| |scale| of a visible pair)."""
    D, g = q.shape[2], q.shape[1] // k.shape[1]
    scale = scale or 1 / math.sqrt(D)
    out = []
    for b in range(len(q_start) - 1):
        qq = q[q_start[b]:q_start[b + 1]].double()
        kk = k[k_start[b]:k_start[b + 1]].double()
        n, m = qq.shape[0], kk.shape[0]
        w, most = torch.zeros(k.shape[1], m, dtype=torch.float64), 0.0
        if n and m:
            hide = torch.arange(m)[None] > torch.arange(n)[:, None] + (m - n)
            for h in range(q.shape[1]):
                s = (qq[:, h] @ kk[:, h // g].T * scale).masked_fill(hide, -math.inf)
                w[h // g] += _softmax(s).masked_fill(hide, 0.0).sum(0)
                mag = (qq[:, h].abs() @ kk[:, h // g].abs().T).masked_fill(hide, 0.0)
                most = max(most, float(torch.nan_to_num(mag, posinf=0.0).max()) * abs(scale))
        out.append((w, most))
    return out


def weights_decode(q, k, scale):
    """One sequence: ``q [Hq, D]``, ``k [Hkv, n, D]`` -> (w [Hkv, n], the largest sum |q||k| |scale|)."""
    qq = q.double().view(k.shape[0], -1, q.shape[-1])
    kk = k.double()
    w = _softmax(qq @ kk.transpose(1, 2) * scale).sum(1)
    return w, float((qq.abs() @ kk.abs().transpose(1, 2)).max()) * abs(scale)


def token_places(table_row, n, page_tokens):
    """(page, slot) of the tokens 0 .. n - 1 of a sequence."""
    t = torch.arange(n)
    return table_row.long()[t // page_tokens], t % page_tokens


def put_weights(pool, table_row, w, fresh):
    """w [Hkv, n] into a 64-bit pool: the last ``fresh`` tokens set, the others added."""
    n = w.shape[1]
    page, slot = token_places(table_row, n, pool.shape[2])
    old = pool[page, :, slot].clone()                      # [n, Hkv]
    old[n - min(fresh, n):] = 0
    pool[page, :, slot] = old + w.T


def select_row(w, budget, sink, recent):
    """The tokens kept of one context's weights (a list of floats), ascending."""
    n = len(w)
    if n <= budget:
        return list(range(n))
    middle = range(sink, n - recent)
    rank = sorted(middle, key=lambda t: (-(-math.inf if math.isnan(w[t]) else w[t]), t))
    return sorted(list(range(sink)) + rank[:budget - sink - recent] + list(range(n - recent, n)))


def row_code(keep, n):
    """(entries before the first -1, the OR of the SA_IDX_* codes of what is wrong) of a list."""
    m, code, before = len(keep), 0, -2
    for i, v in enumerate(keep):
        if v == -1:
            m = min(m, i)
        elif v < -1:
            code |= 1
        elif before == -1:
            code |= 2
        elif v >= n:
            code |= 4
        elif v == before:
            code |= 16
        elif v < before:
            code |= 8
        before = v
    return m, code


def compact_row(plane, table_row, page_tokens, head, keep):
    """Move the rows ``plane[page, head, slot, ...]`` of one sequence: token i becomes keep[i]."""
    if not keep:
        return
    page, slot = token_places(table_row, max(keep) + 1, page_tokens)
    j = torch.tensor(keep)
    rows = plane[page[j], head, slot[j]].clone()
    i = torch.arange(len(keep))
    plane[page[i], head, slot[i]] = rows
