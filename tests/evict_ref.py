"""Plain 64-bit references of the rotary table and rotation, of the attention
weights that cached rows collect, of the choice of rows and of their move, and
the error bounds of the kernels."""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle

LOG2E = math.log2(math.e)
U_FP32 = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U_FP32}


# -------------------------------------------------------------------- rotary
def speeds(rot, base, scaling="none", factor=1.0, original=0.0, beta_fast=32.0, beta_slow=1.0):
    """w_j of every pair, one at a time."""
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    w = [base ** (-2.0 * j / rot) for j in range(rot // 2)]
    if scaling == "linear":
        w = [x / factor for x in w]
    if scaling == "parts":
        pair = lambda turns: rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))
        lo = max(math.floor(pair(beta_fast)), 0)
        hi = min(math.ceil(pair(beta_slow)), rot - 1)
        for j in range(rot // 2):
            r = min(max((j - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            w[j] = w[j] * (1 - r) + w[j] / factor * r
    return np.array(w)


def table(n, first, rot, base, mscale=1.0, **kw):
    """The table and its bound: an angle's 64-bit roundings (its own size times
    2^-51, here and there), 64 products (2^-44), one rounding to fp32."""
    a = (np.arange(n, dtype=np.float64) + first)[:, None] * speeds(rot, base, **kw)
    out = np.stack([np.cos(a), np.sin(a)], 2).reshape(n, rot) * mscale
    slack = np.repeat(a * 2.0 ** -51, 2, axis=1) + 2.0 ** -44
    return out, U_FP32 * np.abs(out) * 1.01 + mscale * slack * 1.01


def rope(x, positions, freqs, offset, half, transpose):
    """x [T, H, D] (any type) -> its rotation in fp64 and the bound."""
    T, H, D = x.shape
    R = freqs.shape[1]
    out = x.double().clone()
    tol = torch.zeros_like(out)
    u = U[x.dtype]
    for j in range(R // 2):
        a, b = (offset + j, offset + R // 2 + j) if half else (offset + 2 * j, offset + 2 * j + 1)
        c = freqs[positions.long(), 2 * j].double()[:, None]
        s = freqs[positions.long(), 2 * j + 1].double()[:, None]
        if transpose:
            s = -s
        xa, xb = x[..., a].double(), x[..., b].double()
        out[..., a], out[..., b] = xa * c - xb * s, xa * s + xb * c
        # two fp32 products and their sum (at most 3 roundings), then one to the type
        for d, big in ((a, (xa * c).abs() + (xb * s).abs()), (b, (xa * s).abs() + (xb * c).abs())):
            tol[..., d] = 3 * U_FP32 * big * 1.01 + u * 1.01 * out[..., d].abs()
    if x.dtype == torch.float16:
        tol = tol + 2.0 ** -25                 # half of the least subnormal step
    return out, tol


# ------------------------------------------------------------------- weights
def weigh(q, lse, rows, valid, seen, scale):
    """q [n, H, 512] fp64, lse [n, H] fp32, rows [R, 512] fp64, seen [n, R] ->
    what each row collects and its bound.

    A score is an fp32 sum of 512 exact products, taken to the exponent of 2 by
    one fused product: d2 = 516 u sum |q x| scale log2(e) + 3 u (|score| + |lse|) in
    the exponent, a relative ln2 d2 + 4 u of a weight (2 u of them the
    exponential's); M weights are added in fp32, M u relative at most."""
    n, H, _ = q.shape
    fin = torch.isfinite(lse)
    x = torch.where(torch.isfinite(rows).all(1)[:, None], rows, torch.zeros_like(rows))
    use = valid & torch.isfinite(rows).all(1) & seen.any(0)
    qz = torch.where(fin[..., None], q, torch.zeros_like(q)).reshape(n * H, 512)
    s2 = (qz @ x.T).view(n, H, -1) * (scale * LOG2E)
    l2 = torch.where(fin, lse, torch.zeros_like(lse)).double()[..., None]
    w = torch.exp2(s2 - l2)
    w = torch.where(seen[:, None, :] & fin[..., None] & use, w, torch.zeros_like(w))
    d2 = 516 * U_FP32 * scale * LOG2E * (qz.abs() @ x.abs().T).view(n, H, -1)
    d2 = d2 + 3 * U_FP32 * (s2.abs() + l2.abs())
    rel = math.log(2) * d2 * 1.01 + 4 * U_FP32
    total = w.sum((0, 1))
    tol = (w * rel).sum((0, 1)) * 1.01 + (n * H + 16) * U_FP32 * total + 1e-37
    return total, tol


# -------------------------------------------------------------------- choice
def select(lens, weights, budgets, K, ratio, first, recent):
    """(kept [S, K], counts [S], kept_weights [S, K], status) by sorting."""
    S, W = weights.shape
    kept = np.full((S, K), -1, np.int32)
    counts = np.full(S, -1, np.int32)
    kw = np.zeros((S, K), np.float32)
    status = 0
    for b in range(S):
        if lens[b] < 0:
            continue
        n = int(lens[b]) // ratio
        if n > W:
            status |= 4
            continue
        B = int(budgets[b])
        if B < 0 or B > K:
            B = K
        ids = list(range(n))
        if n > B:
            f = min(first, B)
            g = min(recent, B - f)
            value = lambda r: -math.inf if math.isnan(weights[b, r]) else float(weights[b, r])
            # (a NaN below -inf, equals by the lower row)
            mid = sorted(range(f, n - g), key=lambda r: (math.isnan(weights[b, r]), -value(r), r))
            ids = sorted(list(range(f)) + mid[:B - f - g] + list(range(n - g, n)))
        counts[b] = len(ids)
        kept[b, :len(ids)] = ids
        kw[b, :len(ids)] = weights[b, ids]
    return kept, counts, kw, status


# ---------------------------------------------------------------------- move
def compact(cache, layout, page_size, ratio, lens, kept, counts, table, free, freed_cap=None,
            kept_weights=None, weights=None):
    """A row and a page at a time; arrays come back as new ones."""
    db, sb, _, _ = oracle.layout_bytes(layout)
    cache, out = cache.copy(), cache.copy()
    P = cache.shape[0]
    S, width = table.shape
    new_table, new_lens = np.zeros_like(table), np.array(lens, np.int32)
    weights = None if weights is None else weights.copy()
    freed, status = [], 0
    taken = given = dropped = refused = asked_take = asked_give = 0
    up = lambda a, b: -(-a // b)
    part = lambda img, page, r: (img[page, r * db:(r + 1) * db],
                                 img[page, page_size * db + r * sb:page_size * db + (r + 1) * sb])
    for b in range(S):
        n = int(lens[b]) // ratio if lens[b] >= 0 else 0
        c = int(counts[b])
        held = up(n, page_size)
        new_table[b, :min(held, width)] = table[b, :min(held, width)]
        if not 0 <= c < n:
            continue
        if held > width or c > kept.shape[1] or (weights is not None and c > weights.shape[1]):
            status |= 4
            refused += 1
            continue
        need = up(c, page_size)
        asked_take += need
        asked_give += held
        if asked_take > min(len(free), P - 1) or (freed_cap is not None and asked_give > freed_cap):
            status |= 128
            refused += 1
            continue
        pages = [int(free[taken + k]) for k in range(need)]
        new_table[b] = 0
        new_table[b, :need] = pages
        for i in range(c):
            r, to = int(kept[b, i]), pages[i // page_size]
            src = None
            if not 0 <= r < n:
                status |= 1
            else:
                page = int(table[b, r // page_size])
                if 0 <= page < P:
                    src = part(cache, page, r % page_size)
                else:
                    status |= 2
            if not 1 <= to < P:
                status |= 2
                continue
            for dst, k in zip(part(out, to, i % page_size), (0, 1)):
                dst[:] = 0 if src is None else src[k]
        if weights is not None:
            weights[b, :c] = kept_weights[b, :c]
        freed += [int(v) for v in table[b, :held]]
        new_lens[b] = c * ratio + int(lens[b]) % ratio
        taken, given, dropped = taken + need, given + held, dropped + n - c
    return dict(cache=out, new_table=new_table, new_lens=new_lens, weights=weights, freed=freed,
                totals=[taken, given, min(dropped, 2 ** 31 - 1), refused], status=status)
