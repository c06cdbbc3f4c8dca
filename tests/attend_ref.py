"""Plain references of the batch planner (Python integers) and of the attention
over cached rows (64-bit floats), and the error bounds of the kernels."""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle

LOG2E = math.log2(math.e)
U_BF16 = 2.0 ** -8       # half a bf16 step, relative
U_FP32 = 2.0 ** -24


# ------------------------------------------------------------------ slot map
def slot_map(*, ratio, page_size, num_pages, lens, new_lens, page_table, free_pages, max_tokens,
             token_stride=0, depth=None):
    """The tables one token and one page at a time; ``new_lens`` None: the
    token stride.  Returns a dict of int32 arrays and the status bits."""
    S = len(lens)
    table = np.array(page_table, np.int32, copy=True).reshape(S, -1)
    width = table.shape[1]
    off = np.zeros((2, S), np.int32)
    start = np.full(S, -1, np.int32)
    loc = np.zeros(max_tokens, np.int32)
    pos = np.zeros(max_tokens, np.int32)
    req = np.full(max_tokens, -1, np.int32)
    status = asked = taken = first = made = refused = 0
    full = False
    up = lambda a, b: -(-a // b)
    for b in range(S):
        off[0, b] = b * token_stride if token_stride else first
        l = int(lens[b])
        n = int(token_stride if new_lens is None else new_lens[b])
        if l < 0:
            continue
        n = max(n, 0)
        have, want = up(l // ratio, page_size), up((l + n) // ratio, page_size)
        if want > width or l + n > 2 ** 31 - 1:
            status |= 4
            refused += 1
            continue
        if token_stride and n > token_stride:
            status |= 64
            refused += 1
            continue
        asked += want - have
        if want > have and asked > len(free_pages):
            status |= 128
            refused += 1
            continue
        if not token_stride and n and (full or first + n > max_tokens):
            full = True
            status |= 64
            refused += 1
            continue
        for k in range(have, want):
            table[b, k] = free_pages[asked - (want - k)]
        if want > have:
            taken = asked
        off[1, b], start[b] = n, l
        for j in range(n):
            t = int(off[0, b]) + j
            p = l + j
            req[t] = b
            pos[t] = p if depth is None else l + int(depth[t])
            if ratio == 1 or p % 2 == 1:
                c = p // ratio
                page = int(table[b, c // page_size])
                made += 1
                if 0 <= page < num_pages:
                    loc[t] = page * page_size + c % page_size
                else:
                    status |= 2
        if not token_stride:
            first += n
    totals = np.array([int(off[1].sum()), made, taken, refused], np.int32)
    return dict(offsets=off, start_pos=start, page_table=table, out_loc=loc, positions=pos,
                token_to_req=req, totals=totals), status


# ----------------------------------------------------------------- attention
def cached_rows(cache: np.ndarray, layout: str, page_size: int, table_row, count: int):
    """(values [count, 512] fp64, valid [count]) of logical rows 0 .. count - 1;
    a row with no page in the cache is not valid."""
    ids = np.arange(count)
    page = np.full(count, -1, np.int64)
    lp = ids // page_size
    inside = lp < len(table_row)
    page[inside] = np.asarray(table_row)[lp[inside]]
    valid = (page >= 0) & (page < cache.shape[0])
    slots = np.where(valid, page * page_size + ids % page_size, -1).astype(np.int32)
    rows, _ = oracle.dequant_gather(cache, layout, page_size, None, slots)
    f = (rows.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return torch.from_numpy(f), torch.from_numpy(valid)


def attend(q, rows, seen, scale, sink=None):
    """q [n, H, 512] fp64, rows [R, 512] fp64, seen [n, R] bool -> out, lse and
    their bounds (all fp64).  Rows no query sees are left out of the sums."""
    n, H, _ = q.shape
    if n > 1 and not torch.isfinite(rows).all():
        # a weight of 0 does not cancel a NaN: each token over its own rows
        each = [attend(q[t:t + 1], rows[seen[t]], seen[t:t + 1, seen[t]], scale, sink)
                for t in range(n)]
        return tuple(torch.cat(v) for v in zip(*each))
    used = seen.any(0)
    x = torch.where(used[:, None], rows, torch.zeros_like(rows))
    s = (q.reshape(n * H, 512) @ x.T).view(n, H, -1) * scale
    s = s.masked_fill(~seen[:, None, :], -math.inf)
    top = s.amax(2) if s.shape[2] else torch.full((n, H), -math.inf, dtype=torch.float64)
    sk = torch.full((H,), -math.inf, dtype=torch.float64) if sink is None else sink.double()
    m = torch.maximum(top, sk)
    base = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    w = torch.exp(s - base[..., None])
    den = w.sum(2) + torch.exp(sk - base)
    safe = torch.where(den == 0, torch.ones_like(den), den)      # NaN stays NaN
    w = w / safe[..., None]
    out = (w.view(n * H, -1) @ x).view(n, H, 512)
    lse = torch.where(den == 0, torch.full_like(den, -math.inf), base * LOG2E + torch.log2(safe))
    # Bounds.  A score is a 512-term fp32 sum of exact products, scaled once and
    # taken to the exponent of 2: its error is at most ds = (512 + 4) u32 sum
    # |q x| |scale|, and a weight's relative error ds (+ 4 u32 of the exponential)
    # on top of its rounding to bf16.  The division is by the sum of the rounded
    # weights, so a relative error d_r of weight w_r moves out by w_r d_r (x_r -
    # out): at most max|d_r| (sum w |x| + |out| sum w).  Rounding out adds half a
    # bf16 step; the fp32 sums over R rows R u32 relative (to sum w |x|).
    R = x.shape[0]
    ds = (516 * U_FP32 * abs(scale) * (q.abs().reshape(n * H, 512) @ x.abs().T)).view(n, H, R)
    ds = ds.masked_fill(~seen[:, None, :], 0).amax(2) if R else torch.zeros(n, H, dtype=torch.float64)
    ds = ds + (base.abs() + 4) * 4 * U_FP32
    wx = (w.view(n * H, -1) @ x.abs()).view(n, H, 512)
    d = (1.01 * U_BF16 + 2 * ds + 4 * U_FP32)[..., None]
    out_tol = d * (wx + out.abs()) + U_BF16 * 1.01 * out.abs() + (R + 16) * U_FP32 * wx + 1e-38
    lse_tol = LOG2E * (2 * ds + (R + 16) * U_FP32) + 4 * U_FP32 * lse.abs()
    return out, lse, out_tol, lse_tol


def check(got_out, got_lse, ref, what=""):
    """The kernel's outputs against ``attend``'s within its bounds."""
    out, lse, out_tol, lse_tol = ref
    g = got_out.double().cpu()
    assert torch.equal(torch.isnan(g), torch.isnan(out)), f"{what}: NaN pattern of out"
    bad = (g - out).abs() > out_tol
    assert not bad.any(), (f"{what}: out off at {int(bad.sum())} of {bad.numel()}, worst "
                           f"{((g - out).abs() / out_tol).nan_to_num().max():.3g} of the bound")
    if got_lse is not None:
        g = got_lse.double().cpu()
        same = (g == lse) | (torch.isnan(g) & torch.isnan(lse))
        bad = ~same & ~((g - lse).abs() <= lse_tol)
        assert not bad.any(), (f"{what}: lse off at {int(bad.sum())}, worst "
                               f"{((g - lse).abs() / lse_tol).nan_to_num().max():.3g} of the bound")
