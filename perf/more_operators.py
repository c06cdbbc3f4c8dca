"""Timed cases of the rotary positions (``kvc_rope_table``, ``kvc_rope_rows``)
and of the eviction from the paged cache by accumulated attention weight
(``kvc_weigh_prefill``, ``kvc_weigh_tree``, ``kvc_evict_select``,
``kvc_cache_compact``), with the plain forms they are compared with.

A case is a dict; ``prepare`` makes what a serving program holds before the
call, ``run`` makes one call -- elementary torch operations, or the library's
entry points when ``own`` is set -- and ``exact`` evaluates the definitions
again in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DIM = 512
ROW = {"V4": (576, 8), "V41": (512, 16), "V41_FP4": (256, 32)}   # data, scale bytes per row
LOG2E = math.log2(math.e)
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the table a server makes when it starts, 4,096 positions, no scaling
        dict(name="table-4096", op="table", n=4096, first=0, rot=64, base=10000.0, kind="none",
             factor=1.0, original=0, mscale=1.0),
        # the same for contexts of a million tokens, scaled by parts from 65,536
        dict(name="table-1m-parts", op="table", n=1 << 20, first=0, rot=64, base=10000.0,
             kind="parts", factor=16.0, original=65536, mscale=1.2),
        # a decode step: the 64 rope dims of 64 tokens' 64 query heads of 512
        dict(name="rope-decode-64x64", op="rope", tokens=64, heads=64, dim=512, rot=64, off=448,
             part=1, half=0, transpose=0, type="bf16", max_pos=131072),
        # a prompt of 8,192 tokens, 128 heads: whole heads, the attention's outputs turned back
        dict(name="rope-prompt-8192x128", op="rope", tokens=8192, heads=128, dim=512, rot=64,
             off=448, part=0, half=0, transpose=1, type="bf16", max_pos=131072),
        # one decoded token of one request, few heads: latency
        dict(name="weigh-decode-1x16-v41", op="weigh", form="tree", layout="V41", slots=1, draft=1,
             heads=16, page=64, ratio=1, held_lo=1000, held_hi=1000, tree=0),
        # a decode batch with 64 heads over FP4 rows
        dict(name="weigh-decode-64x64-fp4", op="weigh", form="tree", layout="V41_FP4", slots=64,
             draft=1, heads=64, page=64, ratio=1, held_lo=2000, held_hi=16000, tree=0),
        # a ragged prefill batch over its own pooled rows
        dict(name="weigh-prefill-16-fp4", op="weigh", form="prefill", layout="V41_FP4", slots=16,
             heads=32, page=128, ratio=2, new_lo=1500, new_hi=2600, held_lo=0, held_hi=0),
        # one long prompt with every head
        dict(name="weigh-prefill-8192-v41", op="weigh", form="prefill", layout="V41", slots=1,
             heads=128, page=64, ratio=1, new_lo=8192, new_hi=8192, held_lo=0, held_hi=0),
        # 64 requests that have grown past 4,096 rows are cut back to them
        dict(name="select-64x16k", op="select", slots=64, rows_lo=4200, rows_hi=16384, budget=4096,
             ratio=1, first=4, recent=512, ties=0),
        # one request of a million rows cut to a sixteenth
        dict(name="select-1x1m", op="select", slots=1, rows_lo=1048500, rows_hi=1048500,
             budget=65536, ratio=1, first=16, recent=4096, ties=0),
        # one short request, its rows moved to pages of their own
        dict(name="compact-1x1100-fp4", op="compact", layout="V41_FP4", slots=1, page=64, ratio=1,
             rows_lo=1100, rows_hi=1100, budget=1024),
        # the 64 requests above, compacted
        dict(name="compact-64x16k-v41", op="compact", layout="V41", slots=64, page=64, ratio=1,
             rows_lo=4200, rows_hi=16384, budget=4096),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["table", "rope", "rope", "weigh", "weigh", "weigh", "select", "select",
                     "compact", "compact"])
    if op == "table":
        kind = rng.choice(["none", "linear", "base", "parts"])
        rot = rng.choice([64, 64, 32, 128, 2 * _spread(rng, 2, 128)])
        return dict(op=op, n=_spread(rng, 1000, (1 << 26) // rot), first=rng.choice([0, 0, 40001]),
                    rot=rot, base=rng.choice([10000.0, 160000.0, 500000.0]), kind=kind,
                    factor=1.0 if kind == "none" else rng.choice([2.0, 4.0, 16.0, 40.0]),
                    original=rng.choice([4096, 65536]) if kind == "parts" else 0,
                    mscale=rng.choice([1.0, 1.0, 1.2]))
    if op == "rope":
        dim = rng.choice([512, 512, 128, 192, 64, 8 * _spread(rng, 2, 72), _spread(rng, 5, 300)])
        rot = min(dim // 2 * 2, rng.choice([64, 64, 128, 2 * _spread(rng, 1, 64)]))
        off = rng.choice([dim - rot, 0, rng.randint(0, dim - rot)])
        heads = rng.choice([1, 16, 64, 128, _spread(rng, 1, 100)])
        kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        most = (1 << 29) // (dim * heads * (2 if kind == "fp32" else 1))
        return dict(op=op, tokens=_spread(rng, 1, min(20000, most)), heads=heads, dim=dim, rot=rot,
                    off=off, part=int(rng.random() < 0.5), half=int(rng.random() < 0.5),
                    transpose=int(rng.random() < 0.5), type=kind,
                    max_pos=rng.choice([8192, 131072, 524288]))
    layout = rng.choice(["V4", "V41", "V41_FP4"])
    page = rng.choice([1, 16, 64, 64, 128])
    ratio = rng.choice([1, 2])
    if op == "weigh":
        heads = rng.choice([8, 16, 32, 64, 128, _spread(rng, 5, 100)])
        budget = 5e8                     # pairs of a query and a row, at most
        if rng.random() < 0.6:
            draft = rng.choice([1, 1, 4, _spread(rng, 1, 64)])
            slots = _spread(rng, 1, 200)
            tree = int(draft > 1 and rng.random() < 0.6)
            top = int(max(200, min(200000, budget / (slots * draft * heads))))
            hi = _spread(rng, 200, top)
            return dict(op=op, form="tree", layout=layout, slots=slots, draft=draft, heads=heads,
                        page=page, ratio=1 if tree else ratio, held_lo=_spread(rng, 64, hi),
                        held_hi=hi, tree=tree)
        slots = _spread(rng, 1, 12)
        hi = _spread(rng, 40, int(max(60, min(6000, math.sqrt(budget / (slots * heads))))))
        start = 0 if rng.random() < 0.5 else _spread(rng, 1, int(max(10, min(
            40000, budget / (slots * hi * heads)))))
        return dict(op=op, form="prefill", layout=layout, slots=slots, heads=heads, page=page,
                    ratio=ratio, new_lo=max(1, hi // 3), new_hi=hi, held_lo=start // 3,
                    held_hi=start)
    slots = _spread(rng, 1, 200)
    hi = _spread(rng, 40, int((1 << 20) / slots) if op == "select" else int((1 << 19) / slots))
    budget = _spread(rng, 1, hi if op == "select" else max(1, min(hi, (1 << 18) // slots)))
    if op == "select":
        first = min(budget, rng.choice([0, 4, 16]))
        return dict(op=op, slots=slots, rows_lo=max(1, hi // 3), rows_hi=hi, budget=budget, ratio=ratio,
                    first=first, recent=rng.choice([0, (budget - first) // 4, budget]),
                    ties=int(rng.random() < 0.3))
    return dict(op=op, layout=layout, slots=slots, page=page, ratio=ratio, rows_lo=max(1, hi // 3),
                rows_hi=hi, budget=budget)


def _case_rng(case, what=""):
    """Lengths are a function of the case alone: the work of a case does not
    depend on the seed of its values."""
    return random.Random(what + repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case):
    """(held, new) token counts of each slot."""
    rng = _case_rng(case)
    held = [rng.randint(case["held_lo"], case["held_hi"]) for _ in range(case["slots"])]
    if case["form"] == "tree":
        new = [case["draft"]] * case["slots"]
    else:
        new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["slots"])]
    return held, new


def _row_counts(case):
    rng = _case_rng(case)
    return [rng.randint(case["rows_lo"], case["rows_hi"]) for _ in range(case["slots"])]


def _visible(case, pos):
    return (pos + 1) // case["ratio"]


def work(case):
    op = case["op"]
    if op == "table":
        return {"bytes": 4 * case["rot"] * case["n"], "flops": 0}
    if op == "rope":
        width = case["rot"] if case["part"] else case["dim"]
        size = 4 if case["type"] == "fp32" else 2
        # the table's rows and the positions once a token, the rotated (or whole) heads in and out
        return {"bytes": case["tokens"] * (4 + 4 * case["rot"] + 2 * size * case["heads"] * width),
                "flops": 3 * case["tokens"] * case["heads"] * case["rot"]}
    if op == "weigh":
        held, new = _lengths(case)
        h, rb = case["heads"], sum(ROW[case["layout"]])
        rows = pairs = tokens = 0
        masks = _tree_masks(case) if case.get("tree") else None
        for b, (l, n) in enumerate(zip(held, new)):
            tokens += n
            rows += (l + n) // case["ratio"]
            if masks is not None:
                pairs += sum(l + bin(m).count("1") for m in masks[b])
            else:
                pairs += sum(_visible(case, l + j) for j in range(n))
        table = 4 * sum(-(-((l + n) // case["ratio"]) // case["page"]) for l, n in zip(held, new))
        # the rows with their weight before and after, queries and lse
        return {"bytes": rows * (rb + 8) + table + tokens * h * (2 * DIM + 4),
                "flops": 2 * DIM * h * pairs}
    rows = _row_counts(case)
    kept = [min(r, case["budget"]) for r in rows]
    if op == "select":
        return {"bytes": 4 * sum(rows) + 8 * sum(kept), "flops": 0}
    rb = sum(ROW[case["layout"]])
    moved = sum(k for k, r in zip(kept, rows) if k < r)
    pages = sum(-(-r // case["page"]) for r in rows)
    # ids, kept rows in and out with their weights; the old table, the new one, the pages given back
    return {"bytes": moved * (4 + 2 * rb + 8) + 12 * pages, "flops": 0}


# ------------------------------------------------------------------ inputs
def _tree_masks(case):
    """Ancestor masks [slots][draft]: every drafted token hangs under an
    earlier one or under the context."""
    rng = _case_rng(case, "tree")
    out = []
    for _ in range(case["slots"]):
        m = []
        for j in range(case["draft"]):
            parent = rng.randint(max(-1, j - 6), j - 1)
            m.append((m[parent] if parent >= 0 else 0) | 1 << j)
        out.append(m)
    return out


def _quantize(rows, layout):
    """Latent rows [n, 512] fp32 -> their data and scale bytes."""
    n = rows.shape[0]

    def fp8(x, group):
        g = x.view(n, -1, group)
        e = torch.ceil(torch.log2(torch.clamp(g.abs().amax(2) / 448, min=1e-4))).to(torch.int32)
        scale = ((e + 127) << 23).view(torch.float32)
        codes = (g / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        return codes.reshape(n, -1), (e + 127).to(torch.uint8)

    if layout == "V41":
        return fp8(rows, 32)
    if layout == "V4":
        codes, e = fp8(rows[:, :448].contiguous(), 64)
        rope = rows[:, 448:].to(torch.bfloat16).contiguous().view(torch.uint8)
        return torch.cat([codes, rope], 1), torch.cat([e, torch.zeros_like(e[:, :1])], 1)
    g = rows.view(n, 32, 16)
    s = (g.abs().amax(2) / 6).to(torch.float8_e4m3fn)
    y = g / s.to(torch.float32)[..., None].clamp(min=1e-9)
    grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=rows.device)
    mag = torch.bucketize(y.abs(), grid).to(torch.uint8).view(n, 512)
    code = mag | ((rows < 0).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4), s.view(torch.uint8)


def _pages(counts, page, gen, dev):
    """A page table for `counts[b]` rows of every slot, pages in random order
    from 1 on, and the number of pages used."""
    pages = [max(1, -(-c // page)) for c in counts]
    total = sum(pages)
    order = (torch.randperm(total, generator=gen, device=dev) + 1).to(torch.int32)
    have = torch.tensor(pages, device=dev)
    table = torch.zeros(len(counts), max(pages), dtype=torch.int32, device=dev)
    table[torch.arange(max(pages), device=dev) < have[:, None]] = order
    return table, total


def _cache(case, counts, gen, dev):
    """A paged cache holding `counts[b]` latent rows of every slot, arbitrary
    bytes elsewhere, and the page table."""
    db, sb = ROW[case["layout"]]
    ps = case["page"]
    table, total = _pages(counts, ps, gen, dev)
    stride = -(-ps * (db + sb) // 16) * 16
    cache = torch.randint(0, 256, (total + 1, stride), generator=gen, device=dev, dtype=torch.uint8)
    data = cache[:, :ps * db].unflatten(1, (ps, db))
    scale = cache[:, ps * db:ps * (db + sb)].unflatten(1, (ps, sb))
    for b, c in enumerate(counts):
        for r0 in range(0, c, 1 << 17):
            r = torch.arange(r0, min(c, r0 + (1 << 17)), device=dev)
            rows = torch.randn(r.numel(), DIM, generator=gen, device=dev)
            rows = rows / rows.pow(2).mean(1, keepdim=True).sqrt()
            at = table[b, r // ps].long(), r % ps
            data[at], scale[at] = _quantize(rows, case["layout"])
    return cache, table


def _prepare_rope(case, gen, dev):
    T, h, dim = case["tokens"], case["heads"], case["dim"]
    kind = TYPES[case["type"]]
    x = torch.randn(T, h, dim, generator=gen, device=dev).to(kind)
    out = torch.zeros_like(x)
    pos = torch.randint(0, case["max_pos"], (T,), generator=gen, device=dev, dtype=torch.int32)
    w = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=dev) / case["rot"])
    a = torch.arange(case["max_pos"], dtype=torch.float64, device=dev)[:, None] * w
    freqs = torch.stack([a.cos(), a.sin()], 2).flatten(1).float()
    return dict(case=case, x=x, out=out, pos=pos, freqs=freqs)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 6007 + 29)
    op = case["op"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    if op == "table":
        # (the seed moves where the table begins: its only input)
        return dict(case=case, first=case["first"] + seed % 64,
                    out=torch.zeros(case["n"], case["rot"], device=dev))
    if op == "rope":
        return _prepare_rope(case, gen, dev)
    if op == "weigh":
        held, new = _lengths(case)
        r = case["ratio"]
        counts = [(l + n) // r for l, n in zip(held, new)]
        cache, table = _cache(case, counts, gen, dev)
        T, h = sum(new), case["heads"]
        q = (torch.randn(T, h, DIM, generator=gen, device=dev) * 1.5).to(torch.bfloat16)
        st = dict(case=case, held=held, new=new, cache=cache, table=table, q=q, start=i32(held),
                  scale=DIM ** -0.5)
        first = [0]
        for n in new[:-1]:
            first.append(first[-1] + n)
        st["first"] = first
        if case["form"] == "prefill":
            st["offsets"] = i32([first, new])
        if case.get("tree"):
            masks = _tree_masks(case)
            sees = [l + bin(m).count("1") for l, row in zip(held, masks) for m in row]
            st["mask"] = torch.tensor([[m - (1 << 64) if m >> 63 else m for m in row] for row in masks],
                                      dtype=torch.int64, device=dev)
        else:
            sees = [(l + j + 1) // r for l, n in zip(held, new) for j in range(n)]
        # the log-sum-exp of scores of standard deviation 1.5 over the rows a token
        # sees, as its heads have it
        lse = torch.log2(torch.tensor(sees, dtype=torch.float32, device=dev))[:, None] + 1.125 * LOG2E
        st["lse"] = lse + 0.1 * torch.randn(T, h, generator=gen, device=dev)
        W = max(max(counts), 1)
        st["prev"] = torch.rand(case["slots"], W, generator=gen, device=dev) * 4
        st["weights"] = torch.zeros(case["slots"], W, device=dev)
        return st
    rows = _row_counts(case)
    S, W = case["slots"], max(rows)
    # accumulated weights: a heavy tail, some rows with none
    w = torch.exp(1.5 * torch.randn(S, W, generator=gen, device=dev))
    w = torch.where(torch.rand(S, W, generator=gen, device=dev) < 0.05, 0.0, w)
    K = min(case["budget"], W)
    lens = i32([r * case["ratio"] + case["ratio"] - 1 for r in rows])
    if op == "select":
        if case["ties"]:
            w = torch.round(w * 4) / 4
        e = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device=dev)
        return dict(case=case, rows=rows, lens=lens, weights=w, kept=e(S, K), counts=e(S),
                    kept_weights=e(S, K, t=torch.float32))
    ps, (db, sb) = case["page"], ROW[case["layout"]]
    table, used = _pages(rows, ps, gen, dev)
    fresh = sum(-(-min(r, K) // ps) for r in rows if r > K) + 7
    stride = -(-ps * (db + sb) // 16) * 16
    cache = torch.randint(0, 256, (used + 1 + fresh, stride), generator=gen, device=dev,
                          dtype=torch.uint8)
    free = (torch.randperm(fresh, generator=gen, device=dev) + 1 + used).to(torch.int32)
    # a selection: every row its chance, the rows in order
    col = torch.arange(W, device=dev)
    n = i32(rows)
    key = torch.where(col < n[:, None], w, -1.0)
    chosen = key.topk(K, dim=1).indices
    chosen = torch.where(chosen < n[:, None], chosen, W).sort(1).values
    kept = torch.where(chosen < W, chosen, -1).to(torch.int32)
    kept_weights = torch.where(kept >= 0, w.gather(1, kept.clamp(min=0).long()), 0.0)
    return dict(case=case, rows=rows, lens=lens, cache=cache, table=table, free=free, kept=kept,
                counts=torch.minimum(n, i32(K)), kept_weights=kept_weights, weights=w,
                new_table=torch.zeros_like(table), new_lens=torch.zeros_like(lens),
                freed=torch.zeros(used, dtype=torch.int32, device=dev),
                totals=torch.zeros(4, dtype=torch.int32, device=dev))


# -------------------------------------------------------------- plain forms
def _plain_table(st):
    c = st["case"]
    R, dev = c["rot"], st["out"].device
    j = torch.arange(R // 2, dtype=torch.float64, device=dev)
    base = c["base"]
    if c["kind"] == "base":
        base = base * c["factor"] ** (R / (R - 2))
    w = torch.exp(-2 * j / R * math.log(base))
    if c["kind"] == "linear":
        w = w / c["factor"]
    if c["kind"] == "parts":
        at = lambda turns: R * math.log(c["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), R - 1)
        ramp = ((j - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        w = w / c["factor"] * ramp + w * (1 - ramp)
    a = torch.arange(st["first"], st["first"] + c["n"], dtype=torch.float64, device=dev)[:, None] * w
    return torch.stack([a.cos() * c["mscale"], a.sin() * c["mscale"]], 2).flatten(1).float()


def _plain_rope(st):
    c = st["case"]
    off, R = c["off"], c["rot"]
    x = st["x"][..., off:off + R].float()
    f = st["freqs"][st["pos"].long()].view(-1, 1, R // 2, 2)
    cos, sin = f[..., 0], -f[..., 1] if c["transpose"] else f[..., 1]
    if c["half"]:
        a, b = x[..., :R // 2], x[..., R // 2:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], 2)
    else:
        a, b = x[..., 0::2], x[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], 3).flatten(2)
    if not c["part"]:
        st["out"].copy_(st["x"])
    st["out"][..., off:off + R] = y.to(st["out"].dtype)
    return st["out"]


def _rows(st, b, count, dtype):
    """Cached rows 0 .. count - 1 of slot b in `dtype` (exact in every layout)."""
    c = st["case"]
    db, sb = ROW[c["layout"]]
    ps = c["page"]
    pages = st["cache"][st["table"][b, :-(-count // ps)].long()]
    data = pages[:, :ps * db].reshape(-1, db)[:count]
    scale = pages[:, ps * db:ps * (db + sb)].reshape(-1, sb)[:count]
    e4m3 = lambda x: x.contiguous().view(torch.float8_e4m3fn).to(dtype)
    if c["layout"] == "V41_FP4":
        grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                            dtype=dtype, device=data.device)
        codes = torch.stack([data & 15, data >> 4], 2).reshape(count, 32, 16)
        return (grid[codes.int()] * e4m3(scale)[..., None]).view(count, DIM)
    power = (scale.int() << 23).view(torch.float32).to(dtype)
    if c["layout"] == "V41":
        return (e4m3(data).view(count, 16, 32) * power[..., None]).view(count, DIM)
    nope = (e4m3(data[:, :448]).view(count, 7, 64) * power[:, :7, None]).reshape(count, 448)
    return torch.cat([nope, data[:, 448:].contiguous().view(torch.bfloat16).to(dtype)], 1)


def _plain_weigh(st):
    c = st["case"]
    q, h, dev = st["q"], c["heads"], st["q"].device
    out = st["weights"]
    for b, (l, n, t0) in enumerate(zip(st["held"], st["new"], st["first"])):
        count = (l + n) // c["ratio"]
        x = _rows(st, b, max(count, 1), torch.float32)[:count]
        total = torch.zeros(count, device=dev)
        step = max(1, (1 << 29) // max(1, count * h))
        for j0 in range(0, n, step):
            j1 = min(n, j0 + step)
            top = count if c.get("tree") else _visible(c, l + j1 - 1)
            s = (q[t0 + j0:t0 + j1].float().view(-1, DIM) @ x[:top].T).view(j1 - j0, h, top)
            row = torch.arange(top, device=dev)
            if c.get("tree"):
                seen = (st["mask"][b, j0:j1, None] >> (row - l).clamp(0, 63)) & 1
                seen = (row < l) | (seen == 1)
            else:
                limit = (torch.arange(l + j0, l + j1, device=dev) + 1) // c["ratio"]
                seen = row < limit[:, None]
            p = torch.exp2(s * (st["scale"] * LOG2E) - st["lse"][t0 + j0:t0 + j1, :, None])
            total[:top] += torch.where(seen[:, None, :], p, 0.0).sum((0, 1))
        # rows that this call's tokens completed begin at nothing
        old = torch.where(torch.arange(count, device=dev) < l // c["ratio"], st["prev"][b, :count], 0.0)
        out[b, :count] = 0.5 * old + total
    return out


def _plain_select(st):
    c = st["case"]
    w = st["weights"]
    S, W = w.shape
    K = st["kept"].shape[1]
    n = st["lens"][:, None] // c["ratio"]
    count = n.clamp(max=K)
    col = torch.arange(W, device=w.device)
    first = min(c["first"], K)
    recent = min(c["recent"], K - first)
    held = (n <= K) | (col < first) | (col >= n - recent)
    key = torch.where(held, math.inf, w)
    key = torch.where(col < n, key, -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :K]
    live = torch.arange(K, device=w.device) < count
    ids = torch.where(live, order, W).sort(1).values
    st["kept"].copy_(torch.where(live, ids, -1))
    st["counts"].copy_(count[:, 0])
    st["kept_weights"].copy_(torch.where(live, w.gather(1, ids.clamp(max=W - 1)), 0.0))
    return dict(kept=st["kept"], counts=st["counts"], kept_weights=st["kept_weights"])


def _plain_compact(st):
    c = st["case"]
    ps, (db, sb) = c["page"], ROW[c["layout"]]
    table, counts, kept = st["table"], st["counts"].long(), st["kept"].long()
    dev = table.device
    n = st["lens"].long() // c["ratio"]
    cut = counts < n
    take = torch.where(cut, -(-counts // ps), 0)
    give = torch.where(cut, -(-n // ps), 0)
    col = torch.arange(table.shape[1], device=dev)
    place = (take.cumsum(0) - take)[:, None] + col
    fresh = st["free"][place.clamp(max=st["free"].numel() - 1)]
    held = torch.where(col < -(-n // ps)[:, None], table, 0)
    st["new_table"].copy_(torch.where(cut[:, None], torch.where(col < take[:, None], fresh, 0), held))
    # kept rows to their places in the new pages
    i = torch.arange(kept.shape[1], device=dev)
    b, i = torch.nonzero(cut[:, None] & (i < counts[:, None]), as_tuple=True)
    src = kept[b, i]
    at = st["new_table"][b, i // ps].long(), i % ps
    frm = table[b, src // ps].long(), src % ps
    data = st["cache"][:, :ps * db].unflatten(1, (ps, db))
    scale = st["cache"][:, ps * db:ps * (db + sb)].unflatten(1, (ps, sb))
    data[at] = data[frm]
    scale[at] = scale[frm]
    st["weights"][b, i] = st["kept_weights"][b, i]
    st["new_lens"].copy_(torch.where(cut, counts * c["ratio"] + st["lens"] % c["ratio"], st["lens"]))
    back = col < give[:, None]
    st["freed"][(give.cumsum(0) - give)[:, None].add(col)[back]] = table[back]
    st["totals"].copy_(torch.stack([take.sum(), give.sum(), torch.where(cut, n - counts, 0).sum(),
                                    0 * take.sum()]))
    return {k: st[k] for k in ("cache", "new_table", "new_lens", "weights", "freed", "totals")}


PLAIN = dict(table=_plain_table, rope=_plain_rope, weigh=_plain_weigh, select=_plain_select,
             compact=_plain_compact)


def run(state):
    c = state["case"]
    if not own:
        return PLAIN[c["op"]](state)
    import fp8_fp4_quantized_amd as kvc
    if c["op"] == "table":
        kvc.kvc_rope_table(state["out"], first=state["first"], base=c["base"], scaling=c["kind"],
                           factor=c["factor"], original=c["original"], mscale=c["mscale"])
        return state["out"]
    if c["op"] == "rope":
        x, out, off = state["x"], state["out"], c["off"]
        if c["part"]:
            x, out, off = x[..., off:off + c["rot"]], out[..., off:off + c["rot"]], 0
        kvc.kvc_rope_rows(x, state["pos"], state["freqs"], out, offset=off, half=bool(c["half"]),
                          transpose=bool(c["transpose"]))
        return state["out"]
    if c["op"] == "weigh":
        handle = kvc.Cache(state["cache"], c["layout"], c["page"])
        kw = dict(scale=state["scale"], ratio=c["ratio"], prev=state["prev"], decay=0.5)
        if c["form"] == "tree":
            kvc.kvc_weigh_tree(handle, state["q"], state["lse"], state["start"], state["table"],
                               state["weights"], draft_len=c["draft"], tree=state.get("mask"), **kw)
        else:
            kvc.kvc_weigh_prefill(handle, state["q"], state["lse"], state["offsets"], state["start"],
                                  state["table"], state["weights"], **kw)
        return state["weights"]
    if c["op"] == "select":
        kvc.kvc_evict_select(state["lens"], state["weights"], state["kept"], state["counts"],
                             budget=state["kept"].shape[1], ratio=c["ratio"], first=c["first"],
                             recent=c["recent"], kept_weights=state["kept_weights"])
        return {k: state[k] for k in ("kept", "counts", "kept_weights")}
    kvc.kvc_cache_compact(kvc.Cache(state["cache"], c["layout"], c["page"]), state["lens"],
                          state["kept"], state["counts"], state["table"], state["free"],
                          state["new_table"], state["new_lens"], ratio=c["ratio"],
                          kept_weights=state["kept_weights"], weights=state["weights"],
                          freed=state["freed"], totals=state["totals"])
    return {k: state[k] for k in ("cache", "new_table", "new_lens", "weights", "freed", "totals")}


# ------------------------------------------------------------------- 64 bits
def _exact_table(st):
    c = st["case"]
    R, f = c["rot"], c["factor"]
    base = np.float64(c["base"])
    if c["kind"] == "base":
        base = np.float64(c["base"]) * np.power(np.float64(f), np.float64(R) / (R - 2))
    w = np.array([np.power(base, -2.0 * j / R) for j in range(R // 2)], dtype=np.float64)
    if c["kind"] == "linear":
        w /= f
    if c["kind"] == "parts":
        # pairs that make 32 turns or more over the original context keep their
        # speed, pairs that make one or less are slowed down
        def pair_of(turns):
            return R * (np.log(c["original"]) - np.log(2 * np.pi * turns)) / (2 * np.log(base))
        a, z = max(int(np.floor(pair_of(32))), 0), min(int(np.ceil(pair_of(1))), R - 1)
        slow = np.clip((np.arange(R // 2) - a) / (z - a if z > a else 0.001), 0, 1)
        w = w * (1 - slow) + w / f * slow
    p = np.arange(c["n"], dtype=np.float64) + st["first"]
    out = np.empty((c["n"], R))
    for j in range(R // 2):
        out[:, 2 * j] = np.cos(p * w[j]) * c["mscale"]
        out[:, 2 * j + 1] = np.sin(p * w[j]) * c["mscale"]
    return torch.from_numpy(out)


def _exact_rope(st):
    c = st["case"]
    off, R = c["off"], c["rot"]
    x = st["x"].double()
    pairs = x[..., off:off + R]
    pairs = pairs.unflatten(2, (2, R // 2)).transpose(2, 3) if c["half"] else pairs.unflatten(2, (R // 2, 2))
    turn = torch.view_as_complex(st["freqs"][st["pos"].long()].double().unflatten(1, (R // 2, 2)))
    z = torch.view_as_complex(pairs.contiguous()) * (turn.conj() if c["transpose"] else turn)[:, None]
    z = torch.view_as_real(z.resolve_conj())
    y = torch.zeros_like(x) if c["part"] else x
    y[..., off:off + R] = (z.transpose(2, 3) if c["half"] else z).flatten(2)
    return y


def _exact_weigh(st):
    c = st["case"]
    q, h = st["q"], c["heads"]
    out = torch.zeros(st["weights"].shape, dtype=torch.float64, device=q.device)
    masks = _tree_masks(c) if c.get("tree") else None
    t = 0
    for b, (l, n) in enumerate(zip(st["held"], st["new"])):
        count = (l + n) // c["ratio"]
        if count:
            rows = _rows(st, b, count, torch.float64)
            out[b, :l // c["ratio"]] = 0.5 * st["prev"][b, :l // c["ratio"]].double()
            width = max(1, (1 << 27) // (count * h))
            for a in range(0, n, width):
                z = min(n, a + width)
                sees = torch.zeros(z - a, count, dtype=torch.float64, device=q.device) - math.inf
                if masks is None:
                    for j in range(a, z):
                        sees[j - a, :(l + j + 1) // c["ratio"]] = 0
                else:
                    sees[:, :l] = 0
                    for j in range(a, z):
                        for i in range(c["draft"]):
                            if masks[b][j] >> i & 1:
                                sees[j - a, l + i] = 0
                logit = torch.matmul(q[t + a:t + z].reshape(-1, DIM).double(), rows.T.contiguous())
                logit = logit.view(z - a, h, count) * st["scale"] + sees[:, None, :]
                # (a token that sees no row has lse = -inf)
                norm = st["lse"][t + a:t + z].double().clamp(min=-1e300) * math.log(2)
                out[b, :count] += torch.exp(logit - norm[..., None]).sum(dim=(0, 1))
        t += n
    return out


def _exact_select(st):
    c = st["case"]
    w = st["weights"].cpu().numpy()
    S, K = st["kept"].shape
    kept, counts = np.full((S, K), -1, np.int32), np.zeros(S, np.int32)
    kept_weights = np.zeros((S, K))
    for b, n in enumerate(st["rows"]):
        keep = np.ones(n, bool)
        if n > K:
            f = min(c["first"], K)
            g = min(c["recent"], K - f)
            mid = np.arange(f, n - g)
            best = np.lexsort((mid, -w[b, f:n - g].astype(np.float64)))[:K - f - g]
            keep[f:n - g] = False
            keep[mid[best]] = True
        ids = np.flatnonzero(keep)
        counts[b] = len(ids)
        kept[b, :len(ids)] = ids
        kept_weights[b, :len(ids)] = w[b, ids]
    return dict(kept=torch.from_numpy(kept), counts=torch.from_numpy(counts),
                kept_weights=torch.from_numpy(kept_weights))


def _exact_compact(st):
    c = st["case"]
    r, ps, (db, sb) = c["ratio"], c["page"], ROW[c["layout"]]
    cache, table = st["cache"].cpu().numpy().copy(), st["table"].cpu().numpy()
    free, kept, counts = (st[k].cpu().numpy() for k in ("free", "kept", "counts"))
    new_table, freed = np.zeros_like(table), st["freed"].cpu().numpy().copy()
    weights = st["weights"].cpu().numpy().astype(np.float64)
    kept_weights = st["kept_weights"].cpu().numpy()
    new_lens, taken, given, dropped = [], 0, 0, 0
    for b, n in enumerate(st["rows"]):
        old, k = -(-n // ps), int(counts[b])
        length = n * r + r - 1
        if k >= n:
            new_table[b, :old] = table[b, :old]
            new_lens.append(length)
            continue
        for page in range(-(-k // ps)):
            new_table[b, page] = free[taken + page]
        to, frm = np.arange(k), kept[b, :k]
        for size, base in ((db, 0), (sb, ps * db)):
            dst = base + to % ps * size
            src = base + frm % ps * size
            for e in range(size):
                cache[new_table[b, to // ps], dst + e] = cache[table[b, frm // ps], src + e]
        weights[b, :k] = kept_weights[b, :k]
        freed[given:given + old] = table[b, :old]
        taken, given, dropped = taken + -(-k // ps), given + old, dropped + n - k
        new_lens.append(k * r + length % r)
    i32 = lambda v: torch.from_numpy(np.array(v, np.int32))
    return dict(cache=torch.from_numpy(cache), new_table=i32(new_table), new_lens=i32(new_lens),
                weights=torch.from_numpy(weights), freed=i32(freed),
                totals=i32([taken, given, dropped, 0]))


EXACT = dict(table=_exact_table, rope=_exact_rope, weigh=_exact_weigh, select=_exact_select,
             compact=_exact_compact)


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))
