"""The calls together, as a serving loop makes them: tables from lengths, rows
rotated and stored, queries rotated, attention, its outputs turned back, weights
collected, rows chosen and moved, and the attention over what is left; and what
the binding refuses of tensors that are on the device."""
import math

import numpy as np
import pytest
import torch

from tests import attend_ref, evict_ref as ref
from tests.gpu_util import dev, host
from tests.test_gpu_attend import SCALE, kvc  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout,page,H", [("V41", 16, 16), ("V41_FP4", 64, 64), ("V4", 64, 40)])
@pytest.mark.parametrize("captured", [False, True])
def test_serving_loop(kvc, layout, page, H, captured):  # noqa: F811
    """Prompts of different lengths, then decoded tokens one at a time; whoever
    passes 96 rows is cut back to 64.  Every attention is compared with one in 64
    bits over the rows that should be there, kept by their original numbers."""
    S, K, most = 3, 64, 96
    prompts = [70, 95, 20]
    steps = 30
    rb = kvc.kvc_layout_query(layout).row_bytes
    pages = 60
    cache = kvc.Cache(torch.zeros(pages, page * rb, dtype=torch.uint8, device="cuda"), layout, page)
    width = -(-(most + 1) // page) + 1
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    freqs = torch.empty(256, 64, device="cuda")
    kvc.kvc_rope_table(freqs, base=10000.0, scaling="parts", factor=4.0, original=64.0)
    table, new_table = i32(S, width), i32(S, width)
    W = width * page
    weights, kept_weights = torch.zeros(S, W, device="cuda"), torch.zeros(S, K, device="cuda")
    kept, counts, lens, new_lens, totals, moved = i32(S, K), i32(S), i32(S), i32(S), i32(4), i32(4)
    status = i32(1)
    free = torch.arange(1, pages, dtype=torch.int32, device="cuda")
    freed = i32(S * width)
    g = torch.Generator().manual_seed(H)
    truth = [[] for _ in range(S)]             # original row numbers each slot holds
    stored = [[] for _ in range(S)]            # every row as it was stored, by original number
    seen_tokens = list(prompts)

    def rows_now(b):
        n = len(truth[b])
        rows, valid = attend_ref.cached_rows(host(cache.data), layout, page, host(table)[b], n)
        assert valid.all()
        return rows

    def step(new):
        """`new[b]` tokens each (packed)."""
        nonlocal free
        T = sum(new)
        rows = torch.randn(T, 512, generator=g).bfloat16().cuda()
        q = (torch.randn(T, H, 512, generator=g) * 1.3).bfloat16().cuda()
        off, st, loc, pos = i32(2, S), i32(S), i32(T), i32(T)
        kvc.kvc_slot_map(ratio=1, page_size=page, num_pages=pages, lens=lens, new_lens=torch.tensor(
            new, dtype=torch.int32, device="cuda"), page_table=table, free_pages=free, offsets=off, start_pos=st,
            out_loc=loc, positions=pos, totals=totals, status=status)
        # a row's position is the request's own, whatever rows it has lost
        own = torch.cat([torch.arange(n, dtype=torch.int32) + seen_tokens[b] - (n if n else 0)
                         for b, n in enumerate(new)]).cuda()
        kvc.kvc_store_rows_rope(cache, rows, own, freqs, loc, status=status)
        turned, out, lse = torch.empty_like(q), torch.empty_like(q), torch.zeros(T, H, device="cuda")
        kvc.kvc_rope_rows(q, own, freqs, turned, status=status)
        kvc.kvc_attend_prefill(cache, turned, off, st, table, out, scale=SCALE, lse=lse, status=status)
        kvc.kvc_weigh_prefill(cache, turned, lse, off, st, table, weights, scale=SCALE, prev=weights,
                              status=status)
        back = out.clone()
        kvc.kvc_rope_rows(back, own, freqs, transpose=True, status=status)
        free = free[int(totals[2]):]
        lens.add_(torch.tensor(new, dtype=torch.int32, device="cuda"))
        return q, turned, out, back, lse, own

    def evict():
        call = lambda: (kvc.kvc_evict_select(lens, weights, kept, counts, first=2, recent=8,
                                             kept_weights=kept_weights, status=status, budgets=budgets),
                        kvc.kvc_cache_compact(cache, lens, kept, counts, table, spare, new_table, new_lens,
                                              kept_weights=kept_weights, weights=weights, freed=freed,
                                              totals=moved, status=status))
        nonlocal free
        # (a slot under the limit keeps what it has)
        over = lens > most
        budgets = torch.where(over, K, -1).to(torch.int32)
        budgets = torch.where(over | (lens <= K), budgets, -1)
        spare = free[:12].contiguous()
        before = host(weights).copy()
        n_before = host(lens).copy()
        # rows past K of a slot that is not cut cannot be listed: such a slot is left out
        lens_in = torch.where(over, lens, -1).to(torch.int32)
        real = lens.clone()
        lens.copy_(lens_in)
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                call()
            graph.replay()
        else:
            call()
        torch.cuda.synchronize()
        cut = host(over)
        if cut.any():
            t = host(moved)
            free = torch.cat([spare[int(t[0]):], free[12:], freed[:int(t[1])].clone()])
        picked = ref.select(np.where(cut, n_before, -1), before, [K] * S, K, 1, 2, 8)
        assert np.array_equal(host(kept), picked[0]) and np.array_equal(host(counts), picked[1])
        for b in range(S):
            if cut[b]:
                truth[b] = [truth[b][r] for r in picked[0][b]]
        table.copy_(torch.where(over[:, None], new_table, table))
        lens.copy_(torch.where(over, new_lens, real))

    def check(new, res):
        q, turned, out, back, lse, own = res
        at = 0
        for b, n in enumerate(new):
            if not n:
                continue
            rows = rows_now(b)
            count = len(truth[b])
            for r in rows[count - n:]:
                stored[b].append(r)
            assert all(torch.equal(rows[k], stored[b][t]) for k, t in enumerate(truth[b]))
            seen = torch.arange(count)[None] < (count - n + 1 + torch.arange(n))[:, None]
            want, wl, tol, ltol = attend_ref.attend(turned[at:at + n].cpu().double(), rows, seen, SCALE)
            assert ((out[at:at + n].cpu().double() - want).abs() <= tol).all()
            assert ((lse[at:at + n].cpu().double() - wl).abs() <= ltol).all()
            r, rt = ref.rope(q[at:at + n].cpu(), own[at:at + n].cpu(), freqs.cpu(), 448, False, False)
            assert ((turned[at:at + n].cpu().double() - r).abs() <= rt).all()
            r, rt = ref.rope(out[at:at + n].cpu(), own[at:at + n].cpu(), freqs.cpu(), 448, False, True)
            assert ((back[at:at + n].cpu().double() - r).abs() <= rt).all()
            at += n

    new = prompts
    for b, n in enumerate(new):
        truth[b] += list(range(n))
    check(new, step(new))
    cuts = 0
    for k in range(steps):
        evict_now = host(lens) > most
        cuts += int(evict_now.sum())
        evict()
        new = [1, 1, 1 if k % 3 else 0]
        for b, n in enumerate(new):
            truth[b] += list(range(seen_tokens[b], seen_tokens[b] + n))
            seen_tokens[b] += n
        check(new, step(new))
    assert cuts >= 2 and status.item() == 0
    # every page is either free or in one slot's table
    held = [p for b in range(S) for p in host(table)[b, :-(-int(lens[b]) // page)]]
    every = sorted(held + host(free).tolist())
    assert every == list(range(1, pages))


def test_binding_refuses_device_tensors(kvc):  # noqa: F811
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    fl = lambda *s: torch.zeros(*s, device="cuda")
    c = kvc.Cache(torch.zeros(2, 64 * 528, dtype=torch.uint8, device="cuda"), "V41", 64)
    x, f = bf(4, 2, 64), fl(9, 64)
    wide = bf(4, 2, 128)
    W = lambda **kw: dict(dict(q=bf(4, 2, 512), lse=fl(4, 2), start_pos=i(2), page_table=i(2, 3),
                               weights=fl(2, 9)), **kw)
    tree = lambda **kw: kvc.kvc_weigh_tree(c, **W(**kw), scale=0.1, draft_len=2)
    sel = lambda **kw: kvc.kvc_evict_select(**dict(dict(lens=i(2), weights=fl(2, 9), kept=i(2, 4), counts=i(2)), **kw))
    mv = lambda **kw: kvc.kvc_cache_compact(**dict(dict(cache=c, lens=i(2), kept=i(2, 4), counts=i(2),
                                                       page_table=i(2, 3), free_pages=i(5), new_table=i(2, 3),
                                                       new_lens=i(2)), **kw))
    for match, call in (
            ("^out", lambda: kvc.kvc_rope_table(f.half())),
            ("^out", lambda: kvc.kvc_rope_table(fl(64, 9).t())),
            ("^x", lambda: kvc.kvc_rope_rows(x.double(), i(4), f)),
            ("^x", lambda: kvc.kvc_rope_rows(x.transpose(1, 2), i(4), f)),
            ("^out", lambda: kvc.kvc_rope_rows(x, i(4), f, bf(4, 2, 32))),
            ("^out", lambda: kvc.kvc_rope_rows(x, i(4), f, x.half())),
            ("^out: overlaps", lambda: kvc.kvc_rope_rows(wide[..., :64], i(4), f, wide[..., 32:96])),
            ("^out: overlapping rows", lambda: kvc.kvc_rope_rows(x, i(4), f, bf(512).as_strided((4, 2, 64), (96, 64, 1)))),
            ("^positions", lambda: kvc.kvc_rope_rows(x, i(3), f)),
            ("^positions", lambda: kvc.kvc_rope_rows(x, i(4).long(), f)),
            ("^positions", lambda: kvc.kvc_rope_rows(x, i(4).cpu(), f)),
            ("^freqs", lambda: kvc.kvc_rope_rows(x, i(4), f[0])),
            ("^freqs", lambda: kvc.kvc_rope_rows(x, i(4), f.cpu())),
            ("^freqs", lambda: kvc.kvc_rope_rows(x, i(4), fl(9, 128)[:, :64])),
            ("^q", lambda: tree(q=bf(4, 2, 256))),
            ("^lse", lambda: tree(lse=fl(2, 4))),
            ("^lse", lambda: tree(lse=fl(4, 2).cpu())),
            ("^page_table", lambda: tree(page_table=i(1, 3))),
            ("^weights", lambda: tree(weights=fl(1, 9))),
            ("^weights", lambda: tree(weights=fl(18))),
            ("^weights", lambda: tree(weights=fl(2, 9).double())),
            ("^prev", lambda: tree(prev=fl(2, 8))),
            ("^workspace", lambda: tree(workspace=i(9))),
            ("^kept", lambda: sel(kept=i(1, 4))),
            ("^counts", lambda: sel(counts=i(1))),
            ("^budgets", lambda: sel(budgets=i(1))),
            ("^kept_weights", lambda: sel(kept_weights=fl(2, 3))),
            ("^weights", lambda: sel(weights=fl(2, 9).cpu())),
            ("^new_table", lambda: mv(new_table=i(2, 2))),
            ("^new_lens", lambda: mv(new_lens=i(1))),
            ("^kept", lambda: mv(kept=i(8))),
            ("^totals", lambda: mv(totals=i(3))),
            ("^freed", lambda: mv(freed=i(0))),
            ("^kept_weights", lambda: mv(kept_weights=fl(2, 3), weights=fl(2, 9)))):
        with pytest.raises(ValueError, match=match):
            call()
    for call in (lambda: mv(kept_weights=fl(2, 4)), lambda: tree(weights=fl(2, 0)), lambda: sel(kept=i(2, 0)),
                 lambda: sel(first=-1),
                 lambda: kvc.kvc_rope_rows(x, i(4), f, bf(2, 64).expand(4, 2, 64)), lambda: kvc.kvc_rope_table(fl(4, 7))):
        with pytest.raises(kvc.KvcError):
            call()


def test_no_slots_and_no_tokens(kvc):  # noqa: F811
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    fl = lambda *s: torch.zeros(*s, device="cuda")
    c = kvc.Cache(torch.zeros(2, 64 * 528, dtype=torch.uint8, device="cuda"), "V41", 64)
    q = torch.zeros(0, 4, 512, dtype=torch.bfloat16, device="cuda")
    kvc.kvc_weigh_tree(c, q, fl(0, 4), i(0), i(0, 3), fl(0, 9), scale=0.1)
    kvc.kvc_weigh_prefill(c, q, fl(0, 4), i(2, 2), i(2), i(2, 3), fl(2, 9), scale=0.1)
    kvc.kvc_evict_select(i(0), fl(0, 9), i(0, 4), i(0))
    kvc.kvc_cache_compact(c, i(0), i(0, 4), i(0), i(0, 3), i(0), i(0, 3), i(0))
    kvc.kvc_rope_rows(q, i(0), fl(9, 64))
    kvc.kvc_rope_table(fl(0, 64))
    torch.cuda.synchronize()
