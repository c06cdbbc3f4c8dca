"""The weights of a serving loop: collected in place over many steps and carried
through moves, each row's compared with a sum in 64 bits under its original number."""
import numpy as np
import pytest
import torch

from tests import attend_ref, evict_ref as ref
from tests.gpu_util import host
from tests.test_gpu_attend import SCALE, kvc, prefill_seen  # noqa: F401

pytestmark = pytest.mark.gpu


# (three tokens of 16 heads stay in LDS, of 64 they do not)
@pytest.mark.parametrize("layout,page,H,ratio", [("V41", 16, 16, 1), ("V41_FP4", 64, 64, 1), ("V4", 16, 64, 2)])
@pytest.mark.parametrize("form", ["prefill", "tree"])
def test_weights_over_steps_and_moves(kvc, layout, page, H, ratio, form):  # noqa: F811
    S, K, most, pages, decay, steps = 3, 24, 40, 60, 0.875, 24
    lens = [30 * ratio, 39 * ratio + ratio - 1, 5]
    rb = kvc.kvc_layout_query(layout).row_bytes
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    on = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    cache = kvc.Cache(torch.zeros(pages, page * rb, dtype=torch.uint8, device="cuda"), layout, page)
    W = (most // page + 2) * page
    table, new_table = i32(S, W // page), i32(S, W // page)
    weights, kept_weights = torch.full((S, W), 7.0, device="cuda"), torch.zeros(S, K, device="cuda")
    kept, counts, new_lens, moved, status = i32(S, K), i32(S), i32(S), i32(4), i32(1)
    freed = i32(S * (W // page))
    free = list(range(1, pages))
    g = torch.Generator().manual_seed(H)
    held = [[] for _ in range(S)]              # each slot's pages
    want, tol = ([torch.zeros(0, dtype=torch.float64) for _ in range(S)] for _ in range(2))

    def grow(new):
        """Rows for `new[b]` tokens of each slot."""
        slots = []
        for b, n in enumerate(new):
            for r in range(lens[b] // ratio, (lens[b] + n) // ratio):
                if r // page == len(held[b]):
                    held[b].append(free.pop(0))
                    table[b, r // page] = held[b][-1]
                slots.append(held[b][r // page] * page + r % page)
        if slots:
            kvc.kvc_store_rows(cache, torch.randn(len(slots), 512, generator=g).bfloat16().cuda(), on(slots))

    def step(new):
        grow(new)
        T = sum(new)
        q = (torch.randn(T, H, 512, generator=g) * 1.3).bfloat16().cuda()
        out, lse, st = torch.empty_like(q), torch.zeros(T, H, device="cuda"), on(lens)
        kw = dict(scale=SCALE, ratio=ratio, status=status)
        if form == "tree" and len(set(new)) == 1:
            kvc.kvc_attend_tree(cache, q, st, table, out, lse=lse, draft_len=new[0], **kw)
            kvc.kvc_weigh_tree(cache, q, lse, st, table, weights, prev=weights, decay=decay, draft_len=new[0], **kw)
        else:
            off = on([[sum(new[:b]) for b in range(S)], new])
            kvc.kvc_attend_prefill(cache, q, off, st, table, out, lse=lse, **kw)
            kvc.kvc_weigh_prefill(cache, q, lse, off, st, table, weights, prev=weights, decay=decay, **kw)
        got, at = host(weights), 0
        for b, n in enumerate(new):
            count, fresh = (lens[b] + n) // ratio, lens[b] // ratio
            if n and count:
                rows, valid = attend_ref.cached_rows(host(cache.data), layout, page, host(table)[b], count)
                total, t = ref.weigh(q[at:at + n].cpu().double(), lse[at:at + n].cpu(), rows, valid,
                                     prefill_seen(lens[b], n, ratio, count), SCALE)
                zero = torch.zeros(count - fresh, dtype=torch.float64)
                old, ot = torch.cat([want[b], zero]) * decay, torch.cat([tol[b], zero]) * decay
                want[b] = old + total
                tol[b] = ot + t + 2 * ref.U_FP32 * (want[b] + ot + t)
            assert ((torch.from_numpy(got[b, :count]).double() - want[b]).abs() <= tol[b]).all()
            lens[b] += n
            at += n

    def evict():
        cut = [n // ratio > most for n in lens]
        given = [n if c else -1 for n, c in zip(lens, cut)]
        before = host(weights).copy()
        spare = on(free[:12])
        kvc.kvc_evict_select(on(given), weights, kept, counts, ratio=ratio, first=2, recent=6,
                             kept_weights=kept_weights, status=status)
        kvc.kvc_cache_compact(cache, on(given), kept, counts, table, spare, new_table, new_lens, ratio=ratio,
                              kept_weights=kept_weights, weights=weights, freed=freed, totals=moved, status=status)
        picked, n, kw, _ = ref.select(np.array(given), before, [K] * S, K, ratio, 2, 6)
        assert np.array_equal(host(kept), picked) and np.array_equal(host(counts), n)
        assert np.array_equal(host(kept_weights), kw)
        taken, back, _, refused = host(moved).tolist()
        assert refused == 0 and status.item() == 0
        after = host(weights)
        for b in range(S):
            if not cut[b]:
                assert np.array_equal(after[b], before[b])
                continue
            assert np.array_equal(after[b, :K], before[b, picked[b]]) and np.array_equal(after[b, K:], before[b, K:])
            want[b], tol[b] = want[b][picked[b].tolist()], tol[b][picked[b].tolist()]
            table[b] = new_table[b]
            lens[b] = int(new_lens[b])
            held[b] = host(table)[b, :-(-K // page)].tolist()
        free[:taken] = []
        free.extend(host(freed)[:back].tolist())
        return sum(cut)

    first = lens[:]
    lens[:] = [0] * S
    step(first)
    cuts = 0
    for k in range(steps):
        cuts += evict()
        step([1, 3, 1] if k % 3 == 0 else [3, 3, 3] if k % 3 == 1 else [1, 0, 2])
    assert cuts >= 3 and status.item() == 0
    assert sorted(free + sum(held, [])) == list(range(1, pages))
