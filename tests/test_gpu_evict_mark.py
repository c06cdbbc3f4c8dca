"""Only slots past a mark are cut, to fewer rows than that: the budgets come from the
lengths on the device, and slots within the mark stay as they are."""
import numpy as np
import pytest
import torch

from tests import evict_ref as ref
from tests.gpu_util import dev, host
from tests.test_gpu_attend import kvc  # noqa: F401
from tests.test_gpu_evict import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("layout,page,ratio", [("V41", 16, 1), ("V41_FP4", 64, 2), ("V4", 4, 1)])
def test_slots_past_a_mark(kvc, layout, page, ratio, captured):  # noqa: F811
    mark, K = 100, 40
    rows = [100, 101, 41, 40, 0, 99, 160, 3]
    cut = [r > mark for r in rows]
    f = Batch(layout, page, ratio, rows, [K if c else r for r, c in zip(rows, cut)], seed=page)
    lens = np.array([r * ratio + (ratio - 1 if k % 2 else 0) for k, r in enumerate(rows)], np.int32)
    lens[4] = -1
    w = np.random.default_rng(3).random((len(rows), 170)).astype(np.float32)
    cache, d_lens, weights = kvc.Cache(dev(f.host), layout, page), dev(lens), dev(w)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    S = len(rows)
    kept, counts, kw, status = i32(S, mark), i32(S), torch.zeros(S, mark, device="cuda"), i32(1)
    table = dev(f.table)
    new_table, new_lens, freed, totals = torch.full_like(table, 9), i32(S), i32(table.numel()), i32(4)
    free = dev(f.free)

    def call():
        budgets = torch.where(d_lens // ratio > mark, K, mark).to(torch.int32)
        kvc.kvc_evict_select(d_lens, weights, kept, counts, ratio=ratio, first=2, recent=9, budgets=budgets,
                             kept_weights=kw, status=status)
        kvc.kvc_cache_compact(cache, d_lens, kept, counts, table, free, new_table, new_lens, ratio=ratio,
                              kept_weights=kw, weights=weights, freed=freed, totals=totals, status=status)
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graph.replay()
    else:
        call()
    torch.cuda.synchronize()
    want = ref.select(lens, w, [K if c else mark for c in cut], mark, ratio, 2, 9)
    assert np.array_equal(host(kept), want[0]) and np.array_equal(host(counts), want[1])
    moved = ref.compact(f.host, layout, page, ratio, lens, want[0], want[1], f.table, f.free,
                        kept_weights=want[2], weights=w)
    assert np.array_equal(host(cache.data), moved["cache"]) and status.item() == 0
    assert np.array_equal(host(new_table), moved["new_table"]) and np.array_equal(host(new_lens), moved["new_lens"])
    assert np.array_equal(host(weights), moved["weights"]) and host(totals).tolist() == moved["totals"]
    assert host(freed)[:totals[1]].tolist() == moved["freed"]
    for b, c in enumerate(cut):
        held = -(-rows[b] // page) if lens[b] >= 0 else 0
        assert c or (host(new_lens)[b] == lens[b] and np.array_equal(host(new_table)[b, :held], f.table[b, :held]))
    assert sum(cut) == 2
