"""The choice of the rows that stay and their move, on the GPU against plain
references: budgets, protected rows, ties, values that are not finite, lengths
from none to long ones, every layout and page size, refusals, bad pages and
lists, strides, streams, captured graphs."""
import numpy as np
import pytest
import torch

import oracle
from tests import evict_ref as ref
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    import fp8_fp4_quantized_amd as k
    return k


# -------------------------------------------------------------------- choice
def run_select(kvc, lens, weights, K, *, budget=None, budgets=None, ratio=1, first=0, recent=0, pad=0):
    S, W = weights.shape
    kept = torch.full((S, K + pad), 77, dtype=torch.int32, device="cuda")
    kw = torch.full((S, K + pad), 77.0, device="cuda")
    wide = torch.full((S, W + pad), -5.0, device="cuda")
    wide[:, :W] = torch.from_numpy(weights).cuda()
    counts = torch.full((S + 1,), 77, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvc.kvc_evict_select(dev(np.array(lens, np.int32)), wide[:, :W], kept[:, :K], counts, budget=budget,
                         ratio=ratio, first=first, recent=recent, kept_weights=kw[:, :K], status=status,
                         budgets=None if budgets is None else dev(np.array(budgets, np.int32)))
    assert counts[S] == 77 and (kept[:, K:] == 77).all() and (kw[:, K:] == 77).all()
    return host(kept[:, :K]), host(counts[:S]), host(kw[:, :K]), status.item()


def check_select(kvc, lens, weights, K, *, budget=None, budgets=None, ratio=1, first=0, recent=0, pad=0):
    got = run_select(kvc, lens, weights, K, budget=budget, budgets=budgets, ratio=ratio, first=first,
                     recent=recent, pad=pad)
    B = budgets if budgets is not None else [K if budget is None else budget] * len(lens)
    want = ref.select(lens, weights, B, K, ratio, first, recent)
    assert np.array_equal(got[1], want[1]), "counts"
    assert np.array_equal(got[0], want[0]), "kept"
    assert np.array_equal(got[2].view(np.int32), want[2].view(np.int32)), "weights kept"
    assert got[3] == want[3], "status"


def weights_of(S, W, seed, kind="tail"):
    rng = np.random.default_rng(seed)
    w = np.exp(1.5 * rng.standard_normal((S, W))).astype(np.float32)
    w[rng.random((S, W)) < 0.05] = 0
    if kind == "ties":
        w = np.round(w * 2) / 2
    elif kind == "same":
        w[:] = 1.25
    elif kind == "close":                      # keys that part in the last digit alone
        w = (np.float32(1.0).view(np.int32) + rng.integers(0, 1000, (S, W)).astype(np.int32)).view(np.float32)
    elif kind == "signs":
        w = (w * rng.choice([-1, 1], (S, W))).astype(np.float32)
        w[rng.random((S, W)) < 0.1] = -0.0
        w[rng.random((S, W)) < 0.02] = np.nan
        w[rng.random((S, W)) < 0.02] = -np.nan
        w[rng.random((S, W)) < 0.02] = np.inf
        w[rng.random((S, W)) < 0.02] = -np.inf
        w[rng.random((S, W)) < 0.02] = 1e-42
    return w.astype(np.float32)


SELECT = [
    # lens, W, K, more, kind
    ([1], 1, 1, {}, "tail"),
    ([2], 2, 1, {}, "tail"),
    ([0, 1, 2, 3, 4, 5, -1], 5, 3, {}, "tail"),
    ([100, 64, 63, 65, 0, -7, 1], 100, 64, dict(first=4, recent=16), "tail"),
    ([1000, 900, 1023, 1024, 1025], 1100, 200, dict(first=4, recent=50), "ties"),
    ([500] * 9, 500, 77, dict(first=100), "tail"),           # the first rows alone
    ([500] * 3, 500, 77, dict(first=10, recent=500), "tail"),  # first and last alone
    ([500] * 3, 500, 77, dict(recent=76), "tail"),           # one place to win
    ([5000, 4999, 300], 5000, 4998, {}, "close"),            # one or two rows to drop
    ([6000], 6000, 1, {}, "signs"),
    ([6000, 3000], 6001, 2500, dict(first=1, recent=7), "signs"),
    ([4096] * 4, 4096, 1000, {}, "same"),
    ([9001, 8000, 20000], 20000, 3000, dict(ratio=2, first=4, recent=64), "ties"),
    ([70001], 70001, 4096, dict(first=16, recent=512), "close"),
    ([300, 300, 300, 300, 300], 300, 100, dict(budgets=[0, 50, 100, 101, -1], recent=20), "tail"),
    ([300], 300, 100, dict(budget=0), "tail"),
    ([300, 50], 300, 100, dict(budget=70), "tail"),
    ([301, 300, 50], 300, 100, {}, "tail"),                  # a slot past its row of weights
]


@pytest.mark.parametrize("lens,W,K,more,kind", SELECT)
@pytest.mark.parametrize("pad", [0, 5])
def test_select(kvc, lens, W, K, more, kind, pad):
    more = dict(more)
    check_select(kvc, lens, weights_of(len(lens), W, len(lens) + W, kind), K, pad=pad, **more)


@pytest.mark.parametrize("n,K,kind", [(131072, 5000, "tail"), (131073, 100000, "ties"), (300001, 4096, "close"),
                                      (262144, 262143, "signs"), (1000003, 65537, "ties"),
                                      (9000001, 70001, "tail")])      # (the most segments)
def test_select_long(kvc, n, K, kind):
    check_select(kvc, [n], weights_of(1, n, n, kind), K, first=4, recent=100)


def test_select_long_and_short_together(kvc):
    lens = [200000, 5, -1, 150001, 4096, 0, 199999, 200001]
    check_select(kvc, lens, weights_of(8, 200000, 3, "ties"), 4000, first=4, recent=100)


@pytest.mark.parametrize("S", [127, 128, 129])
@pytest.mark.parametrize("W", [16500, 33000])
def test_select_long_rows_of_many_slots(kvc, S, W):
    rng = np.random.default_rng(S)
    lens = rng.integers(0, W, S)
    lens[:3] = [W, 16385, -1]
    check_select(kvc, lens, weights_of(S, W, 4, "ties"), 500, first=2, recent=30)


@pytest.mark.parametrize("W", [16384, 16385, 24576, 24577, 32768, 32769, 49153])
@pytest.mark.parametrize("kind", ["tail", "ties", "signs"])
def test_select_where_the_kernels_change(kvc, W, kind):
    check_select(kvc, [W, W - 1, 9000, W, 0], weights_of(5, W, 6, kind), 4000, first=3, recent=77)
    check_select(kvc, [W], weights_of(1, W, 7, kind), W - 1)


def test_select_many_slots(kvc):
    rng = np.random.default_rng(1)
    lens = rng.integers(-1, 40, 8191)
    check_select(kvc, lens, weights_of(8191, 39, 2, "ties"), 12, first=2, recent=3)


def test_select_streams_and_graphs(kvc):
    lens = dev(np.array([300, 200000], np.int32))
    w = dev(weights_of(2, 200000, 1, "ties"))
    kept = [torch.zeros(2, 128, dtype=torch.int32, device="cuda") for _ in range(2)]
    counts = torch.zeros(2, dtype=torch.int32, device="cuda")
    n = kvc.kvc_evict_workspace(2, 200000)
    space = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    kvc.kvc_evict_select(lens, w, kept[0], counts, recent=10)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        kvc.kvc_evict_select(lens, w, kept[1], counts, recent=10)
    s.synchronize()
    assert torch.equal(kept[0], kept[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvc.kvc_evict_select(lens, w, kept[1], counts, recent=10, workspace=space)
    for turn in range(3):
        w.copy_(dev(weights_of(2, 200000, 5 + turn, "ties")))
        lens.copy_(dev(np.array([100 + 100 * turn, 150000 + turn], np.int32)))
        kept[1].zero_()
        g.replay()
        torch.cuda.synchronize()
        kvc.kvc_evict_select(lens, w, kept[0], counts, recent=10)
        assert torch.equal(kept[0], kept[1])


# ---------------------------------------------------------------------- move
class Batch:
    """A cache of random bytes with `rows[b]` rows of every slot at random
    pages, and a selection of `counts[b]` of them."""

    def __init__(self, layout, page, ratio, rows, counts, seed, spare=3, lens=None, order=False):
        rng = np.random.default_rng(seed)
        db, sb, _, _ = oracle.layout_bytes(layout)
        held = [-(-r // page) for r in rows]
        need = [-(-c // page) for r, c in zip(rows, counts) if 0 <= c < r]
        n = 1 + sum(held) + sum(need) + spare
        self.host = rng.integers(0, 256, (n, -(-page * (db + sb) // 16) * 16 + 32), dtype=np.uint8)
        order_ = rng.permutation(n - 1) + 1
        self.table = np.full((len(rows), max(held + [1]) + 1), 7777, np.int32)
        at = 0
        for b, h in enumerate(held):
            self.table[b, :h] = order_[at:at + h]
            at += h
        self.free = order_[at:].astype(np.int32)
        K = max([c for c in counts] + [1])
        self.kept = np.full((len(rows), K), -1, np.int32)
        for b, (r, c) in enumerate(zip(rows, counts)):
            if c > 0:
                pick = rng.permutation(max(r, 1))[:min(c, r)]
                self.kept[b, :len(pick)] = pick if order else np.sort(pick)
        self.counts = np.array(counts, np.int32)
        self.lens = np.array([r * ratio + (ratio - 1) * (b % 2) for b, r in enumerate(rows)]
                             if lens is None else lens, np.int32)
        self.kept_weights = rng.random(self.kept.shape).astype(np.float32)
        self.weights = rng.random((len(rows), max(list(rows) + [K]))).astype(np.float32)
        self.layout, self.page, self.ratio = layout, page, ratio

    def run(self, kvc, weights=True, freed=None, stream=None):
        """The call's outputs as host arrays."""
        d = {k: dev(getattr(self, k)) for k in ("lens", "kept", "counts", "table", "free")}
        cache = kvc.Cache(dev(self.host), self.layout, self.page)
        S = len(self.lens)
        out = dict(new_table=torch.full(self.table.shape, 55, dtype=torch.int32, device="cuda"),
                   new_lens=torch.full((S,), 55, dtype=torch.int32, device="cuda"),
                   freed=torch.full((self.table.size if freed is None else freed,), 55, dtype=torch.int32,
                                    device="cuda"),
                   totals=torch.full((4,), 55, dtype=torch.int32, device="cuda"),
                   status=torch.zeros(1, dtype=torch.int32, device="cuda"))
        w = dev(self.weights)
        more = dict(kept_weights=dev(self.kept_weights), weights=w) if weights else {}
        for _ in range(2):                     # a repeated call gives the same
            kvc.kvc_cache_compact(cache, d["lens"], d["kept"], d["counts"], d["table"], d["free"],
                                  out["new_table"], out["new_lens"], ratio=self.ratio, freed=out["freed"],
                                  totals=out["totals"], status=out["status"], stream=stream, **more)
        torch.cuda.synchronize()
        return dict({k: host(v) for k, v in out.items()}, cache=host(cache.data), weights=host(w))

    def check(self, kvc, weights=True, freed=None):
        got = self.run(kvc, weights, freed)
        want = ref.compact(self.host, self.layout, self.page, self.ratio, self.lens, self.kept, self.counts,
                           self.table, self.free, self.table.size if freed is None else freed,
                           self.kept_weights if weights else None, self.weights if weights else None)
        assert np.array_equal(got["new_table"], want["new_table"]), "table"
        assert np.array_equal(got["new_lens"], want["new_lens"]), "lens"
        assert got["totals"].tolist() == want["totals"], "totals"
        assert got["status"][0] == want["status"], "status"
        n = len(want["freed"])
        assert got["freed"][:n].tolist() == want["freed"] and (got["freed"][n:] == 55).all(), "freed"
        assert np.array_equal(got["cache"], want["cache"]), "cache"
        assert np.array_equal(got["weights"], want["weights"] if weights else self.weights), "weights"
        return want


MOVES = [
    # layout, page, ratio, rows, counts
    ("V41", 64, 1, [1], [0]),
    ("V41", 64, 1, [2], [1]),
    ("V41_FP4", 64, 2, [200, 64, 65, 0, 130], [100, 64, 64, 0, -1]),
    ("V4", 16, 1, [100, 33, 17, 500], [16, 17, 16, 499]),
    ("V4", 1, 2, [40, 7], [11, 3]),
    ("V41", 4096, 1, [5000, 100], [4097, 50]),
    ("V41_FP4", 128, 1, [1000] * 7, [1, 127, 128, 129, 0, 999, 1000]),
    ("V41", 64, 2, [3000, 10, 2500], [2048, 10, 1]),
    ("V4", 64, 1, [0, 0], [0, -1]),
]


@pytest.mark.parametrize("layout,page,ratio,rows,counts", MOVES)
def test_compact(kvc, layout, page, ratio, rows, counts):
    Batch(layout, page, ratio, rows, counts, 5).check(kvc)
    Batch(layout, page, ratio, rows, counts, 6, spare=0, order=True).check(kvc, weights=False)


@pytest.mark.parametrize("layout", ["V4", "V41", "V41_FP4"])
def test_compact_of_more_rows_than_a_turn_takes(kvc, layout):
    """Row counts past what all waves take at once."""
    want = Batch(layout, 64, 1, [150000, 3, 70000], [140001, 2, 9], 3, order=True).check(kvc)
    assert want["totals"][2] == 150000 - 140001 + 1 + 70000 - 9


def test_compact_refusals(kvc):
    """Inactive slots, tables and lists too short, free pages too few: those
    slots stay as they are, and so does every later one that wants pages."""
    b = Batch("V41", 64, 1, [200, 300, 400, 100, 260], [70, 100, 200, 100, 10], 1)
    need = 2 + 2 + 4 + 1
    for n in range(need + 1):
        c = Batch("V41", 64, 1, [200, 300, 400, 100, 260], [70, 100, 200, 100, 10], 1)
        c.free = b.free[:n]
        c.check(kvc)
    with pytest.raises(ValueError, match="^freed"):          # (no address: taken as none given)
        b.check(kvc, freed=0)
    for cap in [1] + list(range(2, 18, 2)):
        b.check(kvc, freed=cap)
    b.lens[1] = -5
    b.check(kvc)
    b.table = b.table[:, :5].copy()                          # slot 2 has 7 pages
    b.check(kvc)
    b.counts[0], b.kept = 150, b.kept[:, :120].copy()
    b.kept_weights = b.kept_weights[:, :120].copy()
    b.check(kvc)
    b.weights = b.weights[:, :5].copy()
    b.check(kvc)


def test_compact_of_bad_pages_and_lists(kvc):
    b = Batch("V41_FP4", 64, 1, [200, 300], [130, 100], 1)
    b.kept[0, 5], b.kept[0, 6], b.kept[1, 0] = -1, 200, 2 ** 31 - 1
    b.check(kvc)
    b.table[1, 2], b.table[0, 0] = -1, b.host.shape[0]
    b.check(kvc)
    b.free[1], b.free[3] = 0, b.host.shape[0] + 3
    want = b.check(kvc)
    assert want["status"] == 3
    b.kept[1, :50] = 7                                       # one row many times
    b.check(kvc)


def test_compact_of_many_slots(kvc):
    rng = np.random.default_rng(2)
    rows = rng.integers(0, 9, 8191)
    counts = [int(rng.integers(-1, r + 1)) for r in rows]
    Batch("V41_FP4", 4, 1, [int(r) for r in rows], counts, 2).check(kvc)
    rows[:] = 0
    counts = [0] * 8191
    rows[[0, 1024, 5000, 8190]] = 100
    for k in (0, 5000, 8190):
        counts[k] = 33
    counts[1024] = 100
    Batch("V41", 16, 2, [int(r) for r in rows], counts, 2).check(kvc)


def test_compact_keeps_shared_pages(kvc):
    """Two slots with the same pages: one is cut, the other keeps its rows."""
    b = Batch("V41", 64, 1, [200, 200], [70, 200], 1)
    b.table[1] = b.table[0]
    want = b.check(kvc)
    assert np.array_equal(want["new_table"][1][:4], b.table[0][:4])


def test_compact_strides(kvc):
    """Lists, tables and weights inside wider tensors."""
    b = Batch("V41", 64, 1, [200, 300], [130, 100], 1)
    want = ref.compact(b.host, "V41", 64, 1, b.lens, b.kept, b.counts, b.table, b.free, None,
                       b.kept_weights, b.weights)

    def inside(a, fill):
        t = torch.full((a.shape[0], a.shape[1] + 9), fill, dtype=torch.from_numpy(a).dtype, device="cuda")
        t[:, 4:4 + a.shape[1]] = dev(a)
        return t, t[:, 4:4 + a.shape[1]]
    cache = kvc.Cache(dev(b.host), "V41", 64)
    kept, table = inside(b.kept, -9)[1], inside(b.table, -9)[1]
    kw, (w_all, w) = inside(b.kept_weights, -9.0)[1], inside(b.weights, -9.0)
    new_all, new = inside(np.zeros_like(b.table), -9)
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    kvc.kvc_cache_compact(cache, dev(b.lens), kept, dev(b.counts), table, dev(b.free), new, lens,
                          kept_weights=kw, weights=w)
    assert np.array_equal(host(new), want["new_table"]) and np.array_equal(host(w), want["weights"])
    assert np.array_equal(host(cache.data), want["cache"]) and host(lens).tolist() == want["new_lens"].tolist()
    for t, n in ((w_all, b.weights.shape[1]), (new_all, b.table.shape[1])):
        assert (t[:, :4] == -9).all() and (t[:, 4 + n:] == -9).all()


def test_compact_streams_and_graphs(kvc):
    b = Batch("V41_FP4", 64, 1, [500, 300], [130, 100], 4)
    first = b.run(kvc)
    s = torch.cuda.Stream()
    second = b.run(kvc, stream=s)
    for k in first:
        assert np.array_equal(first[k], second[k]), k
    d = {k: dev(getattr(b, k)) for k in ("lens", "kept", "counts", "table", "free")}
    cache = kvc.Cache(dev(b.host), "V41_FP4", 64)
    new, lens = torch.zeros_like(d["table"]), torch.zeros_like(d["lens"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvc.kvc_cache_compact(cache, d["lens"], d["kept"], d["counts"], d["table"], d["free"], new, lens)
    for turn in range(3):
        b.counts = np.array([130 - 50 * turn, 100 + 100 * turn], np.int32)
        want = ref.compact(b.host, "V41_FP4", 64, 1, b.lens, b.kept, np.minimum(b.counts, b.kept.shape[1]),
                           b.table, b.free)
        d["counts"].copy_(dev(np.minimum(b.counts, b.kept.shape[1]).astype(np.int32)))
        cache.data.copy_(dev(b.host))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(cache.data), want["cache"]) and np.array_equal(host(new), want["new_table"])
        assert np.array_equal(host(lens), want["new_lens"])


def test_compact_of_no_slots(kvc):
    """An empty batch takes and gives back nothing, and says so."""
    cache = kvc.Cache(torch.zeros(3, 64 * 528, dtype=torch.uint8, device="cuda"), "V41", 64)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    table, kept = torch.zeros(0, 2, dtype=torch.int32, device="cuda"), torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    totals = torch.full((4,), 7, dtype=torch.int32, device="cuda")
    kvc.kvc_cache_compact(cache, none, kept, none, table, torch.tensor([1, 2], dtype=torch.int32, device="cuda"),
                          torch.zeros_like(table), torch.zeros_like(none), totals=totals)
    assert totals.tolist() == [0, 0, 0, 0]
