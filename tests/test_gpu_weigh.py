"""Attention weight that cached rows collect, on the GPU against 64-bit
references: packed prompts, chains, trees and single tokens, every layout, few
and many queries, ragged and odd sizes, masks that leave nothing, rows and
queries that are not finite, decay, strides, streams, captured graphs."""
import ctypes as C
import math
import random

import numpy as np
import pytest
import torch

from tests import attend_ref, evict_ref as ref
from tests.gpu_util import dev
from tests.test_gpu_attend import (Filled, SCALE, as_i64, kvc, prefill_seen, queries,  # noqa: F401
                                   random_tree, tree_seen)

pytestmark = pytest.mark.gpu


def natural_lse(q, rows, seen):
    """The log-sum-exp of each query over the rows it sees, in fp32."""
    _, lse, _, _ = attend_ref.attend(q.double(), rows, seen, SCALE)
    return lse.float()


def check(got, old, total, tol, decay, fresh):
    """One slot's rows: old [R] before the call, the first `fresh` of which count."""
    was = torch.where(torch.arange(len(total)) < fresh, old[:len(total)].double() * decay, 0.0)
    bad = ~((got[:len(total)].double() - was - total).abs() <= tol + 2 * ref.U_FP32 * (was.abs() + total))
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} rows, first {bad.nonzero()[:4].flatten().tolist()}"


def offsets_of(slots):
    n = [s[1] for s in slots]
    return torch.tensor([[sum(n[:i]) for i in range(len(n))], n], dtype=torch.int32)


# layout, page, ratio, heads, [(start, new) per slot]
PREFILL = [
    ("V41", 64, 1, 4, [(0, 1)]),                             # a token, a row
    ("V41", 64, 2, 8, [(0, 64)]),
    ("V41_FP4", 64, 1, 1, [(0, 128)]),                       # as many pairs as are kept in LDS
    ("V41", 64, 1, 1, [(0, 129)]),                           # one more
    ("V41_FP4", 128, 2, 32, [(0, 33), (0, 1), (0, 2), (0, 160)]),
    ("V4", 64, 1, 24, [(0, 5), (31, 40), (257, 3)]),
    ("V41", 16, 1, 5, [(0, 100), (100, 31)]),
    ("V41_FP4", 1, 1, 3, [(0, 70)]),                         # a page per row
    ("V4", 4096, 2, 64, [(511, 66)]),                        # an odd start
    ("V41", 64, 2, 100, [(0, 1)]),                           # no row to see
    ("V41", 32, 1, 16, [(0, 0), (7, 9), (0, 0), (0, 0), (3, 1)]),  # empty slots
    ("V4", 64, 1, 8, [(4000, 17)]),                          # many rows: cut blocks and several of them
    ("V41", 64, 1, 16, [(0, 700)]),
    ("V41_FP4", 64, 2, 1024, [(9, 2)]),
    ("V41", 64, 1, 16, [(255, 1), (0, 256), (1, 256), (0, 257)]),  # around a block of rows
    ("V41_FP4", 64, 1, 64, [(100, 300)]),
]


@pytest.mark.parametrize("layout,page,ratio,H,slots", PREFILL)
def test_prefill(kvc, layout, page, ratio, H, slots):  # noqa: F811
    counts = [(s + n) // ratio for s, n in slots]
    f = Filled(kvc, layout, page, counts, seed=len(slots) + H)
    T = sum(n for _, n in slots)
    q = queries(T, H, seed=H, scale=1.3)
    W = max(counts + [1]) + 3
    g = torch.Generator().manual_seed(T)
    old = torch.rand(len(slots), W, generator=g) * 5
    lse = torch.zeros(T, H)
    want = []
    at = 0
    for b, (s, n) in enumerate(slots):
        if n and counts[b]:
            rows, valid = f.rows(b, counts[b])
            seen = prefill_seen(s, n, ratio, counts[b])
            lse[at:at + n] = natural_lse(q[at:at + n], rows, seen)
            want.append(ref.weigh(q[at:at + n].double(), lse[at:at + n], rows, valid, seen, SCALE))
        else:
            lse[at:at + n] = -math.inf
            want.append(None)
        at += n
    args = (f.cache, q.cuda(), lse.cuda(), offsets_of(slots).cuda(),
            torch.tensor([s for s, _ in slots], dtype=torch.int32, device="cuda"), dev(f.table))
    for decay, prev in ((1.0, True), (0.5, True), (1.0, False)):
        out = torch.full((len(slots), W), 9.0, device="cuda")
        kvc.kvc_weigh_prefill(*args, out, scale=SCALE, ratio=ratio, decay=decay,
                              prev=old.cuda() if prev else None)
        got = out.cpu()
        for b, (s, n) in enumerate(slots):
            done = counts[b] if n else 0
            assert (got[b, done:] == 9.0).all()
            if want[b] is not None:
                check(got[b], old[b], *want[b], decay if prev else 0.0, s // ratio)
                if decay == 1.0 and not prev:
                    # the weights of a query sum to 1
                    live = int((torch.isfinite(lse[sum(x for _, x in slots[:b]):][:n])).sum())
                    assert abs(got[b, :done].double().sum().item() - live) <= 1e-4 * live + 1e-6
    # in place
    out = old.cuda()
    kvc.kvc_weigh_prefill(*args, out, scale=SCALE, ratio=ratio, decay=0.5, prev=out)
    for b, (s, n) in enumerate(slots):
        if want[b] is not None:
            check(out.cpu()[b], old[b], *want[b], 0.5, s // ratio)


# layout, page, ratio, heads, D, [start per slot], tree
TREE = [
    ("V41", 64, 1, 16, 1, [0], False),                       # a token, a row
    ("V41", 64, 1, 16, 1, [999], False),
    ("V41_FP4", 64, 1, 64, 1, [5, 300, 31, 32, 33, 0], False),
    ("V4", 64, 2, 32, 4, [0, 1, 2, 130, 777], False),
    ("V4", 64, 2, 16, 1, [0, 1], False),                     # a slot that sees no row
    ("V41", 128, 1, 128, 1, [600, 10], False),               # 128 pairs
    ("V41", 16, 1, 33, 3, [40, 63], False),                  # 99 pairs
    ("V41_FP4", 64, 1, 20, 7, [100, 0, 257], True),          # 140 pairs: many
    ("V41", 64, 1, 2, 64, [63, 500], True),
    ("V4", 64, 1, 16, 64, [300, 1, 0], True),
    ("V41_FP4", 1, 1, 8, 5, [50, 51], True),
    ("V41", 64, 1, 1024, 1, [70], False),
    ("V41", 64, 1, 128, 7, [9000], True),                    # cut blocks
]


@pytest.mark.parametrize("layout,page,ratio,H,D,starts,tree", TREE)
def test_tree(kvc, layout, page, ratio, H, D, starts, tree):  # noqa: F811
    S = len(starts)
    counts = [(s + D) // ratio for s in starts]
    f = Filled(kvc, layout, page, counts, seed=S + H + D)
    q = queries(S * D, H, seed=H + D, scale=1.3)
    rng = random.Random(D)
    masks = [random_tree(D, rng) for _ in starts] if tree else None
    if tree:
        masks[0][D // 2] = 0                                 # sees the context alone, or nothing
    W = max(counts + [1])
    old = torch.rand(S, W, generator=torch.Generator().manual_seed(S)) * 5
    lse = torch.full((S * D, H), -math.inf)
    want = []
    for b, s in enumerate(starts):
        if not counts[b]:
            want.append(None)
            continue
        rows, valid = f.rows(b, counts[b])
        seen = tree_seen(s, masks[b], counts[b]) if tree else prefill_seen(s, D, ratio, counts[b])
        part = slice(b * D, b * D + D)
        lse[part] = natural_lse(q[part], rows, seen)
        want.append(ref.weigh(q[part].double(), lse[part], rows, valid, seen, SCALE))
    out = torch.full((S, W), 9.0, device="cuda")
    kvc.kvc_weigh_tree(f.cache, q.cuda(), lse.cuda(), torch.tensor(starts, dtype=torch.int32, device="cuda"),
                       dev(f.table), out, scale=SCALE, draft_len=D, ratio=ratio, decay=0.75,
                       prev=old.cuda(), tree=as_i64(masks).cuda() if tree else None)
    got = out.cpu()
    for b, s in enumerate(starts):
        assert (got[b, counts[b]:] == 9.0).all()
        if want[b] is not None:
            check(got[b], old[b], *want[b], 0.75, s // ratio)


@pytest.mark.parametrize("H,D", [(16, 1), (16, 12)])
def test_skipped_slots_bad_pages_and_short_tables(kvc, H, D):  # noqa: F811
    """Inactive slots, pages outside the cache, rows past the table and past
    the weights, and their status bits."""
    starts = [200, -1, 130, 90]
    counts = [s + D if s >= 0 else 0 for s in starts]
    f = Filled(kvc, "V41", 32, counts, seed=4)
    f.table[0, 2] = -3                                       # rows 64 .. 95
    f.table[2, 1] = f.host.shape[0]                          # rows 32 .. 63
    q = queries(4 * D, H, seed=5)
    lse = torch.full((4 * D, H), 3.0)
    W = 180                                                  # (slot 0 has 200 rows and more)
    old = torch.rand(4, 256, generator=torch.Generator().manual_seed(6))
    table = dev(f.table)
    out = torch.full((4, 256), 9.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvc.kvc_weigh_tree(f.cache, q.cuda(), lse.cuda(), torch.tensor(starts, dtype=torch.int32, device="cuda"),
                       table[:, :5], out[:, :W], scale=SCALE, draft_len=D, prev=old.cuda(), status=status)
    assert status.item() == kvc.STATUS_PAGE_RANGE | kvc.STATUS_PT_RANGE
    got = out.cpu()
    for b, s in enumerate(starts):
        most = min(counts[b], 5 * 32, W)
        assert (got[b, most:] == 9.0).all()
        if not most:
            continue
        rows, valid = f.rows(b, counts[b])
        seen = prefill_seen(s, D, 1, counts[b])
        part = slice(b * D, b * D + D)
        total, tol = ref.weigh(q[part].double(), lse[part], rows, valid, seen, SCALE)
        check(got[b], old[b], total[:most], tol[:most], 1.0, s)


def test_prefill_rows_outside_the_batch(kvc):  # noqa: F811
    f = Filled(kvc, "V41", 64, [50, 50], seed=4)
    q = queries(20, 16, seed=5)
    off = torch.tensor([[-1, 11], [5, 10]], dtype=torch.int32, device="cuda")
    out = torch.full((2, 50), 9.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    kvc.kvc_weigh_prefill(f.cache, q.cuda(), torch.zeros(20, 16, device="cuda"), off, zero, dev(f.table),
                          out, scale=SCALE, status=status)
    assert status.item() == kvc.STATUS_TOKEN_RANGE and (out == 9.0).all()
    status.zero_()
    late = zero + (2 ** 31 - 100)
    off = torch.tensor([[0, 10], [5, 10]], dtype=torch.int32, device="cuda")
    kvc.kvc_weigh_prefill(f.cache, q.cuda(), torch.zeros(20, 16, device="cuda"), off, late, dev(f.table),
                          out, scale=SCALE, status=status)
    assert status.item() == kvc.STATUS_POS_RANGE and (out == 9.0).all()


@pytest.mark.parametrize("H,D", [(16, 3), (64, 5)])
@pytest.mark.parametrize("layout", ["V4", "V41"])
def test_rows_and_queries_that_are_not_finite(kvc, layout, H, D):  # noqa: F811
    """A row with a NaN or an infinity collects nothing, a query without a
    finite lse gives nothing, and nobody else is the worse for them."""
    start, count = 300, 300 + D
    f = Filled(kvc, layout, 64, [count], seed=9)
    bad = [5, 64, 299, 301]
    for r in bad:
        page, at = int(f.table[0, r // 64]), r % 64
        if layout == "V4":
            f.host[page, at * 576 + 448:at * 576 + 450] = [0x80, 0x7F] if r % 2 else [0xC1, 0x7F]
        else:
            f.host[page, at * 512 + 7] = 0x7F                # a NaN code
    cache = kvc.Cache(dev(f.host), layout, 64)
    q = queries(D, H, seed=1)
    rows, valid = f.rows(0, count)
    seen = prefill_seen(start, D, 1, count)
    clean = torch.where(torch.isfinite(rows).all(1)[:, None], rows, torch.zeros_like(rows))
    lse = natural_lse(q, clean, seen)
    lse[0, 3], lse[1, 0], lse[2, 5] = math.nan, math.inf, -math.inf
    q[0, 3, 17] = math.nan
    q[1, 0, 2] = math.inf
    total, tol = ref.weigh(q.double(), lse, rows, valid, seen, SCALE)
    out = torch.full((1, count), 9.0, device="cuda")
    kvc.kvc_weigh_tree(cache, q.cuda(), lse.cuda(), torch.tensor([start], dtype=torch.int32, device="cuda"),
                       dev(f.table), out, scale=SCALE, draft_len=D)
    check(out.cpu()[0], torch.zeros(count), total, tol, 0.0, 0)
    assert (out.cpu()[0, bad] == 0).all()


def test_masked_rows_hold_anything(kvc):  # noqa: F811
    """Rows of the last page that no token of the call sees, and drafted rows
    that a token does not see, may hold NaN."""
    start, D, H = 100, 4, 16
    f = Filled(kvc, "V4", 64, [start + D], seed=3)
    page, at = int(f.table[0, 1]), (start + 2) % 64
    f.host[page, at * 576 + 448:at * 576 + 450] = [0xC1, 0x7F]
    cache = kvc.Cache(dev(f.host), "V4", 64)
    masks = [[1, 3, 0, 9]]                                   # nobody sees drafted row 2
    q = queries(D, H, seed=2)
    rows, valid = f.rows(0, start + D)
    seen = tree_seen(start, masks[0], start + D)
    clean = torch.where(torch.isfinite(rows).all(1)[:, None], rows, torch.zeros_like(rows))
    lse = natural_lse(q, clean, seen)
    total, tol = ref.weigh(q.double(), lse, rows, valid, seen, SCALE)
    for heads in (H,):
        out = torch.full((1, start + D), 9.0, device="cuda")
        kvc.kvc_weigh_tree(cache, q.cuda(), lse.cuda(), torch.tensor([start], dtype=torch.int32, device="cuda"),
                           dev(f.table), out, scale=SCALE, draft_len=D, tree=as_i64(masks).cuda())
        check(out.cpu()[0], torch.zeros(start + D), total, tol, 0.0, 0)


@pytest.mark.parametrize("H,D", [(16, 1), (64, 4)])
def test_decay_0_forgets(kvc, H, D):  # noqa: F811
    """With decay 0 what the rows had counts for nothing, whatever it is; rows that
    the call's tokens complete begin at 0 whatever lies there."""
    f = Filled(kvc, "V41", 64, [300 + D], seed=2)
    q = queries(D, H, seed=4).cuda()
    lse = torch.full((D, H), 8.0, device="cuda")
    st = torch.tensor([300], dtype=torch.int32, device="cuda")
    a, b = (torch.full((1, 300 + D), math.nan, device="cuda") for _ in range(2))
    b[0, :300] = 0
    kvc.kvc_weigh_tree(f.cache, q, lse, st, dev(f.table), a, scale=SCALE, draft_len=D, prev=a, decay=0.0)
    kvc.kvc_weigh_tree(f.cache, q, lse, st, dev(f.table), b, scale=SCALE, draft_len=D, prev=b)
    assert torch.isfinite(a).all() and torch.equal(a, b)


@pytest.mark.parametrize("H,D", [(16, 1), (48, 4)])
@pytest.mark.parametrize("S", [1025, 8191])
def test_many_slots_few_of_them_active(kvc, S, H, D):  # noqa: F811
    live = {0: 40, 1: 300, 700: 31, 1023: 0, 1024: 65, S - 2: 500, S - 1: 7}
    f = Filled(kvc, "V41", 64, [live[b] + D for b in live], seed=12)
    starts = torch.full((S,), -1, dtype=torch.int32)
    table = np.zeros((S, f.table.shape[1]), np.int32)
    for k, (b, s) in enumerate(live.items()):
        starts[b] = s
        table[b] = f.table[k]
    g = torch.Generator().manual_seed(1)
    part = (torch.randn(len(live), D, H, 512, generator=g) * 1.2).bfloat16()
    q = torch.zeros(S, D, H, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(S * D, H)
    want = {}
    for k, (b, s) in enumerate(live.items()):
        q[b] = part[k].cuda()
        rows, valid = f.rows(k, s + D)
        seen = prefill_seen(s, D, 1, s + D)
        lse[b * D:b * D + D] = natural_lse(part[k], rows, seen)
        want[b] = ref.weigh(part[k].double(), lse[b * D:b * D + D], rows, valid, seen, SCALE)
    out = torch.full((S, 510), 9.0, device="cuda")
    kvc.kvc_weigh_tree(f.cache, q.view(S * D, H, 512), lse.cuda(), starts.cuda(), dev(table), out,
                       scale=SCALE, draft_len=D)
    got = out.cpu()
    for b, s in live.items():
        check(got[b], torch.zeros(510), *want[b], 0.0, 0)
        assert (got[b, s + D:] == 9.0).all()
    idle = torch.ones(S, dtype=torch.bool)
    idle[list(live)] = False
    assert (got[idle] == 9.0).all()


@pytest.mark.parametrize("H,D", [(16, 2), (40, 6)])
def test_strides(kvc, H, D):  # noqa: F811
    """Queries, weights and tables inside wider tensors, heads before tokens."""
    starts = [77, 140]
    f = Filled(kvc, "V41_FP4", 64, [s + D for s in starts], seed=2)
    q = queries(2 * D, H, seed=4).cuda()
    lse = torch.full((2 * D, H), 5.0, device="cuda")
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    a = torch.zeros(2, 160, device="cuda")
    kvc.kvc_weigh_tree(f.cache, q, lse, st, dev(f.table), a, scale=SCALE, draft_len=D)
    wide = torch.zeros(2 * D, 2, H, 1024, dtype=torch.bfloat16, device="cuda")
    wide[:, 1, :, 512:] = q
    table = torch.full((2, 40), -1, dtype=torch.int32, device="cuda")
    table[:, 7:7 + f.table.shape[1]] = dev(f.table)
    b = torch.full((2, 400), 9.0, device="cuda")
    kvc.kvc_weigh_tree(f.cache, wide[:, 1, :, 512:], lse, st, table[:, 7:7 + f.table.shape[1]],
                       b[:, 100:260], scale=SCALE, draft_len=D)
    n = max(starts) + D
    for k, s in enumerate(starts):
        assert torch.equal(b[k, 100:100 + s + D], a[k, :s + D])
    assert (b[:, :100] == 9).all() and (b[:, 100 + n:] == 9).all()
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)
    c = torch.zeros(2, 160, device="cuda")
    kvc.kvc_weigh_tree(f.cache, turned, lse, st, dev(f.table), c, scale=SCALE, draft_len=D)
    assert torch.equal(a, c)


@pytest.mark.parametrize("H,D", [(16, 2), (64, 8)])
def test_streams_graphs_and_repeats(kvc, H, D):  # noqa: F811
    """The same bits on another stream, from a replayed graph (lengths renewed
    between the replays) and again; two graphs with a workspace each."""
    starts = [900, 40, 333]
    f = Filled(kvc, "V41", 64, [s + D for s in starts], seed=2)
    q = queries(3 * D, H, seed=4).cuda()
    lse = torch.full((3 * D, H), 8.0, device="cuda")
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    table = dev(f.table)
    space = [torch.empty(kvc.kvc_weigh_workspace(), dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.zeros(3, 1000, device="cuda") for _ in range(4)]
    call = lambda o, w: kvc.kvc_weigh_tree(f.cache, q, lse, st, table, o, scale=SCALE, draft_len=D,
                                           workspace=w)
    call(outs[0], None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call(outs[1], None)
    s.synchronize()
    assert torch.equal(outs[0], outs[1])
    graphs = []
    for k in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(outs[2 + k], space[k])
        graphs.append(g)
    for turn in range(3):
        st.copy_(torch.tensor([900 - 77 * turn, 40 + turn, 333], dtype=torch.int32))
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        call(outs[0], None)
        assert torch.equal(outs[2], outs[0]) and torch.equal(outs[3], outs[0])


@pytest.mark.parametrize("sink", [False, True])
def test_weights_of_an_attention_call(kvc, sink):  # noqa: F811
    """With the lse that the attention gave, a query's weights sum to 1, or to
    what its sink leaves."""
    slots = [(0, 200), (77, 30)]
    H = 16
    f = Filled(kvc, "V41", 64, [200, 107], seed=3)
    q = queries(230, H, seed=6, scale=1.2).cuda()
    off, st = offsets_of(slots).cuda(), torch.tensor([0, 77], dtype=torch.int32, device="cuda")
    lse = torch.zeros(230, H, device="cuda")
    sinks = torch.linspace(-2, 3, H, device="cuda") if sink else None
    kvc.kvc_attend_prefill(f.cache, q, off, st, dev(f.table), torch.empty_like(q), scale=SCALE, lse=lse,
                           sink=sinks)
    out = torch.zeros(2, 200, device="cuda")
    kvc.kvc_weigh_prefill(f.cache, q, lse, off, st, dev(f.table), out, scale=SCALE)
    total = 230 * H
    if sink:
        total -= torch.exp2(sinks.double() * ref.LOG2E - lse.double()).sum().item()
    assert abs(out.double().sum().item() - total) <= 2e-5 * total


@pytest.mark.parametrize("H,counts", [(16, [3, 0, 4, 0]), (48, [30, 0, 5, 0])])
def test_slots_without_tokens_are_left(kvc, H, counts):  # noqa: F811
    """Neither their weights nor prev move, whatever decay is."""
    starts = [100, 70, 50, -1]
    f = Filled(kvc, "V41", 64, [s + c for s, c in zip(starts[:3], counts)] + [64], seed=5)
    at = torch.cat([torch.tensor([0]), torch.tensor(counts[:-1]).cumsum(0)])
    q = queries(sum(counts), H, seed=6)
    lse = torch.zeros(sum(counts), H)
    prev, out = torch.rand(4, 200, device="cuda"), torch.full((4, 200), 9.0, device="cuda")
    kvc.kvc_weigh_prefill(f.cache, q.cuda(), lse.cuda(), torch.stack([at, torch.tensor(counts)]).int().cuda(),
                          torch.tensor(starts, dtype=torch.int32, device="cuda"), dev(f.table), out, scale=SCALE,
                          prev=prev, decay=0.5)
    assert (out[[1, 3]] == 9).all()
    for b in (0, 2):
        assert (out[b, :starts[b]] >= 0.5 * prev[b, :starts[b]]).all() and (out[b, starts[b] + counts[b]:] == 9).all()


@pytest.mark.parametrize("H,D", [(16, 1), (64, 4)])
def test_a_width_past_every_page(kvc, H, D):  # noqa: F811
    """One row of the table may be said to be as wide as 64 bits go."""
    f = Filled(kvc, "V41", 64, [130 + D], seed=7)
    q = queries(D, H, seed=8).cuda()
    lse = torch.zeros(D, H, device="cuda")
    start, table = torch.tensor([130], dtype=torch.int32, device="cuda"), dev(f.table)
    want = torch.zeros(1, 130 + D, device="cuda")
    kvc.kvc_weigh_tree(f.cache, q, lse, start, table, want, scale=SCALE, draft_len=D)
    got = torch.zeros_like(want)
    space = torch.empty(kvc.kvc_weigh_workspace(), dtype=torch.uint8, device="cuda")
    a = kvc.kvc_weigh_args(1, H, 1, D, q.data_ptr(), q.stride(0), q.stride(1), D, lse.data_ptr(), None,
                           start.data_ptr(), table.data_ptr(), 2 ** 62, 2 ** 62, None, SCALE, 1.0, None, 0,
                           got.data_ptr(), 130 + D, 130 + D, f.cache.desc(), space.data_ptr(), space.numel(), None)
    assert kvc.lib().kvc_weigh_tree(C.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(got, want) and (want > 0).any()
