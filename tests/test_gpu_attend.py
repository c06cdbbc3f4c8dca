"""Attention over the paged cache on the GPU against 64-bit references: packed
prompts, drafted chains and trees, every layout, ragged and odd sizes, masks
that leave nothing, NaN in masked rows, strides, streams and captured graphs."""
import random

import numpy as np
import pytest
import torch

import oracle
from tests import attend_ref as ref
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    import fp8_fp4_quantized_amd as k
    return k


LAYOUTS = ("V4", "V41", "V41_FP4")


class Filled:
    """A cache with ``counts[b]`` rows in each slot at random pages, other
    bytes random (NaN codes among them), and the host's view of the rows."""

    def __init__(self, kvc, layout, page_size, counts, seed, scale=1.0, extra_width=1):
        rng = np.random.default_rng(seed)
        db, sb, _, _ = oracle.layout_bytes(layout)
        pages = [-(-c // page_size) for c in counts]
        stride = -(-page_size * (db + sb) // 16) * 16
        n = sum(pages) + 2
        self.host = rng.integers(0, 256, (n, stride), dtype=np.uint8)
        order = rng.permutation(n - 1)[:sum(pages)] + 1
        self.table = np.full((len(counts), max(pages + [1]) + extra_width), n + 5, np.int32)
        at = 0
        for b, c in enumerate(counts):
            self.table[b, :pages[b]] = order[at:at + pages[b]]
            at += pages[b]
            if c:
                x = rng.standard_normal((c, 512)).astype(np.float32) * scale
                x[rng.random(c) < 0.02] = 0
                x[:, rng.integers(0, 512, 3)] *= 12
                bits = (torch.from_numpy(x).bfloat16().view(torch.int16).numpy().view(np.uint16))
                ids = np.arange(c)
                slots = self.table[b, ids // page_size].astype(np.int64) * page_size + ids % page_size
                oracle.store_rows(self.host, layout, page_size, bits, slots.astype(np.int32))
        self.layout, self.page_size = layout, page_size
        self.cache = kvc.Cache(dev(self.host), layout, page_size)

    def rows(self, b, count):
        return ref.cached_rows(self.host, self.layout, self.page_size, self.table[b], count)


def queries(T, H, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, H, 512, generator=g) * scale).bfloat16()


SCALE = 512 ** -0.5


def prefill_seen(start, n, ratio, count):
    lim = (start + torch.arange(n) + 1) // ratio
    return torch.arange(count)[None] < lim[:, None]


def tree_seen(start, masks, count):
    r = torch.arange(count)[None] - start
    m = torch.tensor([[(x >> i) & 1 for i in range(64)] for x in masks], dtype=torch.bool)
    return (r < 0) | (m[:, r[0].clamp(0, 63)] & (r >= 0) & (r < len(masks)))


def random_tree(D, rng):
    m = []
    for j in range(D):
        parent = rng.randint(max(-1, j - 5), j - 1)
        m.append((m[parent] if parent >= 0 else 0) | 1 << j)
    return m


def as_i64(masks):
    return torch.tensor([[x - (1 << 64) if x >> 63 else x for x in row] for row in masks],
                        dtype=torch.int64)


# layout, page, ratio, heads, [(start, new) per slot], sink
PREFILL = [
    ("V41", 64, 2, 8, [(0, 64)], False),
    ("V41", 64, 1, 16, [(0, 1)], False),                 # a single token, a single row
    ("V41", 64, 1, 128, [(0, 37)], True),
    ("V41_FP4", 128, 2, 32, [(0, 33), (0, 1), (0, 2), (0, 160)], True),
    ("V4", 64, 1, 24, [(0, 5), (31, 40), (257, 3)], False),
    ("V41", 16, 1, 5, [(0, 100), (100, 31)], True),      # a head count that divides no tile
    ("V41_FP4", 1, 1, 3, [(0, 70)], False),              # a page per row
    ("V4", 4096, 2, 64, [(511, 66)], True),              # an odd start
    ("V41", 64, 1, 1, [(0, 300)], False),
    ("V41", 64, 2, 100, [(0, 1)], False),                # no row to see
    ("V41", 64, 2, 16, [(0, 1), (0, 1), (0, 3)], True),  # the same, with a sink
    ("V41_FP4", 64, 1, 129, [(63, 2), (64, 2), (65, 2)], False),
    ("V41", 32, 1, 16, [(0, 0), (7, 9), (0, 0), (0, 0), (3, 1)], False),  # empty slots
    ("V4", 64, 1, 8, [(4000, 17)], True),                # few queries, many rows: cut units
    ("V41", 64, 1, 16, [(0, 700)], False),
    ("V41_FP4", 64, 2, 1024, [(9, 2)], False),
]


@pytest.mark.parametrize("layout,page,ratio,H,slots,sink", PREFILL)
def test_prefill(kvc, layout, page, ratio, H, slots, sink):
    seed = page + 3 * H + 7 * len(slots)
    counts = [(s + n) // ratio for s, n in slots]
    f = Filled(kvc, layout, page, counts, seed)
    T = sum(n for _, n in slots)
    q = queries(T, H, seed)
    sk = torch.randn(H) if sink else None
    first = np.cumsum([0] + [n for _, n in slots])[:-1]
    off = torch.tensor(np.array([first, [n for _, n in slots]]), dtype=torch.int32).cuda()
    start = torch.tensor([s for s, _ in slots], dtype=torch.int32).cuda()
    out = torch.full((T, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvc.kvc_attend_prefill(f.cache, q.cuda(), off, start, dev(f.table), out, scale=SCALE,
                           ratio=ratio, sink=None if sk is None else sk.cuda(), lse=lse, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    for b, (s, n) in enumerate(slots):
        if n == 0:
            continue
        rows, valid = f.rows(b, counts[b])
        assert valid.all()
        t = slice(int(first[b]), int(first[b]) + n)
        r = ref.attend(q[t].double(), rows, prefill_seen(s, n, ratio, counts[b]), SCALE, sk)
        ref.check(out[t], lse[t], r, f"slot {b}")


# layout, page, ratio, heads, D, starts, tree, sink
TREE = [
    ("V41", 64, 1, 16, 1, [1000], False, False),
    ("V41", 64, 1, 8, 1, [0, 1, 63, 64, 65, 500], False, True),
    ("V41_FP4", 64, 1, 64, 1, [5, 300, 129], False, False),
    ("V4", 64, 2, 16, 4, [0, 1, 2, 127, 600], False, True),
    ("V41", 16, 1, 16, 7, [0, 33, 250], True, False),
    ("V41_FP4", 128, 1, 12, 64, [0, 77], True, True),
    ("V4", 64, 1, 1, 1, [700], False, False),
    ("V41", 64, 1, 128, 2, [31, 90], True, False),
    ("V41", 1, 1, 32, 1, [40, 41], False, False),
    ("V41_FP4", 64, 2, 128, 3, [0, 9], False, False),
    ("V4", 64, 1, 21, 3, [200, 0, 1], True, True),
    ("V41", 64, 1, 8, 1, [9000], False, False),          # one query block, cut between many
    ("V41_FP4", 64, 1, 16, 4, [6000, 3], True, True),
    ("V4", 64, 1, 40, 1, [5000, 4000], False, False),
]


@pytest.mark.parametrize("layout,page,ratio,H,D,starts,tree,sink", TREE)
def test_tree(kvc, layout, page, ratio, H, D, starts, tree, sink):
    seed = page + 3 * H + 7 * D
    rng = random.Random(seed)
    counts = [(s + D) // ratio for s in starts]
    f = Filled(kvc, layout, page, counts, seed)
    S = len(starts)
    q = queries(S * D, H, seed)
    sk = torch.randn(H) if sink else None
    masks = [random_tree(D, rng) for _ in starts] if tree else None
    out = torch.full((S * D, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((S * D, H), 7.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvc.kvc_attend_tree(f.cache, q.cuda(), torch.tensor(starts, dtype=torch.int32).cuda(),
                        dev(f.table), out, scale=SCALE, draft_len=D, ratio=ratio,
                        tree=as_i64(masks).cuda() if tree else None,
                        sink=None if sk is None else sk.cuda(), lse=lse, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    for b, s in enumerate(starts):
        rows, _ = f.rows(b, counts[b])
        seen = tree_seen(s, masks[b], counts[b]) if tree else prefill_seen(s, D, ratio, counts[b])
        t = slice(b * D, b * D + D)
        ref.check(out[t], lse[t], ref.attend(q[t].double(), rows, seen, SCALE, sk), f"slot {b}")


@pytest.mark.parametrize("scale_q,scale", [(6.0, SCALE), (0.05, SCALE), (1.0, 3.0), (1.0, 1e-4)])
def test_sharp_and_flat_scores(kvc, scale_q, scale):
    """One row taking nearly all the weight, maxima that rise late, and weights
    all alike."""
    f = Filled(kvc, "V41", 64, [900], 5)
    q = queries(3, 16, 5, scale_q)
    out = torch.empty(3, 16, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(3, 16, device="cuda")
    kvc.kvc_attend_tree(f.cache, q.cuda(), torch.tensor([897], dtype=torch.int32).cuda(),
                        dev(f.table), out, scale=scale, draft_len=3, lse=lse)
    rows, _ = f.rows(0, 900)
    ref.check(out, lse, ref.attend(q.double(), rows, prefill_seen(897, 3, 1, 900), scale))


@pytest.mark.parametrize("layout", LAYOUTS)
def test_empty_masks_of_a_tree(kvc, layout):
    """Drafted tokens whose mask leaves nothing (no context either): 0 and -inf,
    or the sink; the other tokens of the slot are as usual."""
    D, H = 5, 16
    f = Filled(kvc, layout, 64, [D, 130 + D], 3)
    masks = [[0, 1, 0, 0b111, 0], [0, 0, 0b11, 1 << 4, ~0 & (1 << 64) - 1]]
    q = queries(2 * D, H, 3)
    for sk in (None, torch.randn(H)):
        out = torch.full((2 * D, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((2 * D, H), 7.0, device="cuda")
        kvc.kvc_attend_tree(f.cache, q.cuda(), torch.tensor([0, 130], dtype=torch.int32).cuda(),
                            dev(f.table), out, scale=SCALE, draft_len=D, tree=as_i64(masks).cuda(),
                            sink=None if sk is None else sk.cuda(), lse=lse)
        for b, s in enumerate((0, 130)):
            rows, _ = f.rows(b, s + D)
            t = slice(b * D, b * D + D)
            ref.check(out[t], lse[t], ref.attend(q[t].double(), rows, tree_seen(s, masks[b], s + D),
                                                 SCALE, sk), f"slot {b}")
        assert (out[0].float() == 0).all()
        want = torch.full((H,), float("-inf")) if sk is None else sk * ref.LOG2E
        assert torch.allclose(lse[0].cpu(), want, rtol=1e-6, atol=0)


@pytest.mark.parametrize("layout,H", [("V41", 16), ("V4", 8), ("V41_FP4", 64), ("V41", 128)])
def test_nan_rows_reach_only_those_that_see_them(kvc, layout, H):
    """NaN (and in V4's rope dims infinite) rows among the drafted ones: the
    tokens that see them are NaN, the others untouched; the random bytes behind
    the last row reach nobody."""
    D, start = 6, 70
    f = Filled(kvc, layout, 64, [start + D], 11)
    db, sb, _, _ = oracle.layout_bytes(layout)
    for r in (start + 2, start + 4):
        page, i = int(f.table[0, r // 64]), r % 64
        if layout == "V41_FP4":
            f.host[page, 64 * db + i * sb + 3] = 0x7F          # a NaN scale
        else:
            f.host[page, i * db + 17] = 0x7F                   # a NaN code
    f.cache = kvc.Cache(dev(f.host), layout, 64)
    masks = [0b000001, 0b000011, 0b000101, 0b001011, 0b010101, 0b100011]
    q = queries(D, H, 11)
    out = torch.empty(D, H, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(D, H, device="cuda")
    kvc.kvc_attend_tree(f.cache, q.cuda(), torch.tensor([start], dtype=torch.int32).cuda(),
                        dev(f.table), out, scale=SCALE, draft_len=D, tree=as_i64([masks]).cuda(),
                        lse=lse)
    rows, _ = f.rows(0, start + D)
    seen = tree_seen(start, masks, start + D)
    ref.check(out, lse, ref.attend(q.double(), rows, seen, SCALE))
    nan = torch.isnan(out.float()).all(2).all(1).cpu()
    assert nan.tolist() == [False, False, True, False, True, False]


def test_causal_nan_row(kvc):
    """A NaN row in a prompt: earlier tokens, in the same tile too, are exact."""
    n, H = 90, 32
    f = Filled(kvc, "V41", 64, [n], 13)
    db = 512
    page, i = int(f.table[0, 50 // 64]), 50
    f.host[page, i * db + 3] = 0xFF
    f.cache = kvc.Cache(dev(f.host), "V41", 64)
    q = queries(n, H, 13)
    out = torch.empty(n, H, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(n, H, device="cuda")
    off = torch.tensor([[0], [n]], dtype=torch.int32).cuda()
    kvc.kvc_attend_prefill(f.cache, q.cuda(), off, torch.zeros(1, dtype=torch.int32).cuda(),
                           dev(f.table), out, scale=SCALE, lse=lse)
    rows, _ = f.rows(0, n)
    ref.check(out, lse, ref.attend(q.double(), rows, prefill_seen(0, n, 1, n), SCALE))


def test_infinite_rope_values_in_masked_rows(kvc):
    D, start, H = 4, 33, 16
    f = Filled(kvc, "V4", 64, [start + D], 17)
    page = int(f.table[0, 0])
    f.host[page, (start + 1) * 576 + 448 + 6: (start + 1) * 576 + 448 + 8] = (0x80, 0x7F)   # +inf
    f.cache = kvc.Cache(dev(f.host), "V4", 64)
    masks = [0b0001, 0b0001, 0b0101, 0b1000]                   # nobody sees row start + 1
    q = queries(D, H, 17)
    out = torch.empty(D, H, 512, dtype=torch.bfloat16, device="cuda")
    kvc.kvc_attend_tree(f.cache, q.cuda(), torch.tensor([start], dtype=torch.int32).cuda(),
                        dev(f.table), out, scale=SCALE, draft_len=D, tree=as_i64([masks]).cuda())
    rows, _ = f.rows(0, start + D)
    rows[start + 1] = 0
    ref.check(out, None, ref.attend(q.double(), rows, tree_seen(start, masks, start + D), SCALE))


def test_pages_outside_the_cache_are_left_out(kvc):
    """A page past the cache, a negative one and a table too narrow: their rows
    are masked and flagged."""
    H, n = 16, 400
    f = Filled(kvc, "V41", 64, [n], 19, extra_width=0)
    f.table[0, 1], f.table[0, 3] = f.host.shape[0], -7
    q = queries(1, H, 19)
    out = torch.empty(1, H, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(1, H, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    wide = np.full((2, 9), 2, np.int32)
    wide[0, :7] = f.table[0]
    for width, bits in ((7, kvc.STATUS_PAGE_RANGE), (5, kvc.STATUS_PAGE_RANGE | kvc.STATUS_PT_RANGE)):
        st.zero_()
        kvc.kvc_attend_tree(f.cache, q.cuda(), torch.tensor([n - 1], dtype=torch.int32).cuda(),
                            dev(wide)[:1, :width], out, scale=SCALE, lse=lse, status=st)
        assert int(st) == bits
        rows, valid = ref.cached_rows(f.host, "V41", 64, wide[0, :width], n)
        assert int((~valid).sum()) == 128 + (n - 320 if width == 5 else 0)
        ref.check(out, lse, ref.attend(q.double(), rows, valid[None], SCALE))


@pytest.mark.parametrize("H", [8, 33, 96])
def test_skipped_slots_and_padding_are_left_alone(kvc, H):
    """Inactive slots, slots without tokens, slots outside q, padded rows: out
    and lse keep their bytes there."""
    f = Filled(kvc, "V41", 64, [50, 60, 70, 80, 0], 23)
    T = 40
    q = queries(T, H, 23)
    out = torch.full((T, H, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 3.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    off = torch.tensor([[4, 10, 12, 20, 37], [5, -3, 6, 7, 9]], dtype=torch.int32).cuda()
    start = torch.tensor([45, 60, -1, 73, 0], dtype=torch.int32).cuda()
    kvc.kvc_attend_prefill(f.cache, q.cuda(), off, start, dev(f.table), out, scale=SCALE, lse=lse,
                           status=st)
    assert int(st) == kvc.STATUS_TOKEN_RANGE                    # slot 4: rows 37 .. 45 of 40
    used = torch.zeros(T, dtype=torch.bool)
    for b, t0, n, s in ((0, 4, 5, 45), (3, 20, 7, 73)):
        rows, _ = f.rows(b, s + n)
        t = slice(t0, t0 + n)
        used[t] = True
        ref.check(out[t], lse[t], ref.attend(q[t].double(), rows, prefill_seen(s, n, 1, s + n), SCALE))
    assert (out.cpu()[~used] == 3.0).all() and (lse.cpu()[~used] == 3.0).all()
    # tree: an inactive slot between two active ones, and rows past the last
    out.fill_(3.0)
    lse.fill_(3.0)
    starts = torch.tensor([47, -1, 67], dtype=torch.int32).cuda()
    kvc.kvc_attend_tree(f.cache, q.cuda(), starts, dev(f.table), out, scale=SCALE, draft_len=3,
                        lse=lse)
    for b, s in ((0, 47), (2, 67)):
        rows, _ = f.rows(b, s + 3)
        t = slice(3 * b, 3 * b + 3)
        ref.check(out[t], lse[t], ref.attend(q[t].double(), rows, prefill_seen(s, 3, 1, s + 3), SCALE))
    keep = torch.ones(T, dtype=torch.bool)
    keep[0:3] = keep[6:9] = False
    assert (out.cpu()[keep] == 3.0).all() and (lse.cpu()[keep] == 3.0).all()


def test_positions_past_int32_are_refused_on_the_device(kvc):
    f = Filled(kvc, "V41", 64, [64], 29)
    out = torch.full((2, 8, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvc.kvc_attend_tree(f.cache, queries(2, 8, 1).cuda(),
                        torch.tensor([2 ** 31 - 1, 63], dtype=torch.int32).cuda(),
                        dev(np.repeat(f.table, 2, 0)), out, scale=SCALE, status=st)
    assert int(st) == kvc.STATUS_POS_RANGE
    assert (out[0] == 3.0).all() and not (out[1] == 3.0).any()


@pytest.mark.parametrize("H,D", [(16, 1), (24, 3)])
def test_strides(kvc, H, D):
    """q and out as parts of wider buffers, head-major, and one query row for
    all tokens; the page table as columns of a wider one."""
    starts = [100, 37]
    f = Filled(kvc, "V41_FP4", 64, [s + D for s in starts], 31)
    T = 2 * D
    st = torch.tensor(starts, dtype=torch.int32).cuda()
    wide = np.full((2, f.table.shape[1] + 6), 10 ** 6, np.int32)
    wide[:, 3:3 + f.table.shape[1]] = f.table
    table = dev(wide)[:, 3:3 + f.table.shape[1]]
    base = queries(T, H, 31)

    def run(q, out):
        kvc.kvc_attend_tree(f.cache, q, st, table, out, scale=SCALE, draft_len=D)
        torch.cuda.synchronize()

    plain = torch.empty(T, H, 512, dtype=torch.bfloat16, device="cuda")
    run(base.cuda(), plain)
    for b, s in enumerate(starts):
        rows, _ = f.rows(b, s + D)
        t = slice(b * D, b * D + D)
        ref.check(plain[t], None, ref.attend(base[t].double(), rows, prefill_seen(s, D, 1, s + D), SCALE))
    buf = torch.full((T, H + 3, 640), 5.0, dtype=torch.bfloat16, device="cuda")
    buf[:, 2:2 + H, 64:576] = base.cuda()
    obuf = torch.full((T + 1, H + 2, 520), 5.0, dtype=torch.bfloat16, device="cuda")
    run(buf[:, 2:2 + H, 64:576], obuf[:T, 1:1 + H, :512])
    assert torch.equal(obuf[:T, 1:1 + H, :512], plain)
    rest = torch.ones_like(obuf, dtype=torch.bool)
    rest[:T, 1:1 + H, :512] = False
    assert (obuf[rest] == 5.0).all()
    qt = base.cuda().transpose(0, 1).contiguous().transpose(0, 1)         # head-major
    ot = torch.empty(H, T, 512, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    run(qt, ot)
    assert torch.equal(ot, plain)
    one = base[:1, :1].cuda().expand(T, H, 512)
    got, want = torch.empty_like(plain), torch.empty_like(plain)
    run(one, got)
    run(one.contiguous(), want)
    assert torch.equal(got, want)


def test_far_pages(kvc):
    """A cache past 4 GiB: rows at both ends of it."""
    ps, pages = 64, 140_000
    cache = torch.zeros(pages, ps * 528, dtype=torch.uint8, device="cuda")
    f = Filled(kvc, "V41", ps, [300], 37)
    table = np.array([[pages - 1, 1, pages - 2, 70_000, pages // 2 + 77]], np.int32)
    for i in range(5):
        cache[int(table[0, i])] = dev(f.host[f.table[0, i]])
    q = queries(1, 16, 37)
    out = torch.empty(1, 16, 512, dtype=torch.bfloat16, device="cuda")
    kvc.kvc_attend_tree(kvc.Cache(cache, "V41", ps), q.cuda(),
                        torch.tensor([299], dtype=torch.int32).cuda(), dev(table), out, scale=SCALE)
    rows, _ = f.rows(0, 300)
    ref.check(out, None, ref.attend(q.double(), rows, prefill_seen(299, 1, 1, 300), SCALE))


def test_long_ragged_batch_cut_everywhere(kvc):
    """Many units cut between workgroups at once: 40 slots of 1 .. 2600 rows."""
    rng = random.Random(41)
    starts = [rng.randint(1, 2600) for _ in range(40)]
    f = Filled(kvc, "V41", 64, [s + 2 for s in starts], 41)
    q = queries(80, 24, 41)
    out = torch.empty(80, 24, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(80, 24, device="cuda")
    kvc.kvc_attend_tree(f.cache, q.cuda(), torch.tensor(starts, dtype=torch.int32).cuda(),
                        dev(f.table), out, scale=SCALE, draft_len=2, lse=lse)
    for b, s in enumerate(starts):
        rows, _ = f.rows(b, s + 2)
        t = slice(2 * b, 2 * b + 2)
        ref.check(out[t], lse[t], ref.attend(q[t].double(), rows, prefill_seen(s, 2, 1, s + 2), SCALE),
                  f"slot {b}")


# at and past the units up to which workgroups plan for themselves
@pytest.mark.parametrize("S,D,H", [(256, 1, 16), (257, 1, 40), (64, 4, 128), (65, 4, 128), (1, 64, 513)])
def test_batches_around_the_planning_limit(kvc, S, D, H):
    rng = random.Random(S + H)
    starts = [rng.choice((-1, 0, 1, 62, 63, rng.randint(2, 150))) for _ in range(S)]
    starts[0] = 150
    f = Filled(kvc, "V41", 64, [max(0, s + D) if s >= 0 else 0 for s in starts], S)
    q = queries(S * D, H, S)
    out = torch.full((S * D, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((S * D, H), 7.0, device="cuda")
    kvc.kvc_attend_tree(f.cache, q.cuda(), torch.tensor(starts, dtype=torch.int32).cuda(),
                        dev(f.table), out, scale=SCALE, draft_len=D, lse=lse)
    out, lse = out.cpu(), lse.cpu()
    for b, s in enumerate(starts):
        t = slice(b * D, b * D + D)
        if s < 0:
            assert (out[t] == 7.0).all() and (lse[t] == 7.0).all()
            continue
        rows, _ = f.rows(b, s + D)
        ref.check(out[t], lse[t], ref.attend(q[t].double(), rows, prefill_seen(s, D, 1, s + D), SCALE),
                  f"slot {b}")


@pytest.mark.parametrize("S,H,most", [(70, 100, 9), (200, 8, 3), (3, 16, 400)])
def test_packed_batches_of_many_prompts(kvc, S, H, most):
    rng = random.Random(S + H)
    slots = [(rng.randint(0, 90), rng.choice((0, 1, rng.randint(0, most)))) for _ in range(S)]
    slots[-1] = (17, most)
    counts = [s + n for s, n in slots]
    f = Filled(kvc, "V41_FP4", 32, counts, S)
    T = sum(n for _, n in slots) + 5                     # and padded rows
    q = queries(T, H, S)
    first = np.cumsum([0] + [n for _, n in slots])[:-1]
    off = torch.tensor(np.array([first, [n for _, n in slots]]), dtype=torch.int32).cuda()
    out = torch.full((T, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    kvc.kvc_attend_prefill(f.cache, q.cuda(), off, torch.tensor([s for s, _ in slots], dtype=torch.int32).cuda(),
                           dev(f.table), out, scale=SCALE, lse=lse)
    out, lse = out.cpu(), lse.cpu()
    for b, (s, n) in enumerate(slots):
        if n == 0:
            continue
        rows, _ = f.rows(b, s + n)
        t = slice(int(first[b]), int(first[b]) + n)
        ref.check(out[t], lse[t], ref.attend(q[t].double(), rows, prefill_seen(s, n, 1, s + n), SCALE),
                  f"slot {b}")
    assert (out[T - 5:] == 7.0).all() and (lse[T - 5:] == 7.0).all()


@pytest.mark.parametrize("packed", [False, True])
def test_most_slots_few_of_them_active(kvc, packed):
    S, H, D = 8191, 3, 2
    rng = random.Random(67 + packed)
    active = sorted(rng.sample(range(S), 40) + [0, S - 1])
    starts, new = [-1] * S, [0] * S
    for b in active:
        starts[b], new[b] = rng.randint(0, 90), rng.randint(1, 5) if packed else D
    counts = [s + n if s >= 0 else 0 for s, n in zip(starts, new)]
    f = Filled(kvc, "V41", 64, counts, 67)
    first = np.cumsum([0] + new)[:-1] if packed else np.arange(S) * D
    T = sum(new) if packed else S * D
    q = queries(T, H, 67)
    out = torch.full((T, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    start = torch.tensor(starts, dtype=torch.int32).cuda()
    if packed:
        off = torch.tensor(np.array([first, new]), dtype=torch.int32).cuda()
        kvc.kvc_attend_prefill(f.cache, q.cuda(), off, start, dev(f.table), out, scale=SCALE, lse=lse)
    else:
        kvc.kvc_attend_tree(f.cache, q.cuda(), start, dev(f.table), out, scale=SCALE, draft_len=D, lse=lse)
    out, lse = out.cpu(), lse.cpu()
    rest = torch.ones(T, dtype=torch.bool)
    for b in active:
        s, n = starts[b], new[b]
        rows, _ = f.rows(b, s + n)
        t = slice(int(first[b]), int(first[b]) + n)
        rest[t] = False
        ref.check(out[t], lse[t], ref.attend(q[t].double(), rows, prefill_seen(s, n, 1, s + n), SCALE),
                  f"slot {b}")
    assert (out[rest] == 7.0).all() and (lse[rest] == 7.0).all()


def test_repeats_bit_for_bit_and_on_another_stream(kvc):
    starts = [1200, 30, 500]
    f = Filled(kvc, "V41", 64, [s + 4 for s in starts], 43)
    q = queries(12, 32, 43).cuda()
    args = (f.cache, q, torch.tensor(starts, dtype=torch.int32).cuda(), dev(f.table))
    first = torch.empty_like(q)
    kvc.kvc_attend_tree(*args, first, scale=SCALE, draft_len=4)
    torch.cuda.synchronize()
    space = torch.full((kvc.kvc_attend_workspace(3, 12, 32) + 512,), 0xFF, dtype=torch.uint8,
                       device="cuda")[:-512]
    side = torch.cuda.Stream()
    for k in range(3):
        again = torch.empty_like(q)
        side.wait_stream(torch.cuda.current_stream())
        kvc.kvc_attend_tree(*args, again, scale=SCALE, draft_len=4, stream=side if k else None,
                            workspace=space if k < 2 else None)
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(first, again)


def test_two_calls_at_once_with_a_workspace_each(kvc):
    f = Filled(kvc, "V41_FP4", 64, [3000, 2000], 47)
    t = dev(f.table)
    qs = [queries(2, 64, 47 + i).cuda() for i in range(2)]
    st = torch.tensor([2999, 1999], dtype=torch.int32).cuda()
    want = []
    for q in qs:
        o = torch.empty_like(q)
        kvc.kvc_attend_tree(f.cache, q, st, t, o, scale=SCALE)
        torch.cuda.synchronize()
        want.append(o)
    streams = [torch.cuda.Stream() for _ in qs]
    got = [torch.zeros_like(q) for q in qs]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, q, o in zip(streams, qs, got):
            kvc.kvc_attend_tree(f.cache, q, st, t, o, scale=SCALE, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        assert torch.equal(o, w)


def test_graph_replays_follow_refreshed_inputs(kvc):
    """One capture; every replay reads the lengths, tables and queries of its
    moment, with eager calls of the same operator in between."""
    H, D = 16, 2
    f = Filled(kvc, "V41", 64, [3000, 3000], 53)
    table = dev(f.table)
    q = queries(2 * D, H, 53).cuda()
    start = torch.tensor([10, 20], dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    lse = torch.empty(2 * D, H, device="cuda")
    other = torch.empty_like(q)
    kvc.kvc_attend_tree(f.cache, q, start, table, out, scale=SCALE, draft_len=D, lse=lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvc.kvc_attend_tree(f.cache, q, start, table, out, scale=SCALE, draft_len=D, lse=lse)
    for k, starts in enumerate(([2990, 5], [-1, 900], [64, 63], [0, 2998], [2990, 5])):
        qn = queries(2 * D, H, 60 + k)
        q.copy_(qn)
        start.copy_(torch.tensor(starts, dtype=torch.int32))
        out.fill_(3.0)
        g.replay()
        kvc.kvc_attend_tree(f.cache, q, start, table, other, scale=SCALE, draft_len=D)
        torch.cuda.synchronize()
        for b, s in enumerate(starts):
            t = slice(b * D, b * D + D)
            if s < 0:
                assert (out[t] == 3.0).all()
                continue
            assert torch.equal(out[t], other[t])
            rows, _ = f.rows(b, s + D)
            ref.check(out[t], lse[t], ref.attend(qn[t].double(), rows, prefill_seen(s, D, 1, s + D),
                                                 SCALE), f"replay {k} slot {b}")


def test_graph_replays_of_a_packed_batch_with_its_own_plan(kvc):
    """A batch planned by a kernel of its own, captured once: every replay
    follows the offsets and starts of its moment, eager calls in between."""
    S, H, T = 40, 100, 150
    f = Filled(kvc, "V4", 64, [300] * S, 71)
    table = dev(f.table)
    q = queries(T, H, 71)
    qd = q.cuda()
    off = torch.zeros(2, S, dtype=torch.int32).cuda()
    start = torch.zeros(S, dtype=torch.int32).cuda()
    out = torch.empty_like(qd)
    other = torch.empty_like(qd)
    lse = torch.empty(T, H, device="cuda")
    kvc.kvc_attend_prefill(f.cache, qd, off, start, table, out, scale=SCALE, lse=lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvc.kvc_attend_prefill(f.cache, qd, off, start, table, out, scale=SCALE, lse=lse)
    for k in range(4):
        rng = random.Random(80 + k)
        new = [rng.choice((0, 1, 3, 7)) for _ in range(S)]
        while sum(new) > T:
            new[new.index(max(new))] = 0
        starts = [rng.randint(0, 290) for _ in range(S)]
        if k == 2:
            starts = [-1] * S                 # nothing to do
        first = np.cumsum([0] + new)[:-1]
        off.copy_(torch.tensor(np.array([first, new]), dtype=torch.int32))
        start.copy_(torch.tensor(starts, dtype=torch.int32))
        out.fill_(3.0)
        other.fill_(3.0)
        g.replay()
        kvc.kvc_attend_prefill(f.cache, qd, off, start, table, other, scale=SCALE)
        torch.cuda.synchronize()
        assert torch.equal(out, other)
        for b in [b for b in range(S) if new[b] and starts[b] >= 0][::7]:
            rows, _ = f.rows(b, starts[b] + new[b])
            t = slice(int(first[b]), int(first[b]) + new[b])
            ref.check(out[t], lse[t], ref.attend(q[t].double(), rows,
                                                 prefill_seen(starts[b], new[b], 1, starts[b] + new[b]),
                                                 SCALE), f"replay {k} slot {b}")
        assert (out[sum(new):] == 3.0).all()


def test_zero_slots_and_zero_rows(kvc):
    f = Filled(kvc, "V41", 64, [64], 59)
    e = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")
    q = torch.empty(0, 8, 512, dtype=torch.bfloat16, device="cuda")
    kvc.kvc_attend_tree(f.cache, q, e(0), e(0, 4), torch.empty_like(q), scale=SCALE)
    kvc.kvc_attend_prefill(f.cache, q, torch.zeros(2, 1, dtype=torch.int32).cuda(),
                           torch.zeros(1, dtype=torch.int32).cuda(), dev(f.table),
                           torch.empty_like(q), scale=SCALE)
    q = queries(3, 8, 1).cuda()
    out = torch.full_like(q, 3.0)
    kvc.kvc_attend_prefill(f.cache, q, torch.zeros(2, 2, dtype=torch.int32).cuda(),
                           torch.zeros(2, dtype=torch.int32).cuda(), dev(np.repeat(f.table, 2, 0)),
                           out, scale=SCALE)
    torch.cuda.synchronize()
    assert (out == 3.0).all()
