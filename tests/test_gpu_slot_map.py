"""kvc_slot_map on the GPU against Python integers, and a step of the library's
calls run off its tables: slot map, rotary store, attention."""
import random

import numpy as np
import pytest
import torch

import oracle
import workloads as W
from tests import attend_ref as ref
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    import fp8_fp4_quantized_amd as k
    return k


def batch(S, ratio, ps, held, new, rng, spare=5, width=None):
    lens = [rng.randint(*held) for _ in range(S)]
    n = [rng.randint(*new) for _ in range(S)]
    up = lambda a, b: -(-a // b)
    have = [up(max(l, 0) // ratio, ps) for l in lens]
    want = [up((max(l, 0) + max(k, 0)) // ratio, ps) for l, k in zip(lens, n)]
    w = max(want + [1]) + 1 if width is None else width
    pages = list(range(1, sum(have) + sum(want) + spare + 1))
    rng.shuffle(pages)
    table = np.full((S, w), -9, np.int32)
    for b in range(S):
        for k in range(min(have[b], w)):
            table[b, k] = pages.pop()
    free = np.array(pages[:max(0, sum(want) - sum(have) + spare)], np.int32)
    return lens, n, table, free, sum(have) + sum(want) + spare + 1


def run(kvc, *, lens, new_lens, table, free, ratio, ps, num_pages, tokens, stride=0, depth=None,
        fill=77):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    S = len(lens)
    e = lambda *s: torch.full(s, fill, dtype=torch.int32, device="cuda")
    o = dict(offsets=e(2, S), start_pos=e(S), out_loc=e(tokens + 3), positions=e(tokens + 3),
             token_to_req=e(tokens + 3), totals=e(4))
    t = dev(table)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(2):                       # repeating the call changes nothing
        kvc.kvc_slot_map(ratio=ratio, page_size=ps, num_pages=num_pages, lens=i32(lens),
                         new_lens=None if new_lens is None else i32(new_lens), page_table=t,
                         free_pages=dev(free), token_stride=stride,
                         depth=None if depth is None else i32(depth), max_tokens=tokens, status=st,
                         **o)
    torch.cuda.synchronize()
    want, bits = ref.slot_map(ratio=ratio, page_size=ps, num_pages=num_pages, lens=lens,
                              new_lens=new_lens, page_table=table, free_pages=free,
                              max_tokens=tokens, token_stride=stride, depth=depth)
    for k in ("offsets", "start_pos", "totals"):
        np.testing.assert_array_equal(host(o[k]), want[k], err_msg=k)
    for k in ("out_loc", "positions", "token_to_req"):
        got = host(o[k])
        np.testing.assert_array_equal(got[:tokens], want[k], err_msg=k)
        assert (got[tokens:] == fill).all(), k
    np.testing.assert_array_equal(host(t), want["page_table"], err_msg="page_table")
    assert int(st) == bits
    return want, bits


PACKED = [  # slots, ratio, page, held, new
    (1, 1, 64, (0, 0), (1, 1)),
    (1, 2, 64, (0, 0), (1, 1)),
    (1, 2, 1, (3, 3), (64, 64)),
    (16, 2, 128, (0, 0), (1500, 2600)),
    (300, 1, 16, (0, 900), (0, 37)),
    (1023, 2, 64, (0, 500), (-2, 9)),
    (1024, 1, 64, (-3, 500), (0, 3)),
    (1025, 1, 4, (0, 60), (0, 5)),
    (8191, 2, 64, (-1, 300), (0, 3)),
    (5, 1, 4096, (0, 9000), (0, 9000)),
    (64, 1, 64, (64, 64), (64, 64)),        # whole pages, exactly
]


@pytest.mark.parametrize("S,ratio,ps,held,new", PACKED)
def test_packed(kvc, S, ratio, ps, held, new):
    lens, n, table, free, num = batch(S, ratio, ps, held, new, random.Random(S + ratio))
    tokens = sum(k for l, k in zip(lens, n) if l >= 0 and k > 0)
    for cap in (tokens, tokens + 131):
        _, bits = run(kvc, lens=lens, new_lens=n, table=table, free=free, ratio=ratio, ps=ps,
                      num_pages=num, tokens=cap)
        assert bits == 0


STRIDED = [  # slots, ratio, page, D, held, given lengths, depths
    (1024, 2, 64, 1, (0, 4000), False, False),
    (7, 1, 16, 64, (0, 100), True, True),
    (200, 1, 64, 5, (-2, 700), True, False),
    (129, 2, 64, 4, (0, 300), True, False),
    (33, 1, 1, 7, (0, 40), False, True),
]


@pytest.mark.parametrize("S,ratio,ps,D,held,given,deep", STRIDED)
def test_strided(kvc, S, ratio, ps, D, held, given, deep):
    rng = random.Random(S + D)
    lens, n, table, free, num = batch(S, ratio, ps, held, (-1, D) if given else (D, D), rng)
    tokens = S * D + 9
    depth = [rng.randint(0, 6) for _ in range(tokens)] if deep else None
    run(kvc, lens=lens, new_lens=n if given else None, table=table, free=free, ratio=ratio, ps=ps,
        num_pages=num, tokens=tokens, stride=D, depth=depth)


@pytest.mark.parametrize("stride", [0, 20])
def test_refusals_on_the_device(kvc, stride):
    """A free list that runs short, a table too narrow, too many tokens: those
    slots are refused whole, in the documented order, and flagged."""
    rng = random.Random(9)
    for trial in range(12):
        S = rng.choice([3, 40, 1100])
        ratio, ps = rng.choice([1, 2]), rng.choice([4, 16])
        lens, n, table, free, num = batch(S, ratio, ps, (-1, 90), (0, 25), rng)
        total = sum(k for l, k in zip(lens, n) if l >= 0)
        free = free[:rng.randint(0, len(free))]
        if trial % 3 == 0:
            table = table[:, :max(1, table.shape[1] - 2)].copy()
        tokens = S * stride if stride else rng.randint(0, total + 5)
        run(kvc, lens=lens, new_lens=n, table=table, free=free, ratio=ratio, ps=ps, num_pages=num,
            tokens=tokens, stride=stride)


def test_lengths_near_int32_and_huge_requests(kvc):
    """Lengths whose sums pass 32 bits are refused, not wrapped."""
    big = 2 ** 31 - 1
    lens = [big, big - 3, 0, 5, 7]
    n = [1, 3, big, 2, big]
    table = np.arange(20, dtype=np.int32).reshape(5, 4) + 1
    w, bits = run(kvc, lens=lens, new_lens=n, table=table, free=np.array([90, 91], np.int32), ratio=1,
                  ps=64, num_pages=100, tokens=8)
    assert w["start_pos"].tolist() == [-1, -1, -1, 5, -1] and bits == kvc.STATUS_PT_RANGE


def test_pages_outside_the_cache(kvc):
    lens, n = [10, 3, 0], [10, 3, 4]
    table = np.array([[50, 0], [-4, 0], [0, 0]], np.int32)
    w, bits = run(kvc, lens=lens, new_lens=n, table=table, free=np.array([7, 99], np.int32), ratio=1,
                  ps=16, num_pages=50, tokens=17)
    assert bits == kvc.STATUS_PAGE_RANGE
    assert w["out_loc"].tolist()[:13] == [0] * 6 + [7 * 16 + i for i in range(4)] + [0] * 3


def test_outputs_are_optional_and_other_stream(kvc):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    start = torch.full((2,), 9, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kvc.kvc_slot_map(ratio=1, page_size=4, num_pages=9, lens=i32([0, 2]), new_lens=i32([5, 1]),
                     page_table=table, free_pages=i32([3, 5, 7]), start_pos=start, max_tokens=6,
                     stream=s)
    s.synchronize()
    assert table.tolist() == [[3, 5, 0], [0, 0, 0]] and start.tolist() == [0, 2]
    kvc.kvc_slot_map(ratio=1, page_size=4, num_pages=9, lens=i32([]), new_lens=i32([]),
                     page_table=table, free_pages=i32([]), out_loc=(o := i32([4, 4])))
    torch.cuda.synchronize()
    assert o.tolist() == [0, 0]


def test_graph_replays_follow_the_lengths(kvc):
    S, ps, cap = 40, 16, 600
    rng = random.Random(5)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    lens, n, table, free, num = batch(S, 1, ps, (0, 200), (0, 14), rng, width=30)
    free = np.arange(1, 400, dtype=np.int32)
    L, N, T, F = i32(lens), i32(n), dev(table), dev(free)
    e = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")
    o = dict(offsets=e(2, S), start_pos=e(S), out_loc=e(cap), positions=e(cap), token_to_req=e(cap),
             totals=e(4))
    call = lambda: kvc.kvc_slot_map(ratio=1, page_size=ps, num_pages=500, lens=L, new_lens=N,
                                    page_table=T, free_pages=F, **o)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for k in range(4):
        lens, n, table, _, _ = batch(S, 1, ps, (-1, 200), (0, 14), rng, width=30)
        L.copy_(i32(lens)), N.copy_(i32(n)), T.copy_(dev(table))
        g.replay()
        torch.cuda.synchronize()
        want, _ = ref.slot_map(ratio=1, page_size=ps, num_pages=500, lens=lens, new_lens=n,
                               page_table=table, free_pages=free, max_tokens=cap)
        for key, t in {**o, "page_table": T}.items():
            np.testing.assert_array_equal(host(t), want[key], err_msg=f"replay {k}: {key}")


@pytest.mark.parametrize("layout", ["V41", "V41_FP4", "V4"])
def test_a_serving_run(kvc, layout):
    """Requests of different lengths as a server takes them: prompts in one
    packed step, then a drafted tree, every table from kvc_slot_map, rows through
    the rotary store, attention over what was stored."""
    H, ps, D, S = 16, 16, 6, 3
    rng = random.Random(3)
    num_pages, width = 60, 12
    freqs = torch.from_numpy(np.ascontiguousarray(W.rope_freqs(400))).cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    e = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")
    rb = kvc.kvc_layout_query(layout).row_bytes
    cache = kvc.Cache(torch.randint(0, 256, (num_pages, ps * rb), dtype=torch.uint8).cuda(), layout, ps)
    free = list(range(1, num_pages))
    rng.shuffle(free)
    table = torch.zeros(S, width, dtype=torch.int32, device="cuda")
    lens, rows_of = [0, 0, 0], [[], [], []]
    steps = [("prefill", [33, 1, 80], None), ("tree", [D] * S, [random_tree(D, rng) for _ in range(S)]),
             ("prefill", [5, 20, 0], None)]
    for kind, new, trees in steps:
        masks = None
        T = sum(new)
        stride = D if kind == "tree" else 0
        depth = None
        if trees:
            masks, depths = zip(*trees)
            depth = i32([d for row in depths for d in row])
        off, start, loc, pos, req, tot = e(2, S), e(S), e(T), e(T), e(T), e(4)
        kvc.kvc_slot_map(ratio=1, page_size=ps, num_pages=num_pages, lens=i32(lens),
                         new_lens=i32(new), page_table=table, free_pages=i32(free), offsets=off,
                         start_pos=start, out_loc=loc, positions=pos, token_to_req=req, totals=tot,
                         token_stride=stride, depth=depth)
        g = torch.Generator().manual_seed(len(free))
        rows = torch.randn(T, 512, generator=g).bfloat16()
        q = torch.randn(T, H, 512, generator=g).bfloat16()
        kvc.kvc_store_rows_rope(cache, rows.cuda(), pos, freqs, loc)
        out, lse = torch.empty(T, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, device="cuda")
        if kind == "tree":
            kvc.kvc_attend_tree(cache, q.cuda(), start, table, out, scale=0.05, draft_len=D,
                                tree=torch.tensor(masks, dtype=torch.int64).cuda(), lse=lse)
        else:
            kvc.kvc_attend_prefill(cache, q.cuda(), off, start, table, out, scale=0.05, lse=lse)
        torch.cuda.synchronize()
        free = free[int(tot[2]):]
        hc, ht = host(cache.data), host(table)
        t = 0
        for b, n in enumerate(new):
            # the stored rows are the rotated bf16 rows, quantized
            at = rows[t:t + n].view(torch.int16).numpy().view(np.uint16)
            hp = host(pos)[t:t + n]
            one = np.zeros((1, (n + 1) * rb + 16), np.uint8)
            rot, _ = oracle.store_rows_rope(np.zeros((n + 1, -(-rb // 16) * 16), np.uint8), layout, 1, at, hp,
                                            freqs.cpu().numpy(), np.arange(1, n + 1, dtype=np.int32))
            for i in range(n):
                rows_of[b].append(oracle.dequant_row(layout, *oracle.store_row(layout, rot[i:i + 1])))
            count = lens[b] + n
            x, valid = ref.cached_rows(hc, layout, ps, ht[b], count)
            assert valid.all()
            mine = np.concatenate(rows_of[b]).reshape(count, 512) if count else np.zeros((0, 512), np.uint16)
            f = torch.from_numpy((mine.astype(np.uint32) << 16).view(np.float32).astype(np.float64))
            assert torch.equal(x, f), f"{kind}: rows of slot {b}"
            if n:
                if kind == "tree":
                    r = torch.arange(count)[None] - lens[b]
                    m = torch.tensor([[(v >> i) & 1 for i in range(D)] for v in masks[b]], dtype=torch.bool)
                    seen = (r < 0) | (m[:, r[0].clamp(0, D - 1)] & (r >= 0))
                else:
                    seen = torch.arange(count)[None] < (lens[b] + torch.arange(n) + 1)[:, None]
                ref.check(out[t:t + n], lse[t:t + n], ref.attend(q[t:t + n].double(), x, seen, 0.05),
                          f"{kind} slot {b}")
            t += n
        if kind == "tree":
            # the first two tokens of every tree's first path are accepted: row
            # start and the row of the token below it, moved up by storing it again
            for b in range(S):
                rows_of[b] = rows_of[b][:lens[b] + 1]
                lens[b] += 1
            # pages the dropped drafts had taken beyond the kept rows go back
            for b in range(S):
                keep = -(-lens[b] // ps)
                held = -(-(lens[b] - 1 + D) // ps)
                free = [int(v) for v in ht[b, keep:held]] + free
        else:
            lens = [l + n for l, n in zip(lens, new)]


def random_tree(D, rng):
    """(ancestor masks, depths) of D drafted tokens."""
    m, d = [], []
    for j in range(D):
        parent = rng.randint(max(-1, j - 3), j - 1) if j else -1
        m.append((m[parent] if parent >= 0 else 0) | 1 << j)
        d.append(d[parent] + 1 if parent >= 0 else 0)
    return m, d
