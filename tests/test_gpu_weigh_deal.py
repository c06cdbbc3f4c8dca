"""Attention weights of many queries where the deal of the work takes its rarer ways: a
slot of more than 1,024 segments, a batch with more parts than there are places for, and
sums of segments that differ by 2^24."""
import math

import pytest
import torch

from tests import evict_ref as ref
from tests.gpu_util import dev
from tests.test_gpu_attend import Filled, SCALE, kvc, prefill_seen, queries  # noqa: F401
from tests.test_gpu_weigh import check, natural_lse

pytestmark = pytest.mark.gpu
T, H = 2500, 1024                # segments of two tokens: 1,250 of them


def prompt(kvc, f, q, lse):  # noqa: F811
    """One prompt of T tokens whose queries are the same for every token."""
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    out = torch.full((1, T + 5), 9.0, device="cuda")
    kvc.kvc_weigh_prefill(f.cache, q.cuda().expand(T, H, 512), lse.cuda(), i(0, T).view(2, 1), i(0), dev(f.table),
                          out, scale=SCALE)
    assert (out[0, T:] == 9).all()
    return out.cpu()[0, :T].double()


def test_more_than_1024_segments(kvc):  # noqa: F811
    """lse is the attention's and some, another amount for every token and head, so that a
    token counted twice, or for a row that it does not see, shows."""
    f = Filled(kvc, "V41", 64, [T], seed=3)
    q = queries(1, H, seed=4, scale=1.3)
    rows, valid = f.rows(0, T)
    assert valid.all()
    s = (q[0].double() @ rows.T) * (SCALE * ref.LOG2E)                 # [H, T]
    e = torch.exp2(s)
    g = torch.Generator().manual_seed(5)
    lse = (torch.log2(e.cumsum(1)).T + 3 * torch.randn(T, H, generator=g).double()).float().contiguous()
    later = lambda v: v.T.flip(1).cumsum(1).flip(1)                    # [H, T]: tokens that see the row
    w = torch.exp2(-lse.double())
    one, far = later(w), later(w * lse.double().abs())
    want = (e * one).sum(0)
    # a weight: as evict_ref.weigh has it; its sum: in a chunk 16 additions, of 8 chunks 8, and
    # those whose errors are carried, of a wave's halves, of groups and of segments: 2 each
    d2 = 516 * SCALE * ref.LOG2E * (q[0].double().abs() @ rows.abs().T) + 3 * s.abs()
    tol = ref.U_FP32 * ((e * one * (math.log(2) * d2 * 1.01 + 4)).sum(0) + (e * far).sum(0) * 3.03 * math.log(2) + 40 * want)
    got = prompt(kvc, f, q, lse)
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), bad.nonzero()[:5].tolist()


def test_small_sums_of_segments_behind_a_large_one(kvc):  # noqa: F811
    """Queries of zeros weigh 2^-lse: 2^13 each in the first segment (2^24 in all), 1
    for one query of each later one; others give nothing."""
    f = Filled(kvc, "V41_FP4", 64, [T], seed=3)
    lse = torch.full((T, H), math.inf)
    lse[:2] = -13
    lse[2::2, 7] = 0
    got = prompt(kvc, f, torch.zeros(1, H, 512, dtype=torch.bfloat16), lse)
    want = torch.exp2(-lse.double()).sum(1).flip(0).cumsum(0).flip(0)
    # (whole numbers; the carried sums of segments, 2 additions of groups, the last rounding,
    # and an exponential's 2)
    assert ((got - want).abs() <= 8 * ref.U_FP32 * want).all(), (got - want).abs().max()


def test_more_parts_than_places(kvc):  # noqa: F811
    """5,600 prompts of 257 tokens with 6 heads, all of the same tokens and rows, would have
    16,800 parts of two segments; a longer one among them is cut all the same."""
    S, n, H = 5600, 257, 6
    f = Filled(kvc, "V41", 64, [n, 1000], seed=6)
    q = queries(700, H, seed=7, scale=1.2)
    rows, valid = f.rows(0, n)
    lse = torch.zeros(700, H)
    lse[:n] = natural_lse(q[:n], rows, prefill_seen(0, n, 1, n))
    long, lvalid = f.rows(1, 1000)
    seen = prefill_seen(300, 700, 1, 1000)
    lse[n:] = natural_lse(q[n:], long, seen[n:])
    counts = torch.full((S + 1,), n, dtype=torch.int32)
    starts = torch.zeros(S + 1, dtype=torch.int32)
    table = torch.from_numpy(f.table)[:1].repeat(S + 1, 1)
    at = 4321
    counts[at], starts[at], table[at] = 700, 300, torch.from_numpy(f.table)[1]
    out = torch.full((S + 1, 1010), 9.0, device="cuda")
    kvc.kvc_weigh_prefill(f.cache, q.cuda(), lse.cuda(), torch.stack([torch.zeros_like(counts), counts]).cuda(),
                          starts.cuda(), table.cuda(), out, scale=SCALE)
    got = out.cpu()
    check(got[at], torch.zeros(1010), *ref.weigh(q.double(), lse, long, lvalid, seen, SCALE), 0.0, 0)
    total, tol = ref.weigh(q[:n].double(), lse[:n], rows, valid, prefill_seen(0, n, 1, n), SCALE)
    short = torch.arange(S + 1) != at
    assert ((got[short, :n].double() - total).abs() <= tol).all()
    assert (got[short, n:] == 9).all() and (got[at, 1000:] == 9).all()
