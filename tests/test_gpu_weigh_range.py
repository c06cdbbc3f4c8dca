"""Attention weights of queries of any magnitude, and of V41_FP4 rows whose scale is NaN."""
import math

import pytest
import torch

from tests import evict_ref as ref
from tests.gpu_util import dev
from tests.test_gpu_attend import Filled, SCALE, kvc, prefill_seen, queries  # noqa: F401
from tests.test_gpu_weigh import check, natural_lse

pytestmark = pytest.mark.gpu


# (two tokens stay in LDS with 16 heads, not with 80)
@pytest.mark.parametrize("H", [16, 80])
@pytest.mark.parametrize("layout", ["V4", "V41", "V41_FP4"])
@pytest.mark.parametrize("power", [117, 60, -60])
def test_queries_of_any_magnitude(kvc, layout, H, power):  # noqa: F811
    """Times a power of two that the scale takes back: the same scores.  Every other
    head's are 2^-20 of the others', some of a query's dims 2^-25 of its greatest."""
    D, start = 2, 150
    f = Filled(kvc, layout, 64, [start + D], seed=H)
    q = queries(D, H, seed=5, scale=1.3).double()
    q[:, 1::2] *= 2.0 ** -20
    q[:, :, ::5] *= 2.0 ** -25
    rows, valid = f.rows(0, start + D)
    seen = prefill_seen(start, D, 1, start + D)
    lse = natural_lse(q, rows, seen)
    total, tol = ref.weigh(q, lse, rows, valid, seen, SCALE)
    out = torch.full((1, start + D), 9.0, device="cuda")
    big = (q * 2.0 ** power).bfloat16()
    assert torch.equal(big.double() * 2.0 ** -power, q)
    kvc.kvc_weigh_tree(f.cache, big.cuda(), lse.cuda(), torch.tensor([start], dtype=torch.int32, device="cuda"),
                       dev(f.table), out, scale=SCALE * 2.0 ** -power, draft_len=D)
    check(out.cpu()[0], torch.zeros(start + D), total, tol, 0.0, 0)


@pytest.mark.parametrize("H,D", [(16, 3), (64, 5)])
def test_fp4_rows_with_a_nan_scale(kvc, H, D):  # noqa: F811
    """They collect nothing, and nobody else is the worse for them."""
    start = 300
    f = Filled(kvc, "V41_FP4", 64, [start + D], seed=9)
    bad = [5, 64, 299, 301]
    for k, r in enumerate(bad):
        page, at = int(f.table[0, r // 64]), r % 64
        f.host[page, 64 * 256 + at * 32 + 9 * k] = 0x7F if k % 2 else 0xFF
    cache = kvc.Cache(dev(f.host), "V41_FP4", 64)
    q = queries(D, H, seed=1)
    rows, valid = f.rows(0, start + D)
    assert torch.isfinite(rows).all(1).logical_not().nonzero().flatten().tolist() == bad
    seen = prefill_seen(start, D, 1, start + D)
    lse = natural_lse(q, torch.where(torch.isfinite(rows).all(1)[:, None], rows, 0.0), seen)
    total, tol = ref.weigh(q.double(), lse, rows, valid, seen, SCALE)
    out = torch.full((1, start + D), 9.0, device="cuda")
    kvc.kvc_weigh_tree(cache, q.cuda(), lse.cuda(), torch.tensor([start], dtype=torch.int32, device="cuda"),
                       dev(f.table), out, scale=SCALE, draft_len=D)
    check(out.cpu()[0], torch.zeros(start + D), total, tol, 0.0, 0)
    assert (out.cpu()[0, bad] == 0).all() and not math.isnan(out.sum().item())
