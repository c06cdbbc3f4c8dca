"""Sinks at the ends of their range: infinite ones, and ones whose base-2 form
passes fp32."""
import math

import pytest
import torch

from tests import attend_ref as ref
from tests.gpu_util import dev
from tests.test_gpu_attend import SCALE, Filled, prefill_seen, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    import fp8_fp4_quantized_amd as k
    return k


@pytest.mark.parametrize("H", [8, 32, 128])              # units of 32, 64 and 128 queries
@pytest.mark.parametrize("start", [0, 40, 6000])         # no row to see, whole units, joined ones
def test_sinks_without_a_finite_power(kvc, H, start):
    D = 2
    f = Filled(kvc, "V41", 64, [(start + D) // 2], H + start)
    q = queries(D, H, H)
    sink = torch.randn(H)
    sink[0], sink[1], sink[2], sink[3] = math.inf, 3e38, -math.inf, -3e38
    out = torch.full((D, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((D, H), 7.0, device="cuda")
    kvc.kvc_attend_tree(f.cache, q.cuda(), torch.tensor([start], dtype=torch.int32).cuda(),
                        dev(f.table), out, scale=SCALE, draft_len=D, ratio=2, sink=sink.cuda(), lse=lse)
    out, lse = out.cpu(), lse.cpu()
    # e^sink outweighs everything: out = 0, lse = sink log2(e), past fp32
    assert (out[:, :2].float() == 0).all() and (lse[:, :2] == math.inf).all()
    rows, _ = f.rows(0, (start + D) // 2)
    # e^sink is 0 (but for a query that sees nothing: its lse is the sink)
    none = ref.attend(q[:, 2:4].double(), rows, prefill_seen(start, D, 2, rows.shape[0]), SCALE)
    if start == 0:
        none[1][0] = -math.inf
    ref.check(out[:, 2:4], lse[:, 2:4], none, "negative")
    rest = ref.attend(q[:, 4:].double(), rows, prefill_seen(start, D, 2, rows.shape[0]), SCALE, sink[4:])
    ref.check(out[:, 4:], lse[:, 4:], rest, "finite")
