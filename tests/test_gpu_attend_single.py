"""Queries and outputs of one head or one token, whose stride over that axis
says nothing: any is taken."""
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


@pytest.mark.parametrize("T,H", [(5, 1), (1, 5), (1, 1)])
def test_strides_of_a_single_head_or_token(kvc, T, H):
    start = 40
    f = Filled(kvc, "V41", 64, [start + T], 3)
    q = queries(T, H, 3)
    rows, _ = f.rows(0, start + T)
    want = ref.attend(q.double(), rows, prefill_seen(start, T, 1, start + T), SCALE)
    odd = (512 * H if T > 1 else 3, 512 if H > 1 else 1, 1)
    zero = (512 * H if T > 1 else 0, 512 if H > 1 else 0, 1)
    for qs in (odd, zero):
        for os in (odd, zero):
            qd = q.cuda().as_strided((T, H, 512), qs)
            out = torch.empty(T * H * 512, dtype=torch.bfloat16, device="cuda").as_strided((T, H, 512), os)
            lse = torch.empty(T, H, device="cuda")
            kvc.kvc_attend_tree(f.cache, qd, torch.tensor([start], dtype=torch.int32).cuda(), dev(f.table), out,
                                scale=SCALE, draft_len=T, lse=lse)
            ref.check(out, lse, want, f"{qs} {os}")
