"""Attention weights of one slot, accumulated in place in part of a wider row."""
import pytest
import torch

from tests.gpu_util import dev
from tests.test_gpu_attend import Filled, SCALE, kvc, queries  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,D", [(16, 1), (64, 4)])
def test_in_place_in_a_wider_row(kvc, H, D):  # noqa: F811
    f = Filled(kvc, "V41", 64, [120 + D], seed=2)
    q, lse = queries(D, H, seed=4).cuda(), torch.full((D, H), 8.0, device="cuda")
    st = torch.tensor([120], dtype=torch.int32, device="cuda")
    old = torch.rand(1, 200, generator=torch.Generator().manual_seed(1)).cuda()
    kw = dict(scale=SCALE, draft_len=D, decay=0.5)
    want = old.clone()
    kvc.kvc_weigh_tree(f.cache, q, lse, st, dev(f.table), want, prev=want, **kw)
    assert not torch.equal(want, old) and torch.equal(want[:, 120 + D:], old[:, 120 + D:])
    for width in (150, 120 + D):
        buf = old.clone()
        kvc.kvc_weigh_tree(f.cache, q, lse, st, dev(f.table), buf[:, :width], prev=buf, **kw)
        assert torch.equal(buf, want)
