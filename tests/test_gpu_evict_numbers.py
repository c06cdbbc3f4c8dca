"""Numbers of rows past 32 bits: as many as there can be, none of them wrapped."""
import numpy as np
import pytest
import torch

from tests import evict_ref as ref
from tests.gpu_util import host
from tests.test_gpu_attend import kvc  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("far", [2 ** 31, 2 ** 32, 2 ** 32 + 3, 2 ** 40 + 1, 2 ** 63])
@pytest.mark.parametrize("which", ["budget", "first", "recent"])
def test_numbers_of_rows(kvc, far, which):  # noqa: F811
    lens, K = [50, 9], 12
    w = torch.rand(2, 60, generator=torch.Generator().manual_seed(2))
    kept, counts = (torch.zeros(*s, dtype=torch.int32, device="cuda") for s in ((2, K), (2,)))
    kw = {**dict(budget=10, first=2, recent=3), which: far}
    kvc.kvc_evict_select(torch.tensor(lens, dtype=torch.int32, device="cuda"), w.cuda(), kept, counts, **kw)
    want = ref.select(np.array(lens), w.numpy(), [min(kw["budget"], K)] * 2, K, 1, kw["first"], kw["recent"])
    assert np.array_equal(host(kept), want[0]) and np.array_equal(host(counts), want[1])
    for name in ("first", "recent"):
        with pytest.raises(kvc.KvcError):
            kvc.kvc_evict_select(torch.tensor(lens, dtype=torch.int32, device="cuda"), w.cuda(), kept, counts,
                                 **{name: -far})
