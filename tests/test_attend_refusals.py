"""Arguments that the attention and the slot map refuse beside those of
test_attend_args.py: on the host, nothing is launched."""
import math

import pytest
import torch

from tests.test_attend_args import attend


@pytest.fixture(scope="module")
def kvc():
    import fp8_fp4_quantized_amd as k
    return k


@pytest.mark.parametrize("call", ["kvc_attend_tree", "kvc_attend_prefill"])
def test_scale_whose_base_2_form_passes_fp32(kvc, call):
    """Scores are taken to the power of 2, by scale * log2(e): with that
    infinite every row at a right angle to its query would be 0 * inf."""
    top = float(torch.finfo(torch.float32).max)
    for scale in (top, 2.5e38, top / math.log2(math.e) * 1.0001):
        assert attend(kvc, call, scale=scale) == kvc.KVC_EINVAL, scale
        assert "scale" in kvc.kvc_last_error()
