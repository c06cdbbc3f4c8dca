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


def test_shapes_whose_rows_would_be_taken_apart(kvc):
    """Tensors that hold enough entries in rows of another length: read as they
    lie, every slot but the first would get a neighbour's."""
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    cache = kvc.Cache(torch.zeros(2, 64 * 528, dtype=torch.uint8), "V41", 64)
    q = bf(12, 16, 512)
    for shape in ((4, 64), (3, 4), (6, 2)):
        with pytest.raises(ValueError, match="^tree"):
            kvc.kvc_attend_tree(cache, q, i(4), i(4, 3), q.clone(), scale=0.1, draft_len=3,
                                tree=torch.zeros(*shape, dtype=torch.int64))
    for shape in ((4, 2), (1, 8)):
        with pytest.raises(ValueError, match="^offsets"):
            kvc.kvc_attend_prefill(cache, q, i(*shape), i(4), i(4, 3), q.clone(), scale=0.1)
    ok = dict(lens=i(4), new_lens=i(4), page_table=i(4, 3), free_pages=i(2), ratio=1, page_size=64,
              num_pages=2, out_loc=i(12))
    for shape in ((2, 8), (4, 2), (8, 4)):
        with pytest.raises(ValueError, match="^offsets"):
            kvc.kvc_slot_map(**ok, offsets=i(*shape))
    for shape in ((4, 64), (2, 6)):
        with pytest.raises(ValueError, match="^depth"):
            kvc.kvc_slot_map(**ok, token_stride=3, depth=i(*shape))
    # rows of the right length, and flat ones, go on to the device checks
    for more in (dict(offsets=i(2, 4)), dict(offsets=i(20)), dict(token_stride=3, depth=i(4, 3)),
                 dict(token_stride=3, depth=i(12))):
        with pytest.raises(ValueError, match="^lens"):
            kvc.kvc_slot_map(**ok, **more)
    for tree in (torch.zeros(4, 3, dtype=torch.int64), torch.zeros(5, 3, dtype=torch.int64),
                 torch.zeros(12, dtype=torch.int64)):
        with pytest.raises(ValueError, match="^q"):
            kvc.kvc_attend_tree(cache, q, i(4), i(4, 3), q.clone(), scale=0.1, draft_len=3, tree=tree)
