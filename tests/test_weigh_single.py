"""Attention weights of one slot: a row alone has no stride.  C-ABI checks with fake
pointers; every call is refused before a launch."""
import pytest

from tests.test_evict_args import FAKE, kvc, weigh  # noqa: F401


@pytest.mark.parametrize("call", ["kvc_weigh_tree", "kvc_weigh_prefill"])
@pytest.mark.parametrize("slots,message", [(1, "workspace"), (2, "another stride")])
def test_prev_is_weights_with_another_stride(kvc, call, slots, message):  # noqa: F811
    """Refused for several slots; with one, only for what comes after (no workspace)."""
    assert weigh(kvc, call, num_slots=slots, prev=FAKE + 128, prev_stride=200, workspace=None) == kvc.KVC_EINVAL
    assert message in kvc.kvc_last_error()
