"""Workspace sizes of the attention: one sized for the largest batch serves
every smaller one, in slots, tokens or heads."""
import itertools

import pytest
import torch


@pytest.fixture(scope="module")
def kvc():
    import fp8_fp4_quantized_amd as k
    return k


SLOTS, TOKENS, HEADS = (0, 1, 2, 8, 63, 256, 8191), (0, 1, 2, 7, 64, 512, 70000), (1, 5, 16, 64, 128, 1024)


def test_sizes_do_not_shrink_as_a_batch_grows(kvc):
    size = {c: kvc.kvc_attend_workspace(*c) for c in itertools.product(SLOTS, TOKENS, HEADS)}
    # steps along each axis, whose maxima give every larger batch
    for s, t, h in size:
        for more in ((s2, t2, h2) for s2 in SLOTS for t2 in TOKENS for h2 in HEADS
                     if s2 >= s and t2 >= t and h2 >= h):
            assert size[more] >= size[s, t, h], ((s, t, h), more)


def test_fewer_slots_for_the_same_tokens(kvc):
    f = kvc.kvc_attend_workspace
    assert f(256, 512, 16) >= f(8, 512, 16) == f(1, 512, 16)


@pytest.mark.gpu
def test_one_workspace_for_a_batch_as_it_shrinks(kvc):
    """Slots leave a batch whose buffers are sized for all of them."""
    from tests import attend_ref as ref
    from tests.gpu_util import dev
    from tests.test_gpu_attend import SCALE, Filled, prefill_seen, queries

    S, T, H = 64, 128, 16
    f = Filled(kvc, "V41", 64, [130] * S, 3)
    q = queries(T, H, 3)
    qd, table = q.cuda(), dev(f.table)
    space = torch.empty(kvc.kvc_attend_workspace(S, T, H), dtype=torch.uint8, device="cuda")
    for slots in (64, 16, 4, 1):
        n = T // slots                              # tokens of each: units of 32 up to 128
        starts = [max(0, 130 - n)] * slots
        off = torch.tensor([[n * b for b in range(slots)], [n] * slots], dtype=torch.int32).cuda()
        out = torch.full((T, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((T, H), 7.0, device="cuda")
        kvc.kvc_attend_prefill(f.cache, qd, off, torch.tensor(starts, dtype=torch.int32).cuda(), table, out,
                               scale=SCALE, lse=lse, workspace=space)
        out, lse = out.cpu(), lse.cpu()
        for b in range(0, slots, 3):
            rows, _ = f.rows(b, starts[b] + n)
            t = slice(n * b, n * b + n)
            ref.check(out[t], lse[t], ref.attend(q[t].double(), rows,
                                                 prefill_seen(starts[b], n, 1, starts[b] + n), SCALE),
                      f"{slots} slots, slot {b}")
