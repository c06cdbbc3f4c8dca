"""What the slot map and the attention refuse, on the host: C-ABI argument
checks (fake pointers, nothing is launched) and the binding's size checks."""
import ctypes as C
import inspect

import pytest
import torch

FAKE = 0x7F0000000000   # never dereferenced: every call below returns before a launch


@pytest.fixture(scope="module")
def kvc():
    import fp8_fp4_quantized_amd as k
    return k


def slot_map(kvc, **kw):
    a = kvc.kvc_slot_map_args()
    base = dict(ratio=1, page_size=64, num_pages=10, num_slots=4, token_stride=0, lens=FAKE,
                new_lens=FAKE + 64, depth=None, page_table=FAKE, pt_stride=8, pt_width=8,
                free_pages=FAKE, n_free=5, max_tokens=100, offsets=FAKE, start_pos=FAKE + 128,
                out_loc=FAKE, positions=FAKE, token_to_req=FAKE, totals=FAKE, status=None)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return kvc.lib().kvc_slot_map(C.byref(a), None)


def test_slot_map_arguments(kvc):
    big = (1 << 31) - 1
    for kw in (dict(page_size=0), dict(page_size=48), dict(page_size=8192), dict(num_pages=0),
               dict(num_pages=1 << 26), dict(num_slots=-1), dict(num_slots=8192),
               dict(max_tokens=-1), dict(max_tokens=big), dict(n_free=-1), dict(n_free=big),
               dict(token_stride=-1), dict(token_stride=26), dict(lens=None), dict(new_lens=None),
               dict(start_pos=FAKE), dict(start_pos=FAKE + 64), dict(page_table=None),
               dict(pt_width=0), dict(pt_width=9), dict(free_pages=None)):
        assert slot_map(kvc, **kw) == kvc.KVC_EINVAL, kw
        assert "kvc_slot_map" in kvc.kvc_last_error()
    for kw in (dict(ratio=0), dict(ratio=3), dict(ratio=2, depth=FAKE)):
        assert slot_map(kvc, **kw) == kvc.KVC_EUNSUPPORTED, kw
    assert kvc.lib().kvc_slot_map(None, None) == kvc.KVC_EINVAL


def attend(kvc, call="kvc_attend_tree", **kw):
    a = kvc.kvc_attend_args()
    rb = 528
    base = dict(ratio=1, num_heads=16, num_slots=3, draft_len=4, q=FAKE, q_stride=16 * 512,
                q_head_stride=512, q_rows=12, offsets=FAKE, start_pos=FAKE, page_table=FAKE,
                pt_stride=8, pt_width=8, tree=None, scale=0.05, sink=None, out=FAKE,
                out_stride=16 * 512, out_head_stride=512, lse=None,
                cache=kvc.kvc_cache(FAKE, 1, 64, 64 * rb, 10), workspace=FAKE,
                workspace_bytes=1 << 40, status=None)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return getattr(kvc.lib(), call)(C.byref(a), None)


def test_attention_arguments(kvc):
    need = kvc.kvc_attend_workspace(3, 12, 16)
    shared = [dict(num_heads=0), dict(num_heads=1025), dict(num_slots=-1), dict(num_slots=8192),
              dict(q_rows=-1), dict(q_rows=1 << 28), dict(q=None), dict(q=FAKE + 8), dict(out=None),
              dict(out=FAKE + 8), dict(q_stride=-8), dict(q_stride=4), dict(q_head_stride=12),
              dict(out_stride=504), dict(out_stride=8196), dict(out_head_stride=256),
              dict(start_pos=None), dict(page_table=None), dict(pt_width=0), dict(pt_width=9),
              dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
              dict(workspace=None), dict(workspace=FAKE + 16), dict(workspace_bytes=need - 1),
              dict(cache=kvc.kvc_cache(FAKE, 1, 48, 64 * 528, 10)),
              dict(cache=kvc.kvc_cache(None, 1, 64, 64 * 528, 10))]
    for call in ("kvc_attend_tree", "kvc_attend_prefill"):
        for kw in shared:
            assert attend(kvc, call, **kw) == kvc.KVC_EINVAL, (call, kw)
            assert call in kvc.kvc_last_error()
        assert attend(kvc, call, ratio=3) == kvc.KVC_EUNSUPPORTED
        assert attend(kvc, call, cache=kvc.kvc_cache(FAKE, 9, 64, 64 * 528, 10)) == \
            kvc.KVC_EUNSUPPORTED
        assert getattr(kvc.lib(), call)(None, None) == kvc.KVC_EINVAL
        # nothing to do: answered on the host
        assert attend(kvc, call, num_slots=0) == kvc.KVC_OK
    for kw in (dict(draft_len=0), dict(draft_len=65), dict(q_rows=11)):
        assert attend(kvc, **kw) == kvc.KVC_EINVAL, kw
    assert attend(kvc, ratio=2, tree=FAKE) == kvc.KVC_EUNSUPPORTED
    assert attend(kvc, "kvc_attend_prefill", offsets=None) == kvc.KVC_EINVAL
    assert attend(kvc, "kvc_attend_prefill", q_rows=0) == kvc.KVC_OK


def test_workspace_sizes(kvc):
    f = kvc.kvc_attend_workspace
    # per part of a query: 512 fp32 sums and 16 bytes of statistics, two parts a workgroup
    for slots, tokens, heads, queries in ((1, 1, 32, 32), (1, 2, 32, 64), (4, 4, 65, 128),
                                          (0, 0, 1, 32), (1, 100000, 128, 128)):
        assert 0 <= f(slots, tokens, heads) - 2 * 256 * queries * (2048 + 16) < 30000
        assert f(slots, tokens, heads) % 256 == 0
    for args in ((-1, 1, 1), (8192, 1, 1), (1, -1, 1), (1, 1, 0), (1, 1, 1025), (1, 1 << 30, 2)):
        with pytest.raises(kvc.KvcError):
            f(*args)
    assert kvc.lib().kvc_attend_workspace(1, 1, 1, None) == kvc.KVC_EINVAL


def test_binding_refuses_host_tensors_and_short_ones(kvc):
    """The binding's own checks, on CPU tensors: they come before any launch."""
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    cache = kvc.Cache(torch.zeros(2, 64 * 528, dtype=torch.uint8), "V41", 64)
    ok = dict(lens=i(4), new_lens=i(4), page_table=i(4, 3), free_pages=i(2), ratio=1, page_size=64,
              num_pages=2, out_loc=i(9))
    for kw in (dict(new_lens=i(3)), dict(page_table=i(3, 3)), dict(offsets=i(2, 3)),
               dict(start_pos=i(3)), dict(totals=i(3)), dict(max_tokens=10), dict()):
        with pytest.raises(ValueError):
            kvc.kvc_slot_map(**{**ok, **kw})
    for q, out in ((bf(4, 16, 512), bf(4, 16, 512)), (bf(4, 512), bf(4, 512))):
        with pytest.raises(ValueError):
            kvc.kvc_attend_tree(cache, q, i(4), i(4, 3), out, scale=0.1)
        with pytest.raises(ValueError):
            kvc.kvc_attend_prefill(cache, q, i(2, 4), i(4), i(4, 3), out, scale=0.1)
    for fn in (kvc.kvc_slot_map, kvc.kvc_attend_tree, kvc.kvc_attend_prefill):
        assert "stream" in inspect.signature(fn).parameters and fn.__doc__
