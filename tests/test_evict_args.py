"""What the rotary calls and the eviction refuse, on the host: C-ABI argument
checks (fake pointers, nothing is launched) and the binding's size checks."""
import ctypes as C
import math

import pytest
import torch

FAKE = 0x7F0000000000   # never dereferenced: every call below returns before a launch


@pytest.fixture(scope="module")
def kvc():
    import fp8_fp4_quantized_amd as k
    return k


def fill(a, base, kw):
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


def refused(kvc, call, code, cases):
    for kw in cases:
        assert call(kvc, **kw) == code, kw
        assert "kvc_" in kvc.kvc_last_error()


def cache(kvc, **kw):
    return fill(kvc.kvc_cache(), dict(base=FAKE, layout=1, page_size=64, page_stride=64 * 528, num_pages=9), kw)


# -------------------------------------------------------------------- rotary
def rope_table(kvc, **kw):
    a = fill(kvc.kvc_rope_table_args(), dict(freqs=FAKE, n=10, first=0, rot_dim=64, scaling=0, base=1e4,
                                            factor=1.0, original=4096, beta_fast=32, beta_slow=1, mscale=1), kw)
    return kvc.lib().kvc_rope_table(C.byref(a), None)


def test_rope_table_arguments(kvc):
    refused(kvc, rope_table, kvc.KVC_EINVAL, [
        dict(freqs=None), dict(freqs=FAKE + 8), dict(n=-1), dict(first=-1), dict(first=2 ** 31 - 9),
        dict(n=2 ** 31 + 1), dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=514), dict(rot_dim=-2),
        dict(scaling=2, rot_dim=2), dict(base=1.0), dict(base=-5), dict(base=math.inf), dict(base=math.nan),
        dict(scaling=1, factor=0.0), dict(scaling=1, factor=-1), dict(scaling=2, factor=math.nan),
        dict(scaling=3, original=0), dict(scaling=3, beta_fast=0.5), dict(scaling=3, beta_slow=0),
        dict(scaling=3, beta_fast=math.inf), dict(scaling=3, beta_fast=math.nan), dict(mscale=0),
        dict(mscale=math.inf), dict(scaling=1, factor=1e-320),          # speeds that are not finite
    ])
    refused(kvc, rope_table, kvc.KVC_EUNSUPPORTED, [dict(scaling=4), dict(scaling=-1)])
    assert kvc.lib().kvc_rope_table(None, None) == kvc.KVC_EINVAL
    assert rope_table(kvc, n=0, freqs=None) == kvc.KVC_OK               # nothing to write


def rope_rows(kvc, **kw):
    a = fill(kvc.kvc_rope_args(), dict(dtype=0, num_heads=4, head_dim=128, rot_dim=64, offset=64, half=0,
                                       transpose=0, tokens=3, x=FAKE, x_stride=512, x_head_stride=128,
                                       out=FAKE + 65536, out_stride=512, out_head_stride=128, positions=FAKE,
                                       freqs=FAKE, max_pos=100, status=None), kw)
    return kvc.lib().kvc_rope_rows(C.byref(a), None)


def test_rope_rows_arguments(kvc):
    refused(kvc, rope_rows, kvc.KVC_EINVAL, [
        dict(num_heads=0), dict(num_heads=1025), dict(head_dim=1), dict(head_dim=8193), dict(rot_dim=0),
        dict(rot_dim=63), dict(rot_dim=130), dict(offset=-1), dict(offset=65), dict(tokens=-1),
        dict(tokens=2 ** 31), dict(max_pos=0), dict(x=None), dict(out=None), dict(x=FAKE + 1),
        dict(dtype=2, out=FAKE + 2), dict(x_stride=-1), dict(x_head_stride=-8), dict(out_stride=127),
        dict(out_head_stride=127), dict(out=FAKE, out_stride=1024), dict(out=FAKE, out_head_stride=256),
        dict(positions=None), dict(freqs=None), dict(freqs=FAKE + 4)])
    refused(kvc, rope_rows, kvc.KVC_EUNSUPPORTED, [dict(dtype=3), dict(dtype=-1)])
    assert kvc.lib().kvc_rope_rows(None, None) == kvc.KVC_EINVAL
    assert rope_rows(kvc, tokens=0, x=None) == kvc.KVC_OK


# ------------------------------------------------------------------- weights
def weigh(kvc, call="kvc_weigh_tree", **kw):
    more = {k[6:]: kw.pop(k) for k in list(kw) if k.startswith("cache_")}
    a = fill(kvc.kvc_weigh_args(), dict(ratio=1, num_heads=64, num_slots=3, draft_len=4, q=FAKE,
                                        q_stride=64 * 512, q_head_stride=512, q_rows=12, lse=FAKE + 64,
                                        offsets=FAKE, start_pos=FAKE, page_table=FAKE, pt_stride=8, pt_width=8,
                                        tree=None, scale=0.05, decay=1.0, prev=None, prev_stride=0,
                                        weights=FAKE + 128, w_stride=100, w_width=100, workspace=FAKE,
                                        workspace_bytes=1 << 40, status=None), kw)
    a.cache = cache(kvc, **more)
    return getattr(kvc.lib(), call)(C.byref(a), None)


@pytest.mark.parametrize("call", ["kvc_weigh_tree", "kvc_weigh_prefill"])
def test_weigh_arguments(kvc, call):
    n = kvc.kvc_weigh_workspace()
    top = float(torch.finfo(torch.float32).max)
    cases = [dict(num_heads=0), dict(num_heads=1025), dict(num_slots=-1), dict(num_slots=8192), dict(q_rows=-1),
             dict(q_rows=(2 ** 31 - 256) // 64 + 1), dict(q=None), dict(q=FAKE + 8), dict(q_stride=-8),
             dict(q_stride=4), dict(q_head_stride=12), dict(q_stride=2 ** 31), dict(q_head_stride=2 ** 31),
             dict(lse=None), dict(start_pos=None), dict(page_table=None), dict(pt_width=0), dict(pt_width=9),
             dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=top), dict(decay=-0.5),
             dict(decay=math.nan), dict(decay=math.inf), dict(weights=None), dict(w_width=0),
             dict(w_width=101), dict(prev=FAKE, prev_stride=99), dict(prev=FAKE + 128, prev_stride=101),
             dict(weights=FAKE + 64), dict(workspace=None), dict(workspace=FAKE + 128),
             dict(workspace_bytes=n - 1), dict(cache_base=None), dict(cache_page_size=48),
             dict(cache_page_stride=64 * 528 + 8), dict(cache_num_pages=0)]
    if call == "kvc_weigh_tree":
        cases += [dict(draft_len=0), dict(draft_len=65), dict(q_rows=11)]
    else:
        cases += [dict(offsets=None)]
    refused(kvc, lambda k, **kw: weigh(k, call, **kw), kvc.KVC_EINVAL, cases)
    refused(kvc, lambda k, **kw: weigh(k, call, **kw), kvc.KVC_EUNSUPPORTED, [dict(ratio=0), dict(ratio=3),
                                                                              dict(cache_layout=3)])
    assert getattr(kvc.lib(), call)(None, None) == kvc.KVC_EINVAL
    assert weigh(kvc, call, num_slots=0) == kvc.KVC_OK
    assert weigh(kvc, "kvc_weigh_tree", ratio=2, tree=FAKE) == kvc.KVC_EUNSUPPORTED
    assert kvc.lib().kvc_weigh_workspace(None) == kvc.KVC_EINVAL


# -------------------------------------------------------------------- choice
def select(kvc, **kw):
    a = fill(kvc.kvc_evict_args(), dict(ratio=1, num_slots=4, lens=FAKE, weights=FAKE + 64, w_stride=100000,
                                        w_width=100000, budget=5, first=0, recent=0, budgets=None, kept=FAKE,
                                        kept_stride=10, kept_width=10, counts=FAKE + 256, kept_weights=None,
                                        kw_stride=0, workspace=FAKE, workspace_bytes=1 << 40, status=None), kw)
    return kvc.lib().kvc_evict_select(C.byref(a), None)


def test_select_arguments(kvc):
    need = C.c_int64(0)
    assert kvc.lib().kvc_evict_workspace(4, 100000, C.byref(need)) == kvc.KVC_OK and need.value > 0
    refused(kvc, select, kvc.KVC_EINVAL, [
        dict(num_slots=-1), dict(num_slots=8192), dict(first=-1), dict(recent=-1), dict(lens=None),
        dict(counts=None), dict(counts=FAKE), dict(weights=None), dict(w_width=0), dict(w_width=100001),
        dict(kept=None), dict(kept_width=0), dict(kept_width=11), dict(kept_width=2 ** 31, kept_stride=2 ** 31),
        dict(kept_weights=FAKE, kw_stride=9), dict(kept_weights=FAKE + 64, kw_stride=10), dict(workspace=None),
        dict(workspace=FAKE + 16), dict(workspace_bytes=need.value - 1)])
    refused(kvc, select, kvc.KVC_EUNSUPPORTED, [dict(ratio=0), dict(ratio=3)])
    assert kvc.lib().kvc_evict_select(None, None) == kvc.KVC_EINVAL
    assert select(kvc, num_slots=0) == kvc.KVC_OK


def test_evict_workspace_covers_smaller_calls(kvc):
    """What a call needs never passes the workspace of a larger one."""
    size = kvc.kvc_evict_workspace
    assert size(1, kvc.SELECT_NO_WORKSPACE) == 0 and size(8191, kvc.SELECT_NO_WORKSPACE) == 0
    assert size(1, kvc.SELECT_NO_WORKSPACE + 1) > 0
    widths = [1, 16384, 16385, 20000, 32768, 32769, 100000, 1 << 20, 1 << 23, 1 << 31, (1 << 63) - 1]
    slots = [0, 1, 2, 3, 60, 64, 127, 128, 129, 255, 256, 257, 8191]
    for i, s in enumerate(slots):
        for j, w in enumerate(widths):
            for s2 in slots[:i + 1]:
                for w2 in widths[:j + 1]:
                    assert size(s2, w2) <= size(s, w)
    for s, w in ((-1, 5), (8192, 5), (1, 0)):
        with pytest.raises(kvc.KvcError):
            size(s, w)
    assert kvc.lib().kvc_evict_workspace(1, 1, None) == kvc.KVC_EINVAL


# ---------------------------------------------------------------------- move
def compact(kvc, **kw):
    more = {k[6:]: kw.pop(k) for k in list(kw) if k.startswith("cache_")}
    a = fill(kvc.kvc_compact_args(), dict(ratio=1, num_slots=4, lens=FAKE, kept=FAKE, kept_stride=10,
                                          kept_width=10, counts=FAKE + 64, page_table=FAKE, pt_stride=8,
                                          pt_width=8, free_pages=FAKE + 128, n_free=5, new_table=FAKE + 512,
                                          nt_stride=8, new_lens=FAKE + 192, kept_weights=FAKE, kw_stride=10,
                                          weights=FAKE + 1024, w_stride=100, w_width=100, freed=FAKE + 2048,
                                          freed_cap=7, totals=FAKE, status=None), kw)
    a.cache = cache(kvc, **more)
    return kvc.lib().kvc_cache_compact(C.byref(a), None)


def test_compact_arguments(kvc):
    big = 2 ** 31 - 1
    refused(kvc, compact, kvc.KVC_EINVAL, [
        dict(num_slots=-1), dict(num_slots=8192), dict(n_free=-1), dict(n_free=big), dict(freed_cap=-1),
        dict(freed_cap=big), dict(lens=None), dict(counts=None), dict(new_lens=None), dict(new_lens=FAKE),
        dict(new_lens=FAKE + 64), dict(kept=None), dict(kept_width=0), dict(kept_width=11),
        dict(kept_width=big + 1, kept_stride=big + 1), dict(page_table=None), dict(pt_width=0),
        dict(pt_width=9), dict(new_table=None), dict(nt_stride=7), dict(new_table=FAKE), dict(free_pages=None),
        dict(freed=FAKE + 128), dict(kept_weights=None), dict(weights=None), dict(kw_stride=9),
        dict(w_width=0), dict(w_width=101), dict(weights=FAKE), dict(cache_base=None),
        dict(cache_page_size=3), dict(cache_num_pages=0)])
    refused(kvc, compact, kvc.KVC_EUNSUPPORTED, [dict(ratio=0), dict(ratio=3), dict(cache_layout=9)])
    assert kvc.lib().kvc_cache_compact(None, None) == kvc.KVC_EINVAL
    assert compact(kvc, num_slots=0, totals=None) == kvc.KVC_OK


# ------------------------------------------------------------------- binding
def test_binding_refuses_shapes_and_host_tensors(kvc):
    """Sizes are looked at before devices, so that host tensors show them."""
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    fl = lambda *s: torch.zeros(*s)
    c = kvc.Cache(torch.zeros(2, 64 * 528, dtype=torch.uint8), "V41", 64)
    for match, call in (
            ("^out", lambda: kvc.kvc_rope_table(fl(4))),
            ("^scaling", lambda: kvc.kvc_rope_table(fl(4, 64), scaling="yes")),
            ("^out", lambda: kvc.kvc_rope_table(fl(4, 64))),
            ("^x", lambda: kvc.kvc_rope_rows(bf(4, 2, 64), i(4), fl(9, 64))),
            ("^offsets", lambda: kvc.kvc_weigh_prefill(c, bf(4, 2, 512), fl(4, 2), i(3), i(1), i(1, 3), fl(1, 9),
                                                       scale=1.0)),
            ("^offsets", lambda: kvc.kvc_weigh_prefill(c, bf(4, 2, 512), fl(4, 2), i(4, 2), i(4), i(4, 3),
                                                       fl(4, 9), scale=1.0)),
            ("^q", lambda: kvc.kvc_weigh_tree(c, bf(4, 2, 512), fl(4, 2), i(3), i(3, 3), fl(3, 9), scale=1.0,
                                              draft_len=2)),
            ("^tree", lambda: kvc.kvc_weigh_tree(c, bf(4, 2, 512), fl(4, 2), i(2), i(2, 3), fl(2, 9), scale=1.0,
                                                 draft_len=2, tree=torch.zeros(3, dtype=torch.int64))),
            ("^tree", lambda: kvc.kvc_weigh_tree(c, bf(4, 2, 512), fl(4, 2), i(2), i(2, 3), fl(2, 9), scale=1.0,
                                                 draft_len=2, tree=torch.zeros(2, 64, dtype=torch.int64))),
            ("^q", lambda: kvc.kvc_weigh_tree(c, bf(4, 2, 512), fl(4, 2), i(2), i(2, 3), fl(2, 9), scale=1.0)),
            ("^lens", lambda: kvc.kvc_evict_select(i(2), fl(2, 9), i(2, 4), i(2))),
            ("^lens", lambda: kvc.kvc_cache_compact(c, i(2), i(2, 4), i(2), i(2, 3), i(5), i(2, 3), i(2)))):
        with pytest.raises(ValueError, match=match):
            call()
