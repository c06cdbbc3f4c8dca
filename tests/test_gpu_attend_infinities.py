"""Rows that hold an infinity: a query that sees one is NaN, all of it and its
lse, and nobody else is, whatever tile, unit, piece or batch the row and the
query lie in. Scores that pass fp32 over finite rows are weights of 0."""
import numpy as np
import pytest
import torch

from tests import attend_ref as ref
from tests.gpu_util import dev
from tests.test_gpu_attend import SCALE, Filled, as_i64, prefill_seen, queries, tree_seen

pytestmark = pytest.mark.gpu

# a unit of 32, 64 and 128 queries: heads of a slot of four tokens
HEADS = (8, 16, 32)


@pytest.fixture(scope="module")
def kvc():
    import fp8_fp4_quantized_amd as k
    return k


def set_rope(f, kvc, row, dim, bits):
    """bf16 `bits` as rope dim `dim` of a V4 slot-0 row"""
    ps = f.page_size
    page, i = int(f.table[0, row // ps]), row % ps
    at = i * 576 + 448 + 2 * dim
    f.host[page, at:at + 2] = (bits & 0xFF, bits >> 8)
    f.cache = kvc.Cache(dev(f.host), f.layout, ps)


def expect(out, lse, q, rows, seen, what=""):
    """Queries that see a row that is not finite are NaN whole, the others as
    the reference has them."""
    out, lse = out.cpu(), lse.cpu()
    bad = ~torch.isfinite(rows).all(1)
    hit = (seen & bad[None]).any(1)
    assert torch.isnan(out[hit].float()).all() and torch.isnan(lse[hit]).all(), \
        f"{what}: a query that sees the row is not NaN"
    if hit.all():
        return hit
    clean = torch.where(bad[:, None], torch.zeros_like(rows), rows)
    ref.check(out[~hit], lse[~hit], ref.attend(q[~hit].double(), clean, seen[~hit], SCALE), what)
    return hit


def run_tree(kvc, f, q, start, masks, D, H):
    out = torch.full((D, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((D, H), 7.0, device="cuda")
    kvc.kvc_attend_tree(f.cache, q.cuda(), torch.tensor([start], dtype=torch.int32).cuda(),
                        dev(f.table), out, scale=SCALE, draft_len=D,
                        tree=None if masks is None else as_i64([masks]).cuda(), lse=lse)
    return out, lse


@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("sign", [0x7F80, 0xFF80])
def test_seen_by_some_tokens_of_a_tile(kvc, H, sign):
    """Scores of both signs at the row: heads whose score there is -inf would
    give it the weight 0."""
    D, start = 4, 33
    f = Filled(kvc, "V4", 64, [start + D], 5)
    set_rope(f, kvc, start + 1, 7, sign)
    masks = [0b0001, 0b0011, 0b0101, 0b1010]
    q = queries(D, H, 5)
    out, lse = run_tree(kvc, f, q, start, masks, D, H)
    rows, _ = f.rows(0, start + D)
    hit = expect(out, lse, q, rows, tree_seen(start, masks, start + D))
    assert hit.tolist() == [False, True, False, True]


@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("rows_before", [300, 9000])
def test_in_a_tile_that_all_see(kvc, H, rows_before):
    """Far from any mask; with 9,000 rows in a piece that is joined."""
    D = 4
    f = Filled(kvc, "V4", 64, [rows_before + D], 6)
    set_rope(f, kvc, 40, 3, 0x7F80)
    q = queries(D, H, 6)
    out, lse = run_tree(kvc, f, q, rows_before, None, D, H)
    rows, _ = f.rows(0, rows_before + D)
    assert expect(out, lse, q, rows, prefill_seen(rows_before, D, 1, rows_before + D)).all()


@pytest.mark.parametrize("H", (2, 32))
def test_in_a_prompt(kvc, H):
    """One row of a prompt: tokens before it are exact, all later ones NaN, in
    its own tile and in those behind it."""
    n, row = 200, 50
    f = Filled(kvc, "V4", 64, [n], 7)
    set_rope(f, kvc, row, 60, 0xFF80)
    q = queries(n, H, 7)
    out = torch.full((n, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, H), 7.0, device="cuda")
    kvc.kvc_attend_prefill(f.cache, q.cuda(), torch.tensor([[0], [n]], dtype=torch.int32).cuda(),
                           torch.zeros(1, dtype=torch.int32).cuda(), dev(f.table), out, scale=SCALE,
                           lse=lse)
    rows, _ = f.rows(0, n)
    hit = expect(out, lse, q, rows, prefill_seen(0, n, 1, n))
    assert hit.tolist() == [t >= row for t in range(n)]


@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("masks", [[0b0001, 0b0011, 0b0101, 0b1010], [0b0010] * 4, None])
def test_the_only_row_that_is_seen(kvc, H, masks):
    """No context, so a token's maximum is -inf where its only row's score is."""
    D = 4
    f = Filled(kvc, "V4", 64, [D], 10)
    set_rope(f, kvc, 1, 9, 0x7F80)
    q = queries(D, H, 10)
    out, lse = run_tree(kvc, f, q, 0, masks, D, H)
    rows, _ = f.rows(0, D)
    expect(out, lse, q, rows, tree_seen(0, masks, D) if masks else prefill_seen(0, D, 1, D))


@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("value", [-float("inf"), -3e38])
def test_scores_past_fp32(kvc, H, value):
    """One head's query meets 2.0 in one row and 0 in the others. A finite one's
    score there passes fp32: the row's weight is 0, in every token that sees it.
    An infinite one is NaN (inf times 0)."""
    D, start = 4, 150
    f = Filled(kvc, "V4", 64, [start + D], 8)
    for r in range(start + D):
        page, i = int(f.table[0, r // 64]), r % 64
        f.host[page, i * 576 + 448: i * 576 + 450] = (0, 0x40 if r == start + 1 else 0)
    f.cache = kvc.Cache(dev(f.host), "V4", 64)
    q = queries(D, H, 8)
    q[:, 1, 448] = value
    masks = [0b0001, 0b0010, 0b0100, 0b1011]
    out, lse = run_tree(kvc, f, q, start, masks, D, H)
    out, lse = out.cpu(), lse.cpu()
    rows, _ = f.rows(0, start + D)
    seen = tree_seen(start, masks, start + D)
    rest = [h for h in range(H) if h != 1]
    ref.check(out[:, rest], lse[:, rest], ref.attend(q[:, rest].double(), rows, seen, SCALE))
    if np.isinf(value):
        assert torch.isnan(out[:, 1].float()).all() and torch.isnan(lse[:, 1]).all()
        return
    seen[:, start + 1] = False
    q[:, 1, 448] = 0
    ref.check(out[:, 1:2], lse[:, 1:2], ref.attend(q[:, 1:2].double(), rows, seen, SCALE))


@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("rows_before", [33, 300])
def test_codes_past_bf16(kvc, H, rows_before):
    """A V41 group whose scale byte (one the stores never write) takes its codes
    past bf16."""
    D = 4
    f = Filled(kvc, "V41", 64, [rows_before + D], 12)
    page, i = int(f.table[0, 0]), 30
    f.host[page, i * 512 + 64:i * 512 + 96] = 0x7E
    f.host[page, 64 * 512 + i * 16 + 2] = 254
    f.cache = kvc.Cache(dev(f.host), "V41", 64)
    q = queries(D, H, 12)
    out, lse = run_tree(kvc, f, q, rows_before, None, D, H)
    rows, _ = f.rows(0, rows_before + D)
    assert not torch.isfinite(rows[i]).all()
    assert expect(out, lse, q, rows, prefill_seen(rows_before, D, 1, rows_before + D)).all()
    # a prompt, whose first tokens do not see it
    n = rows_before + D
    q = queries(n, H, 13)
    out = torch.full((n, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, H), 7.0, device="cuda")
    kvc.kvc_attend_prefill(f.cache, q.cuda(), torch.tensor([[0], [n]], dtype=torch.int32).cuda(),
                           torch.zeros(1, dtype=torch.int32).cuda(), dev(f.table), out, scale=SCALE,
                           lse=lse)
    expect(out, lse, q, rows, prefill_seen(0, n, 1, n))


def test_the_same_request_alone_and_beside_others(kvc):
    """A request's answer does not depend on the units its batch is cut into."""
    D, H, start = 2, 16, 70
    f = Filled(kvc, "V4", 64, [start + D] * 3, 9)
    set_rope(f, kvc, start, 1, 0x7F80)
    q = queries(3 * D, H, 9).cuda()
    starts = torch.tensor([start] * 3, dtype=torch.int32).cuda()
    table = dev(f.table)
    masks = as_i64([[0b01, 0b10]] * 3).cuda()
    alone = torch.empty(D, H, 512, dtype=torch.bfloat16, device="cuda")
    kvc.kvc_attend_tree(f.cache, q[:D], starts[:1], table[:1], alone, scale=SCALE, draft_len=D,
                        tree=masks[:1])
    wide = torch.empty_like(q)
    kvc.kvc_attend_prefill(f.cache, q, torch.tensor([[0, 2, 4], [2, 2, 2]], dtype=torch.int32).cuda(),
                           starts, table, wide, scale=SCALE)
    torch.cuda.synchronize()
    assert torch.isnan(alone[0].float()).all() and not torch.isnan(alone[1].float()).any()
    # (a chain: the second token sees the row too)
    assert torch.isnan(wide[:D].float()).all() and not torch.isnan(wide[D:].float()).any()
