"""kvc_slot_map where its sums over the slots pass 32 bits: every slot passes
the checks of its own, and tokens or pages are refused by the batch's limits.
The sums are such that, taken modulo 2^32, the last slot would fit again."""
import pytest
import torch

pytestmark = pytest.mark.gpu

TOKEN_RANGE, NO_PAGE = 64, 128


@pytest.fixture
def kvc():
    import fp8_fp4_quantized_amd as k
    yield k
    torch.cuda.empty_cache()                  # the tables are of 3 to 20 GB


def run(kvc, lens, new, table, free, tokens, page_size, num_pages):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    e = lambda *s: torch.full(s, 77, dtype=torch.int32, device="cuda")
    S = len(lens)
    o = dict(offsets=e(2, S), start_pos=e(S), out_loc=e(tokens), positions=e(tokens),
             token_to_req=e(tokens), totals=e(4))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvc.kvc_slot_map(ratio=1, page_size=page_size, num_pages=num_pages, lens=i32(lens),
                     new_lens=i32(new), page_table=table, free_pages=free, status=st, **o)
    torch.cuda.synchronize()
    return {k: v.tolist() for k, v in o.items()}, int(st)


# slots of the huge requests: neighbours in a wave, waves apart, on both sides of
# the 1,024 slots that are summed in one turn, nearly all
@pytest.mark.parametrize("S,huge", [(9, (1, 2)), (9, (1, 2, 3, 6)), (200, (70, 130)), (200, (0, 70, 130, 199)),
                                    (1500, (5, 1023, 1024, 1400)), (1500, tuple(range(3, 1489)))])
def test_token_sums_past_32_bits(kvc, S, huge):
    """Requests of 2^31 - 1 new tokens for which the table and the free list
    have the pages. They and every later slot with tokens are refused, earlier
    ones and slots without tokens are placed."""
    big, ps, width, cap = 2 ** 31 - 1, 4096, 524288, 20
    lens, new = [0] * S, [0] * S
    for b in (0, S // 2, S - 1):
        lens[b], new[b] = 5, 3
    for b in huge:
        lens[b], new[b] = 0, big
    table = torch.zeros(S, width, dtype=torch.int32, device="cuda")
    table[:, 0] = torch.arange(S, device="cuda") % 400 + 1
    free = torch.arange(1, len(huge) * width + 65, dtype=torch.int32, device="cuda")
    got, bits = run(kvc, lens, new, table, free, cap, ps, 500)
    taken = [b for b in range(min(huge)) if new[b]]
    refused = [b for b in range(S) if new[b] and b not in taken]
    assert bits == TOKEN_RANGE
    assert got["totals"] == [3 * len(taken), 3 * len(taken), 0, len(refused)]
    assert got["start_pos"] == [-1 if b in refused else lens[b] for b in range(S)]
    assert got["offsets"][0] == [3 * sum(t < b for t in taken) for b in range(S)]
    assert got["offsets"][1] == [3 if b in taken else 0 for b in range(S)]
    req, loc = [-1] * cap, [0] * cap
    for k, b in enumerate(taken):
        for j in range(3):
            req[3 * k + j], loc[3 * k + j] = b, (b % 400 + 1) * ps + 5 + j
    assert got["token_to_req"] == req and got["out_loc"] == loc
    assert table[:, 0].tolist() == [b % 400 + 1 for b in range(S)] and not table[:, 1:].any()


@pytest.mark.parametrize("S", [30, 90, 1030])            # one wave, two, two turns
def test_page_sums_past_32_bits(kvc, S):
    """A row a page and requests whose pages come to 2^32 - 3 together: they
    and the last slot, which asks for pages too, are refused for want of pages;
    the slots before them and one that asks for none are placed."""
    huge = range(2, S - 2)
    width = -(-(2 ** 32 - 3) // len(huge))
    lens, new = [0] * S, [0] * S
    new[0], new[1], new[S - 1] = 2, 1, 4
    lens[S - 2] = 6
    for b in huge:
        new[b] = width
    new[huge[-1]] -= width * len(huge) - (2 ** 32 - 3)
    assert sum(new) == 2 ** 32 + 4
    table = torch.empty(S, width, dtype=torch.int32, device="cuda")
    table[:, :8] = -5
    got, bits = run(kvc, lens, new, table, torch.arange(1, 11, dtype=torch.int32, device="cuda"), 9, 1, 100)
    refused = [b for b in range(S) if new[b] and b > 1]
    assert bits == NO_PAGE
    assert got["totals"] == [3, 3, 3, len(refused)]
    assert got["start_pos"] == [-1 if b in refused else lens[b] for b in range(S)]
    assert got["offsets"] == [[0, 2] + [3] * (S - 2), [2, 1] + [0] * (S - 2)]
    assert got["token_to_req"] == [0, 0, 1] + [-1] * 6 and got["out_loc"] == [1, 2, 3] + [0] * 6
    want = [[-5] * 8 for _ in range(S)]
    want[0][:2], want[1][0] = [1, 2], 3
    assert table[:, :8].tolist() == want
