"""The rotary table and the rotation of heads on the GPU against 64-bit
references: scalings, far positions, both pairings, parts of a head, strides,
types, odd sizes, in place, the transposed rotation as the backward pass, other
streams, captured graphs."""
import numpy as np
import pytest
import torch

from tests import evict_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    import fp8_fp4_quantized_amd as k
    return k


# n, first, rot, base, more
TABLES = [
    (1, 0, 64, 10000.0, {}),
    (4097, 0, 64, 10000.0, {}),
    (513, 2 ** 31 - 513, 64, 10000.0, {}),                    # up to the last position
    (1000, 999_000, 64, 500000.0, dict(scaling="linear", factor=4.0)),
    (333, 70_000, 128, 10000.0, dict(scaling="base", factor=8.0)),
    (700, 65_000, 64, 10000.0, dict(scaling="parts", factor=16.0, original=4096, mscale=1.2)),
    (700, 1_000_000, 64, 160000.0, dict(scaling="parts", factor=40.0, original=65536,
                                        beta_fast=32, beta_slow=1)),
    (50, 3, 64, 10000.0, dict(scaling="parts", factor=2.0, original=6.0, beta_fast=1, beta_slow=1)),
    (259, 5, 2, 10000.0, {}),                                 # one pair
    (97, 5, 6, 100.0, dict(scaling="base", factor=2.0)),      # three pairs
    (61, 0, 512, 10000.0, {}),                                # the widest
    (61, 7, 510, 10000.0, {}),                                # the widest odd number of pairs
    (5000, 11, 26, 1e6, {}),
]


@pytest.mark.parametrize("n,first,rot,base,more", TABLES)
def test_table(kvc, n, first, rot, base, more):
    out = torch.full((n + 1, rot), 7.0, device="cuda")
    kvc.kvc_rope_table(out[:n], first=first, base=base, **more)
    want, tol = ref.table(n, first, rot, base, **more)
    got = out.cpu().double().numpy()
    assert (got[n] == 7.0).all()
    assert (np.abs(got[:n] - want) <= tol).all()


def test_table_serves_the_rotary_store(kvc):
    """A table of this call and one of numpy's are the same to the store."""
    from tests.gpu_util import dev
    t = torch.empty(256, 64, device="cuda")
    kvc.kvc_rope_table(t, base=10000.0)
    want, _ = ref.table(256, 0, 64, 10000.0)
    rows = torch.randn(256, 512, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    pos = torch.arange(256, dtype=torch.int32, device="cuda")
    loc = pos + 64
    caches = []
    for f in (t, dev(want.astype(np.float32))):
        c = kvc.Cache(torch.zeros(6, 64 * 528, dtype=torch.uint8, device="cuda"), "V41", 64)
        kvc.kvc_store_rows_rope(c, rows, pos, f, loc)
        caches.append(c.data)
    # (entries that differ by an fp32 step move a code only next to a border)
    assert (caches[0] != caches[1]).float().mean().item() < 1e-4


BF, HF, FL = torch.bfloat16, torch.float16, torch.float32
# type, tokens, heads, dim, rot, offset, half, transpose
HEADS = [
    (BF, 1, 1, 64, 64, 0, False, False),
    (BF, 7, 16, 512, 64, 448, False, False),
    (BF, 33, 128, 512, 64, 448, False, True),
    (BF, 300, 5, 512, 64, 448, True, False),
    (HF, 19, 12, 128, 128, 0, True, True),
    (HF, 5, 3, 192, 64, 128, False, False),
    (FL, 21, 7, 128, 32, 64, True, False),
    (FL, 6, 9, 576, 64, 512, False, True),
    (BF, 9, 4, 96, 48, 8, False, False),       # pairs that end inside 16 bytes of neither
    (BF, 9, 4, 96, 36, 6, False, False),       # ... that begin and end inside 16 bytes
    (BF, 9, 4, 96, 36, 6, True, False),
    (BF, 9, 4, 96, 36, 5, False, True),        # pairs over a 16-byte border
    (HF, 4, 3, 31, 30, 1, False, False),       # odd everything
    (FL, 11, 2, 13, 6, 4, True, True),
    (BF, 3, 2, 2, 2, 0, False, False),
    (BF, 2, 1024, 8, 4, 4, False, False),
    (FL, 2, 2, 8192, 512, 7000, True, False),
    (BF, 4000, 1, 8, 8, 0, True, False),
]


def make(kind, T, H, D, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=g) * 3
    x[torch.rand(T, H, D, generator=g) < 0.05] = 0
    return x.to(kind)


def freqs_of(max_pos, rot):
    f, _ = ref.table(max_pos, 0, rot, 10000.0)
    return torch.from_numpy(f.astype(np.float32))


def close(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, first {bad.nonzero()[:3].tolist()}"


@pytest.mark.parametrize("kind,T,H,D,R,off,half,tr", HEADS)
def test_rotation(kvc, kind, T, H, D, R, off, half, tr):
    x = make(kind, T, H, D, T + H + D)
    pos = torch.randint(0, 200, (T,), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    f = freqs_of(200, R)
    want, tol = ref.rope(x, pos, f, off, half, tr)
    kw = dict(offset=off, half=half, transpose=tr)
    d = x.cuda()
    out = torch.full((T + 1, H, D), 7.0, dtype=kind, device="cuda")
    kvc.kvc_rope_rows(d, pos.cuda(), f.cuda(), out[:T], **kw)
    close(out[:T].cpu(), want, tol)
    assert (out[T] == 7).all() and torch.equal(d.cpu(), x)
    # in place, and heads with other rows between them: the same bits
    wide = torch.full((T, 2, H, D + 16), 5.0, dtype=kind, device="cuda")
    view = wide[:, 1, :, 8:8 + D]
    view.copy_(d)
    kvc.kvc_rope_rows(view, pos.cuda(), f.cuda(), **kw)
    assert torch.equal(view.cpu(), out[:T].cpu())
    assert (wide[:, 0] == 5).all() and (wide[:, 1, :, :8] == 5).all() and (wide[:, 1, :, 8 + D:] == 5).all()
    # heads before tokens
    turned = d.transpose(0, 1).contiguous().transpose(0, 1)
    out2 = torch.zeros(H, T, D, dtype=kind, device="cuda").transpose(0, 1)
    kvc.kvc_rope_rows(turned, pos.cuda(), f.cuda(), out2, **kw)
    assert torch.equal(out2.cpu(), out[:T].cpu())


@pytest.mark.parametrize("shift", [1, 2, 4])
def test_addresses_that_are_not_of_16_bytes(kvc, shift):
    x = make(BF, 5, 3, 64, 1)
    pos = torch.arange(5, dtype=torch.int32)
    f = freqs_of(8, 64)
    want, tol = ref.rope(x, pos, f, 0, False, False)
    buf = torch.zeros(5 * 3 * 64 + 8, dtype=BF, device="cuda")
    view = buf[shift:shift + 5 * 3 * 64].view(5, 3, 64)
    view.copy_(x)
    out = torch.zeros(5, 3, 64, dtype=BF, device="cuda")
    kvc.kvc_rope_rows(view, pos.cuda(), f.cuda(), out)
    close(out.cpu(), want, tol)
    kvc.kvc_rope_rows(x.cuda(), pos.cuda(), f.cuda(), view)
    assert torch.equal(view.cpu(), out.cpu())
    assert (buf[:shift] == 0).all() and (buf[shift + 5 * 3 * 64:] == 0).all()


def test_table_at_an_8_byte_address(kvc):
    x = make(BF, 5, 3, 64, 1)
    pos = torch.arange(5, dtype=torch.int32)
    f = freqs_of(8, 64)
    buf = torch.zeros(8 * 64 + 2, device="cuda")
    at = buf[2:].view(8, 64)
    at.copy_(f)
    a, b = (torch.zeros(5, 3, 64, dtype=BF, device="cuda") for _ in range(2))
    kvc.kvc_rope_rows(x.cuda(), pos.cuda(), f.cuda(), a)
    kvc.kvc_rope_rows(x.cuda(), pos.cuda(), at, b)
    assert torch.equal(a, b)


def test_positions_outside_the_table(kvc):
    x = make(BF, 6, 2, 64, 5).cuda()
    pos = torch.tensor([0, -1, 8, 7, 2 ** 31 - 1, 3], dtype=torch.int32)
    f = freqs_of(8, 64)
    out = torch.full_like(x, 9.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvc.kvc_rope_rows(x, pos.cuda(), f.cuda(), out, status=status)
    assert status.item() == kvc.STATUS_POS_RANGE
    good = torch.tensor([0, 3, 5])
    want, tol = ref.rope(x.cpu()[good], pos[good], f, 0, False, False)
    close(out.cpu()[good], want, tol)
    assert (out.cpu()[[1, 2, 4]] == 9).all()
    kvc.kvc_rope_rows(x[:0], pos[:0].cuda(), f.cuda(), out[:0])    # no tokens


def test_values_that_are_not_finite_stay_in_their_pair(kvc):
    x = make(FL, 3, 2, 64, 6)
    x[1, 0, 4], x[2, 1, 63], x[0, 1, 0] = float("nan"), float("inf"), -float("inf")
    pos = torch.arange(3, dtype=torch.int32) + 1
    f = freqs_of(8, 64)
    want, tol = ref.rope(x, pos, f, 0, False, False)
    out = x.cuda()
    kvc.kvc_rope_rows(out, pos.cuda(), f.cuda())
    got = out.cpu().double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and int((~fin).sum()) == 6
    close(got[fin], want[fin], tol[fin])


@pytest.mark.parametrize("half", [False, True])
def test_backward_is_the_transposed_rotation(kvc, half):
    """Against the gradient of the formula and against differences."""
    T, H, D, R, off = 5, 3, 24, 16, 8
    g = torch.Generator().manual_seed(8)
    x = torch.randn(T, H, D, generator=g)
    dy = torch.randn(T, H, D, generator=g)
    pos = torch.randint(0, 50, (T,), generator=g, dtype=torch.int32)
    f = (freqs_of(50, R) * 1.25)                              # with an mscale
    leaf = x.double().requires_grad_()
    a, b = ((leaf[..., off:off + R // 2], leaf[..., off + R // 2:]) if half
            else (leaf[..., off::2], leaf[..., off + 1::2]))
    c, s = f[pos.long(), 0::2].double()[:, None], f[pos.long(), 1::2].double()[:, None]
    ya, yb = a * c - b * s, a * s + b * c
    y = torch.cat([leaf[..., :off], torch.cat([ya, yb], 2) if half
                   else torch.stack([ya, yb], 3).flatten(2)], 2)
    (y * dy.double()).sum().backward()
    dx = dy.cuda()
    kvc.kvc_rope_rows(dx, pos.cuda(), f.cuda(), offset=off, half=half, transpose=True)
    # (three fp32 roundings of two products each, both at most 1.25 |dy|)
    tol = 4 * 2.0 ** -24 * 2.5 * dy.abs().max().item()
    assert (dx.cpu().double() - leaf.grad).abs().max().item() <= tol

    def loss(v):
        out = v.float().cuda()
        kvc.kvc_rope_rows(out, pos.cuda(), f.cuda(), offset=off, half=half)
        return (out.cpu().double() * dy.double()).sum().item()
    for i in ((0, 0, 0), (1, 2, 8), (4, 1, 15), (2, 0, 23)):
        # (the map is linear: a difference over 2 eps is its entry, up to the
        # outputs' fp32 roundings, of at most 1.25 (|x| + 1) each, over eps)
        e = torch.zeros(T, H, D)
        e[i] = 1.0
        diff = (loss(x + e) - loss(x - e)) / 2
        slack = 4 * 2.0 ** -24 * 2.5 * (x.abs().sum() + 1).item() * dy.abs().max().item()
        assert abs(diff - leaf.grad[i].item()) <= slack


def test_there_and_back(kvc):
    x = make(BF, 40, 16, 512, 9).cuda()
    pos = torch.randint(0, 5000, (40,), generator=torch.Generator().manual_seed(4), dtype=torch.int32).cuda()
    f = freqs_of(5000, 64).cuda()
    y, z = torch.empty_like(x), torch.empty_like(x)
    kvc.kvc_rope_rows(x, pos, f, y)
    kvc.kvc_rope_rows(y, pos, f, z, transpose=True)
    # a rounding of each of a pair's dims and one of the result
    pair = x.double().view(40, 16, 256, 2).pow(2).sum(3).sqrt().repeat_interleave(2, 2)
    assert ((z.double() - x.double()).abs() <= 3 * 2.0 ** -8 * pair + 1e-30).all()
    assert torch.equal(z[..., :448], x[..., :448])


def test_other_stream_and_graph(kvc):
    x = make(BF, 64, 16, 512, 10).cuda()
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    f = torch.empty(128, 64, device="cuda")
    out, eager = torch.zeros_like(x), torch.zeros_like(x)
    kvc.kvc_rope_table(f)
    kvc.kvc_rope_rows(x, pos, f, eager)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        kvc.kvc_rope_rows(x, pos, f, out)
    s.synchronize()
    assert torch.equal(out, eager)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvc.kvc_rope_table(f)
        kvc.kvc_rope_rows(x, pos, f, out)
    for turn in range(3):
        pos.copy_(torch.arange(64, dtype=torch.int32, device="cuda") + 13 * turn)
        out.zero_(), f.zero_()
        g.replay()
        torch.cuda.synchronize()
        kvc.kvc_rope_table(f)
        kvc.kvc_rope_rows(x, pos, f, eager)
        assert torch.equal(out, eager)


# dim, rot, offset, half: by 16 bytes, by any address, pair by pair
@pytest.mark.parametrize("kind", [BF, HF, FL])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("D,R,off,half", [(32, 6, 2, False), (32, 18, 10, False), (32, 6, 3, False), (29, 6, 2, False),
                                          (32, 16, 8, True), (32, 6, 5, True), (3, 2, 0, False)])
def test_copied_dims_keep_their_bits(kvc, kind, in_place, D, R, off, half):
    """Also those of a signalling NaN, a subnormal or a negative zero."""
    whole = torch.int32 if kind == FL else torch.int16
    odd = {BF: [0x7F81, -0x7F, 1, -0x8000, 0x7F80], HF: [0x7C01, -0x3FF, 1, -0x8000, 0x7C00],
           FL: [0x7F800001, -0x7FFFFF, 1, -0x80000000, 0x7F800000]}[kind]
    x = torch.tensor(odd, dtype=whole).repeat(5 * 3 * D)[:5 * 3 * D].view(5, 3, D).cuda()
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    out = x.clone() if in_place else torch.zeros_like(x)
    kvc.kvc_rope_rows(out.view(kind) if in_place else x.view(kind), pos, freqs_of(8, R).cuda(), out.view(kind),
                      offset=off, half=half)
    copied = [d for d in range(D) if not off <= d < off + R]
    assert torch.equal(out[..., copied], x[..., copied])


def test_more_pairs_than_a_launch_has_threads(kvc):
    """Pair by pair (in place, an odd offset), 2^32 pairs and some."""
    T, D, R, n = 2 ** 24 + 5, 515, 512, 300
    some = make(HF, n, 1, D, 9).cuda()
    f = freqs_of(64, R).cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda") % 64
    x = torch.zeros(T, 1, D, dtype=HF, device="cuda")
    for at in (0, 2 ** 23 - 100, T - n):
        x[at:at + n] = some
    kvc.kvc_rope_rows(x, pos, f, offset=1)
    for at in (0, 2 ** 23 - 100, T - n):
        want = some.clone()
        kvc.kvc_rope_rows(want, pos[at:at + n].contiguous(), f, offset=1)
        assert torch.equal(x[at:at + n], want) and not torch.equal(want, some)
    assert not x[n:2 ** 23 - 100].any() and not x[2 ** 23 - 100 + n:T - n].any()
