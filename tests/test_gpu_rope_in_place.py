"""The rotation in place beside other writers of the same heads: the dims that are
not rotated are another stream's to write meanwhile."""
import pytest
import torch

from tests import evict_ref as ref

pytestmark = pytest.mark.gpu
BF, HF, FL = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def kvc():
    import fp8_fp4_quantized_amd as k
    return k


def inputs(kind, T, H, D, R):
    g = torch.Generator().manual_seed(D + R)
    x = torch.randn(T, H, D, generator=g).to(kind).cuda()
    f, _ = ref.table(64, 0, R, 10000.0)
    return x, torch.arange(T, dtype=torch.int32, device="cuda") % 64, torch.from_numpy(f).float().cuda()


# (rotated dims that begin, or end, or do both inside 16 bytes; at whole ones)
@pytest.mark.parametrize("kind,D,R,off", [(BF, 48, 36, 6), (HF, 48, 36, 6), (FL, 24, 12, 6), (BF, 64, 48, 8),
                                          (BF, 64, 4, 10), (BF, 48, 40, 2), (BF, 576, 64, 510), (BF, 64, 32, 16)])
def test_another_stream_writes_the_other_dims(kvc, kind, D, R, off):
    T, H = 2048, 32
    x, pos, f = inputs(kind, T, H, D, R)
    want = x.clone()
    for _ in range(12):
        kvc.kvc_rope_rows(want, pos, f, offset=off)
    here, there = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for k in range(12):
        with torch.cuda.stream(there):
            x[..., :off].fill_(k)
            x[..., off + R:].fill_(k)
        with torch.cuda.stream(here):
            kvc.kvc_rope_rows(x, pos, f, offset=off)
    torch.cuda.synchronize()
    want[..., :off] = 11
    want[..., off + R:] = 11
    assert torch.equal(x, want)


@pytest.mark.parametrize("kind", [BF, HF, FL])
def test_neighbouring_parts_on_two_streams(kvc, kind):
    """Two rotations of one head that meet inside 16 bytes."""
    T, H, D = 2048, 32, 48
    x, pos, f = inputs(kind, T, H, D, 22)
    want = x.clone()
    parts = ((0, False), (22, True))
    for _ in range(12):
        for off, back in parts:
            kvc.kvc_rope_rows(want, pos, f, offset=off, transpose=back)
    streams = [torch.cuda.Stream() for _ in parts]
    torch.cuda.synchronize()
    for _ in range(12):
        for s, (off, back) in zip(streams, parts):
            with torch.cuda.stream(s):
                kvc.kvc_rope_rows(x, pos, f, offset=off, transpose=back)
    torch.cuda.synchronize()
    assert torch.equal(x, want)
