"""The casts' C entry with rows of the 8-bit forms farther apart than they need:
what lies between them stays as it was."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
from block_helpers import DTYPES  # noqa: E402

KEEP = 0xA5


@pytest.fixture(scope="module")
def gns():
    import newton_schulz_gram_gb300 as m
    from newton_schulz_gram_gb300 import build
    build.build()
    m.load()
    yield m
    assert m.gns_get_status() == 0


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("rows,cols", [(128, 8), (70, 40), (130, 129), (256, 256), (3, 250)])
def test_gaps_between_rows_are_left_alone(gns, dtype, rows, cols):
    from newton_schulz_gram_gb300 import _lib
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g, device="cuda").to(DTYPES[dtype])
    want_r, want_c = gns.gns_fp8_quantize(x)
    want_w = gns.gns_fp8_quantize_weight(x)
    used, blocks, kb = -(-cols // 16) * 16, -(-rows // 128), -(-cols // 128)
    stream = torch.cuda.current_stream().cuda_stream
    for ld in (used, used + 16, used + 112):
        full = lambda *s: torch.full(s, KEEP, dtype=torch.uint8, device="cuda")  # noqa: E731
        r, c, w = full(rows, ld), full(blocks * 128, ld), full(rows, ld)
        sr, sc, sw = full(kb, rows + 5), full(blocks, cols + 3), full(blocks, kb)
        _lib.check(gns.load().gns_fp8_quantize(x.data_ptr(), cols, gns.block.DTYPES[x.dtype], rows, cols, None, 1, None, 1, 0,
                                               r.data_ptr(), ld, sr.data_ptr(), rows + 5, c.data_ptr(), ld, sc.data_ptr(),
                                               cols + 3, stream), "gns_fp8_quantize")
        _lib.check(gns.load().gns_fp8_quantize_weight(x.data_ptr(), cols, 0, gns.block.DTYPES[x.dtype], 1, rows, cols, 0,
                                                      w.data_ptr(), ld, sw.data_ptr(), stream), "gns_fp8_quantize_weight")
        for got, form in ((r, want_r.q), (c, want_c.q), (w, want_w.q[0])):
            assert torch.equal(got[:, :used], form.view(torch.uint8))
            assert (got[:, used:] == KEEP).all()
        assert torch.equal(sr[:, :rows], want_r.scale.view(torch.uint8)) and (sr[:, rows:] == KEEP).all()
        assert torch.equal(sc[:, :cols], want_c.scale.view(torch.uint8)) and (sc[:, cols:] == KEEP).all()
        assert torch.equal(sw, want_w.scale[0].view(torch.uint8))
