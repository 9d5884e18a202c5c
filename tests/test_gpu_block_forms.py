"""The forms that a training step of an expert bucket uses: grouped products and
the routed fused layer with 16-bit results, whose last rows of a group leave by
other stores than full pieces; routed casts in which a block of threads takes
several column blocks; fp32 weight gradients of several segments by pairs."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
from block_helpers import DTYPES, assert_close  # noqa: E402
from test_gpu_block_fp8 import adds, check_dense, loud, route_of, values_cols, values_rows, values_weight  # noqa: E402


@pytest.fixture(scope="module")
def gns():
    import newton_schulz_gram_gb300 as m
    from newton_schulz_gram_gb300 import build
    build.build()
    m.load()
    yield m
    assert m.gns_get_status() == 0


@pytest.mark.parametrize("out", ["bf16", "fp16"])
@pytest.mark.parametrize("tokens,topk,experts,n,k,drop", [
    (60, 3, 7, 200, 304, 0.2), (300, 2, 5, 257, 130, 0), (500, 4, 300, 64, 96, 0.1), (64, 8, 1024, 33, 48, 0.5),
    (700, 2, 3, 264, 520, 0.1), (1500, 2, 4, 1032, 640, 0.3), (1100, 1, 6, 136, 1030, 0)])
def test_grouped_products_in_16_bits(gns, out, tokens, topk, experts, n, k, drop):
    rng = np.random.default_rng(tokens + n)
    route, (offsets, rows, slots) = route_of(gns, tokens, topk, experts, drop, n)
    # Moderate magnitudes: the bound is the rounding to 16 bits, not the range of fp16.
    x = loud(tokens, k, 0, torch.bfloat16, rng).clamp(-8, 8)
    dy = loud(tokens * topk, n, 0, torch.bfloat16, rng).clamp(-8, 8)
    wq = gns.gns_fp8_quantize_weight(loud(experts * n, k, 0, torch.bfloat16, rng).clamp(-1, 1).view(experts, n, k) / 16)
    xr, xc = gns.gns_fp8_quantize(x, route=route, gather=True)
    dr, dc = gns.gns_fp8_quantize(dy, route=route)
    dtype = DTYPES[out]
    y, dx = (f(a, wq, route=route, out_dtype=dtype) for f, a in ((gns.gns_fp8_matmul, xr), (gns.gns_fp8_matmul_dgrad, dr)))
    dw = gns.gns_fp8_matmul_wgrad(dc, xc, route=route, out_dtype=dtype)
    live = offsets[-1]
    assert torch.all(y[live:] == 0) and torch.all(dx[live:] == 0)
    wv, xv, dv = values_weight(wq), values_rows(xr), values_rows(dr)
    xcv, dcv = values_cols(xc, offsets), values_cols(dc, offsets)
    for g in range(experts):
        at = slice(offsets[g], offsets[g + 1])
        if at.start == at.stop:
            assert torch.all(dw[g] == 0)
            continue
        for what, got, a, b, inner in (("y", y[at], xv[at], wv[g].T, k), ("dx", dx[at], dv[at], wv[g], n),
                                       ("dw", dw[g], dcv[at].T, xcv[at], at.stop - at.start)):
            assert_close(got, a @ b, np.abs(a) @ np.abs(b), adds(inner), f"{what} of expert {g}")


@pytest.mark.parametrize("out", ["bf16", "fp16"])
@pytest.mark.parametrize("tokens,topk,experts,n,k,drop", [
    (1, 8, 256, 64, 512, 0), (2, 4, 5, 100, 140, 0.4), (16, 2, 40, 200, 140, 0.3), (40, 3, 6, 100, 144, 0.2),
    (200, 2, 9, 264, 384, 0.1)])
def test_routed_layer_in_16_bits(gns, out, tokens, topk, experts, n, k, drop):
    rng = np.random.default_rng(tokens + n + k)
    x = loud(tokens, k, 0, torch.bfloat16, rng).clamp(-8, 8)
    route, (offsets, rows, slots) = route_of(gns, tokens, topk, experts, drop, n, skew=False)
    wq = gns.gns_fp8_quantize_weight(loud(experts * n, k, 0, torch.bfloat16, rng).clamp(-1, 1).view(experts, n, k) / 16)
    got = gns.gns_fp8_linear(x, wq, route=route, out_dtype=DTYPES[out])
    a, b = values_rows(gns.gns_fp8_quantize(x, cols=False)[0])[slots // topk], values_weight(wq)
    assert torch.all(got[offsets[-1]:] == 0)
    for g in range(experts):
        at = slice(offsets[g], offsets[g + 1])
        if at.start < at.stop:
            assert_close(got[at], a[at] @ b[g].T, np.abs(a[at]) @ np.abs(b[g]).T, adds(k), f"expert {g}")


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("cols", [2048, 2050, 1800])
@pytest.mark.parametrize("gather", [True, False])
def test_routed_cast_of_a_large_batch(gns, dtype, cols, gather):
    """32000 slots: a block of threads takes several column blocks. A cast of 128
    columns alone takes one, and its blocks are the same."""
    route, (offsets, _, _) = route_of(gns, 4000, 8, 256, 0.05, cols)
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(4000 if gather else 32000, cols, generator=g, device="cuda")
    x = (x * torch.exp(2 * torch.randn(1, cols, generator=g, device="cuda"))).to(DTYPES[dtype])
    live, blocks = offsets[-1], int(sum(-(-np.diff(offsets) // 128)))
    u8 = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    r, c = gns.gns_fp8_quantize(x, route=route, gather=gather)
    only = gns.gns_fp8_quantize(x, route=route, gather=gather, rows=False)[1]
    for c0 in range(0, cols, 128):
        part = x[:, c0:c0 + 128].contiguous()
        n = part.shape[1]
        pr, pc = gns.gns_fp8_quantize(part, route=route, gather=gather)
        kb = c0 // 128
        assert torch.equal(u8(r.q[:live, c0:c0 + n]), u8(pr.q[:live, :n]))
        assert torch.equal(u8(r.scale[kb, :live]), u8(pr.scale[0, :live]))
        for form in (c, only):
            assert torch.equal(u8(form.q[:128 * blocks, c0:c0 + n]), u8(pc.q[:128 * blocks, :n]))
            assert torch.equal(u8(form.scale[:blocks, c0:c0 + n]), u8(pc.scale[:blocks]))


@pytest.mark.parametrize("tokens,n,k", [(5000, 2304, 2304), (4100, 2500, 2333), (2049, 4608, 1200)])
def test_fp32_results_by_pairs(gns, tokens, n, k):
    rng = np.random.default_rng(n)
    check_dense(gns, loud(tokens, k, 0, torch.bfloat16, rng), loud(n, k, 0, torch.bfloat16, rng),
                loud(tokens, n, 0, torch.bfloat16, rng), torch.float32)


@pytest.mark.parametrize("out", sorted(DTYPES))
def test_contractions_of_several_long_segments(gns, out):
    """16-bit results carry their sums over 32768 terms at a time; groups of one,
    two and three such segments, and one that ends just past a segment."""
    counts = [40000, 70000, 100, 32769, 32768]
    ids = torch.cat([torch.full((n,), e) for e, n in enumerate(counts)]).cuda()
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(0)).cuda()]
    route = gns.gns_moe_sort(ids.view(-1, 1), len(counts))
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.randn(len(ids), n, generator=g, device="cuda") / 16 for n in (300, 140))
    xc, dc = (gns.gns_fp8_quantize(t, route=route, rows=False)[1] for t in (x, dy))
    dw = gns.gns_fp8_matmul_wgrad(dc, xc, route=route, out_dtype=DTYPES[out])
    offsets = np.concatenate([[0], np.cumsum(counts)])
    xv, dv = values_cols(xc, offsets), values_cols(dc, offsets)
    for e in range(len(counts)):
        a, b = dv[offsets[e]:offsets[e + 1]].T, xv[offsets[e]:offsets[e + 1]]
        assert_close(dw[e], a @ b, np.abs(a) @ np.abs(b), adds(counts[e]), f"expert {e}")
