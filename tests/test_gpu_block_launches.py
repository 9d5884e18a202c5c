"""gns_launch_count and gns_profile_read count the kernels of the training-block
operators, those of a call that launches several among them."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gns():
    import newton_schulz_gram_gb300 as m
    from newton_schulz_gram_gb300 import build
    build.build()
    m.load()
    yield m
    assert m.gns_get_status() == 0


@pytest.mark.parametrize("what,expected,classes", [
    ("dropout", 1, {"dropout": 1}), ("sort", 1, {"moe": 1}), ("long sort", 2, {"moe": 2}), ("cast", 1, {"fp8_cast": 1}),
    ("split product", 2, {"fp8_gemm": 2}), ("product", 1, {"fp8_gemm": 1}), ("few rows", 1, {"fp8_gemm": 1}),
    ("some rows", 3, {"fp8_cast": 1, "fp8_gemm": 2}), ("many rows", 2, {"fp8_cast": 1, "fp8_gemm": 1})])
def test_launches_are_counted(gns, what, expected, classes):
    x = torch.randn(4000, 2048, device="cuda").bfloat16()
    ids = torch.randint(0, 9, (5000, 2), device="cuda")
    a, b = (gns.gns_fp8_quantize(x[:n], cols=False)[0] for n in (100, 4000))
    w = gns.gns_fp8_quantize_weight(torch.randn(2048, 2048, device="cuda"))
    narrow = gns.gns_fp8_quantize_weight(torch.randn(256, 2048, device="cuda"))
    f = {"dropout": lambda: gns.gns_dropout(x, 0.5, 0, 0), "sort": lambda: gns.gns_moe_sort(ids[:2000], 9),
         "long sort": lambda: gns.gns_moe_sort(ids, 9), "cast": lambda: gns.gns_fp8_quantize(x),
         "split product": lambda: gns.gns_fp8_matmul(a, narrow), "product": lambda: gns.gns_fp8_matmul(b, w),
         "few rows": lambda: gns.gns_fp8_linear(x[:5], w), "some rows": lambda: gns.gns_fp8_linear(x[:100], narrow),
         "many rows": lambda: gns.gns_fp8_linear(x, w)}[what]
    f()
    before = gns.gns_launch_count()
    f()
    assert gns.gns_launch_count() - before == expected
    gns.gns_profile_read()
    gns.gns_profile_enable(True)
    try:
        f()
        torch.cuda.synchronize()
        read = gns.gns_profile_read()
    finally:
        gns.gns_profile_enable(False)
    assert {k: n for k, (n, _) in read.items() if n} == classes
