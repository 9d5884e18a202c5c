"""The training-block operators at the largest sizes that their entries accept."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

MOST_ROWS = 65535 * 128


@pytest.fixture(scope="module")
def gns():
    import newton_schulz_gram_gb300 as m
    from newton_schulz_gram_gb300 import build
    build.build()
    m.load()
    yield m
    torch.cuda.empty_cache()
    assert m.gns_get_status() == 0


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("experts", [2, 300])
def test_routed_cast_of_the_most_rows(gns, experts):
    """Each group starts a token block of its own, so there are more of them than
    rows / 128: every group's forms are those of its rows alone, and whole
    numbers make the weight gradient over them exact."""
    g = torch.Generator(device="cuda").manual_seed(experts)
    x = torch.randint(-1, 2, (MOST_ROWS, 16), generator=g, device="cuda").bfloat16()
    ids = torch.randint(0, experts, (MOST_ROWS, 1), generator=g, device="cuda")
    route = gns.gns_moe_sort(ids, experts)
    offsets = route.offsets.tolist()
    assert sum(-(-(b - a) // 128) for a, b in zip(offsets, offsets[1:])) > 65535
    rows, cols = gns.gns_fp8_quantize(x, route=route)
    dw = gns.gns_fp8_matmul_wgrad(cols, cols, route=route, out_dtype=torch.float32)
    block = 0
    for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
        r, c = gns.gns_fp8_quantize(x[a:b])
        assert same(rows.q[a:b], r.q) and same(rows.scale[:, a:b], r.scale)
        assert same(cols.q[128 * block:128 * block + c.q.shape[0]], c.q)
        assert same(cols.scale[block:block + c.blocks], c.scale)
        block += c.blocks
        assert torch.equal(dw[e], (x[a:b].double().t() @ x[a:b].double()).float())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("experts", [0, 2])
def test_16_bit_results_of_the_longest_contraction(gns, dtype, experts):
    """Values of one sign, the worst case of an accumulator that truncates. Each of
    its steps, of 32 terms, loses less than one unit in the last place of the sum
    so far (2^-23 of it at most); a result is at most 65536 terms of that away
    from its sum before it is rounded to its type, however many terms there are."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (0.5 + 0.5 * torch.rand(MOST_ROWS, 24, generator=g, device="cuda")) / 32
    dy = (0.5 + 0.5 * torch.rand(MOST_ROWS, 40, generator=g, device="cuda")) / 32
    route = None
    if experts:
        route = gns.gns_moe_sort((torch.rand(MOST_ROWS, 1, generator=g, device="cuda") < 0.3).int(), experts)
    (_, xc), (_, dc) = (gns.gns_fp8_quantize(t, route=route, rows=False) for t in (x, dy))
    offsets = route.offsets.tolist() if experts else [0, MOST_ROWS]
    dw = gns.gns_fp8_matmul_wgrad(dc, xc, route=route, out_dtype=dtype).view(-1, 40, 24)
    block = 0
    for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
        n = -(-(b - a) // 128)
        xv, dv = (c.q[128 * block:128 * (block + n), :c.cols].float().double()
                  .mul_(c.scale[block:block + n].float().double().repeat_interleave(128, 0)) for c in (xc, dc))
        exact = dv.t() @ xv
        error = ((dw[e].double() - exact).abs() / exact).max().item()
        assert error <= torch.finfo(dtype).eps / 2 + 2048 * 2.0 ** -23, (e, error)
        block += n


ONE_SM = """
import sys
import torch
sys.path.insert(0, {root!r})
import newton_schulz_gram_gb300 as gns
x, w = torch.rand(300, 33000, device="cuda"), torch.rand(8200, 33000, device="cuda")
a, b = gns.gns_fp8_quantize(x, cols=False)[0], gns.gns_fp8_quantize_weight(w)
exact = gns.gns_fp8_matmul(a, b, out_dtype=torch.float32)
got = gns.gns_fp8_matmul(a, b).float()
assert ((got - exact).abs() <= (2.0 ** -8 + 2048 * 2.0 ** -23) * exact).all()
assert gns.gns_get_status() == 0
print("near")
"""


def test_long_contraction_on_a_share_of_one_sm(gns):
    """A pair of CTAs is launched whole, and each has its own part of the carried sums."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", ONE_SM.format(root=root)], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, GNS_NUM_SMS="1"))
    assert r.returncode == 0 and r.stdout.strip() == "near", r.stdout + r.stderr
