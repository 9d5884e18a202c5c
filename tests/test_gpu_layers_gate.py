"""The router's gates, balance loss and their gradient on the GPU against the fp64
oracle: the choice exactly, with ties, masks and rows without a token; the rest
within what fp32 arithmetic leaves."""
import numpy as np
import pytest

from oracle import layers as L

torch = pytest.importorskip("torch")
from block_helpers import DTYPES, assert_close, f64  # noqa: E402

pytestmark = pytest.mark.gpu

INF = float("inf")
# fp32 roundings of a row's sums: 32 logits a lane, five steps, the exponential's
# and the logarithm's errors of up to two units each, a few single operations.
DEPTH = 50
# Below 2^-126 an exponential lies on the grid of the subnormals, where expf's error of
# up to two units is up to 2 * 2^-149, whatever the value: exp(-100) = 3.7e-44 is 26.5
# steps of that grid. Divided by a sum of at least 1 or averaged over the rows it is no
# more; as a magnitude, of which 2^-23 is allowed once per rounding:
GRID = 2 * 2.0 ** -149 * 2.0 ** 23


@pytest.fixture(scope="module")
def gns():
    import newton_schulz_gram_gb300 as m
    from newton_schulz_gram_gb300 import build
    build.build()
    m.load()
    yield m
    assert m.gns_get_status() == 0


def logits_of(tokens, experts, dtype, seed, masked=0.0, pad=0):
    rng = np.random.default_rng(seed)
    full = torch.full((tokens, experts + pad), float("nan"), dtype=dtype)
    v = torch.from_numpy(rng.normal(size=(tokens, experts)) * 2)
    if masked:
        v[torch.from_numpy(rng.random((tokens, experts)) < masked)] = -INF
        v[::5] = -INF  # rows without a token
    full[:, :experts] = v.to(dtype)
    return full.cuda()[:, :experts], rng


def check(gns, logits, topk, normalize, rng, balance=0.02, z=0.01, dloss=None):
    l = f64(logits)
    tokens, experts = l.shape
    ids, w, lse, p = L.moe_gate(l, topk, normalize)
    gate = gns.gns_moe_gate(logits, topk, normalize=normalize)
    assert gate.ids.dtype == torch.int64 and np.array_equal(gate.ids.cpu().numpy(), ids)
    live = lse > -np.inf
    finite = np.where(np.isinf(l), np.nan, l)
    span = np.zeros(tokens)  # the exponents' size, whose half step is that much of an exponential
    if live.any():
        span[live] = np.nanmax(finite[live], 1) - np.nanmin(finite[live], 1) + np.abs(lse[live])
    assert_close(gate.weights, w, w * (1 + span[:, None]) + GRID / DEPTH, DEPTH, "weights")
    got = f64(gate.lse)
    assert np.array_equal(np.isinf(got), ~live) and not np.isnan(got).any()
    assert_close(gate.lse[torch.from_numpy(live).cuda()], lse[live], 1 + np.abs(lse[live]), DEPTH, "lse")

    loss, counts, probs = gns.gns_moe_balance(logits, gate, balance, z)
    eloss, ecounts, eprobs = L.moe_balance(l, ids, balance, z)
    assert counts.dtype == torch.int32 and np.array_equal(counts.cpu().numpy(), ecounts)
    n = max(1, int(live.sum()))
    # A warp's rows one after the other, 16 warps, up to 152 blocks.
    sums = DEPTH + -(-tokens // (16 * 152)) + 16 + 152
    perr = (p * (1 + span[:, None])).sum(0) / n + GRID / sums
    assert_close(probs, eprobs, perr, sums, "probs")
    z2 = np.where(live, lse, 0.0)
    mag = balance * experts / (n * topk) * np.sum(ecounts[:-1] * perr) + z / n * np.sum(z2 * z2 + np.abs(z2))
    assert loss.dim() == 0
    assert_close(loss, np.float64(eloss), mag, sums + 64, "loss")

    dw = torch.from_numpy(rng.normal(size=(tokens, topk))).float().cuda()
    dw[gate.ids < 0] = float("nan")  # never read
    D = np.where(ids >= 0, f64(dw), 0.0)
    for with_loss in (False, True):
        args = dict(counts=counts, balance=balance, z=z, dloss=dloss) if with_loss else {}
        got = gns.gns_moe_gate_backward(dw, logits, gate, **args)
        scale = 1.0 if dloss is None else float(dloss)
        want = L.moe_gate_backward(D, l, ids, normalize, *((balance, z, scale) if with_loss else ()))
        inner = (w * np.abs(D)).sum(1, keepdims=True)
        mag = np.zeros((tokens, experts))
        for t in range(tokens):
            on = ids[t] >= 0
            mag[t, ids[t, on]] += w[t, on] * (np.abs(D[t, on]) + (inner[t] if normalize else 0)) * (1 + span[t])
        if not normalize:
            mag += p * inner * (1 + span[:, None])
        if with_loss:
            c = ecounts[:-1]
            mag += abs(scale) * p * (1 + span[:, None]) * (balance * experts / (n * n * topk) * (c + (p * c).sum(1, keepdims=True))
                                                           + 2 * z / n * np.abs(z2)[:, None])
        assert_close(got, want, mag, 3 * DEPTH, f"dlogits, loss {with_loss}")
    return gate


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("tokens,experts,topk", [(1, 1, 1), (1, 256, 8), (3, 7, 7), (50, 33, 3), (200, 64, 2), (9, 1000, 32),
                                                 (17, 1024, 8), (40, 511, 5), (5000, 12, 2)])
def test_types_and_sizes(gns, tokens, experts, topk, dtype):
    for k, (normalize, masked, pad) in enumerate([(True, 0.0, 0), (False, 0.0, 5), (True, 0.6, 0), (False, 0.6, 3)]):
        logits, rng = logits_of(tokens, experts, DTYPES[dtype], 10 * k + tokens, masked, pad)
        check(gns, logits, topk, normalize, rng, dloss=None if k % 2 else torch.tensor(-1.7, device="cuda"))


def test_ties_go_to_the_lowest_expert(gns):
    rng = np.random.default_rng(2)
    v = torch.from_numpy(rng.integers(-2, 3, (300, 100)) * 0.5).bfloat16().cuda()
    v[0] = 0.0
    v[1, ::2], v[1, 1::2] = 0.0, -0.0
    gate = check(gns, v, 9, True, rng)
    assert gate.ids[0].tolist() == list(range(9)) == gate.ids[1].tolist()


def test_values_at_the_border(gns):
    """The largest and smallest numbers, and logits so far apart that all but one vanish."""
    rng = np.random.default_rng(3)
    rows = torch.tensor([[3.0e38, -3.0e38, 0.0, 1.0], [1e-45, -1e-45, 0.0, -0.0], [100.0, -100.0, 0.0, 90.0],
                         [-INF, -INF, -INF, -3.0e38]], device="cuda")
    gate = gns.gns_moe_gate(rows, 3)
    want = L.moe_gate(f64(rows), 3)
    assert np.array_equal(gate.ids.cpu().numpy(), want[0])
    assert np.allclose(f64(gate.weights), want[1], atol=1e-6) and np.allclose(f64(gate.lse), want[2], rtol=1e-6)
    check(gns, rows[2:], 2, True, rng, z=0.0)


def test_large_logits_cost_no_digits(gns):
    """Logits around 1000, whose lse has steps of 2^-14: probabilities and their gradients
    are those of the differences, which are exact."""
    logits, rng = logits_of(64, 50, torch.float32, 12)
    logits = torch.round(logits * 1024) / 1024
    dw = torch.from_numpy(rng.normal(size=(64, 3))).float().cuda()
    outs = []
    for shift in (0.0, 1024.0):
        gate = gns.gns_moe_gate(logits + shift, 3, normalize=False)
        _, counts, probs = gns.gns_moe_balance(logits + shift, gate, 0.5)
        outs.append((gate.ids, gate.weights, probs, gns.gns_moe_gate_backward(dw, logits + shift, gate, counts, 0.5)))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_one_expert_has_no_gradient(gns):
    """Its probability is 1 whatever its logit."""
    logits = torch.randn(40, 1, device="cuda") * 30
    gate = gns.gns_moe_gate(logits, 1, normalize=False)
    loss, counts, _ = gns.gns_moe_balance(logits, gate, 0.5)
    assert loss == 0.5 and (gate.weights == 1).all()
    assert not gns.gns_moe_gate_backward(torch.randn(40, 1, device="cuda"), logits, gate, counts, 0.5).any()


def test_nan_and_infinity_stay_in_their_row(gns):
    logits, _ = logits_of(20, 40, torch.float32, 6)
    clean = gns.gns_moe_gate(logits, 4)
    bad = logits.clone()
    bad[3, 7], bad[9, 11], bad[9, 30] = float("nan"), INF, float("nan")
    gate = gns.gns_moe_gate(bad, 4)
    dw = torch.ones(20, 4, device="cuda")
    a, b = gns.gns_moe_gate_backward(dw, logits, clean), gns.gns_moe_gate_backward(dw, bad, gate)
    for t in range(20):
        if t in (3, 9):
            assert gate.weights[t].isnan().all()
        else:
            assert torch.equal(gate.ids[t], clean.ids[t]) and torch.equal(gate.weights[t], clean.weights[t]) and torch.equal(a[t], b[t])
    assert gate.ids[3, 0] == 7 and gate.ids[9, :2].tolist() == [30, 11]


def test_no_tokens_and_no_token_rows(gns):
    for tokens in (0, 6):
        logits = torch.full((tokens, 5), -INF, device="cuda")
        gate = gns.gns_moe_gate(logits, 2)
        loss, counts, probs = gns.gns_moe_balance(logits, gate, 0.1, 0.1)
        assert (gate.ids == -1).all() and not gate.weights.any() and not counts.any() and not probs.any() and loss == 0
        grad = gns.gns_moe_gate_backward(torch.full((tokens, 2), float("nan"), device="cuda"), logits, gate, counts, 0.1, 0.1)
        assert grad.shape == (tokens, 5) and not grad.any()


def test_a_gate_of_ones_own(gns):
    """Ids that repeat, that name no expert, and weights that are not the library's."""
    logits, rng = logits_of(64, 10, torch.float32, 7)
    ids = torch.from_numpy(rng.integers(-3, 14, (64, 4))).cuda()
    w = torch.rand(64, 4, device="cuda")
    lse = torch.logsumexp(logits, 1)
    gate = gns.MoeGate(ids, w, lse, 10, normalize=False)
    loss, counts, probs = gns.gns_moe_balance(logits, gate, 1.0)
    inside = (ids >= 0) & (ids < 10)
    assert counts.tolist() == torch.bincount(ids[inside], minlength=10).tolist() + [64]
    dw = torch.randn(64, 4, device="cuda")
    got = gns.gns_moe_gate_backward(dw, logits, gate)
    term = torch.where(inside, w * dw, 0.0).double()
    want = torch.zeros(64, 10, dtype=torch.float64, device="cuda").scatter_add_(1, ids.clamp(0, 9), term)
    want -= torch.softmax(logits.double(), 1) * term.sum(1, keepdim=True)
    assert torch.allclose(got.double(), want, atol=1e-5)


def test_repeats_bit_for_bit_and_feeds_the_sort(gns):
    logits, rng = logits_of(9000, 48, torch.bfloat16, 8, masked=0.3)
    gate = gns.gns_moe_gate(logits, 4)
    first = gns.gns_moe_balance(logits, gate, 0.1, 0.1)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, gns.gns_moe_balance(logits, gate, 0.1, 0.1)))
    route = gns.gns_moe_sort(gate.ids, 48)
    assert torch.equal(route.offsets.diff(), first[1][:48])


@pytest.mark.parametrize("experts", [1, 33, 256, 1024])
def test_the_loss_repeats_with_any_number_of_strips(gns, experts):
    """The loss' sum is made of what every CTA of a cluster sends, most of which have no
    expert where there are few: the same every time, calls one behind the other."""
    logits, rng = logits_of(300, experts, torch.float32, experts)
    gate = check(gns, logits, 1, True, rng)
    runs = [gns.gns_moe_balance(logits, gate, 0.02, 0.01) for _ in range(200)]
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(r, runs[0]))


@pytest.mark.parametrize("normalize", [False, True])
def test_gradient_against_differences(gns, normalize):
    """The GPU's own forward pass; the choice stays while the step does not cross a tie."""
    logits, rng = logits_of(60, 20, torch.float32, 9)
    dw = torch.from_numpy(rng.normal(size=(60, 3))).float().cuda()
    gate = gns.gns_moe_gate(logits, 3, normalize=normalize)
    _, counts, _ = gns.gns_moe_balance(logits, gate, 0.5, 0.2)
    grad = gns.gns_moe_gate_backward(dw, logits, gate, counts, 0.5, 0.2).double()
    top = logits.sort(1, descending=True)[0]
    gap = (top[:, 2] - top[:, 3]).min().item()
    d = torch.from_numpy(rng.uniform(-1, 1, size=(60, 20))).float().cuda()
    step = min(5e-3, gap / 3)

    def f(l):
        g = gns.gns_moe_gate(l, 3, normalize=normalize)
        weights = torch.zeros(60, 20, dtype=torch.float64, device="cuda").scatter_(1, g.ids, g.weights.double())
        return (weights.gather(1, gate.ids) * dw.double()).sum().item() + gns.gns_moe_balance(l, g, 0.5, 0.2)[0].double().item()

    got = (f(logits + step * d) - f(logits - step * d)) / (2 * step)
    scale = (grad * d.double()).abs().sum().item()
    # fp32 values of up to about 200 terms, each off by a few 2^-24 of weights up to 1, over the step; and its square.
    assert abs(got - (grad * d.double()).sum().item()) < 200 * 4 * 2.0 ** -24 / step + 10 * step ** 2 * scale
