"""Embedding and the gradient of its table on the GPU against the fp64 oracle:
types, widths, ids outside the table, one id everywhere, ids across runs."""
import numpy as np
import pytest

from oracle import layers as L

torch = pytest.importorskip("torch")
from block_helpers import DTYPES, assert_close, f64, strided  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gns():
    import newton_schulz_gram_gb300 as m
    from newton_schulz_gram_gb300 import build
    build.build()
    m.load()
    yield m
    assert m.gns_get_status() == 0


def gradient(gns, dy, ids, vocab, scale, out_dtype=None):
    got = gns.gns_embedding_backward(dy, ids, vocab, scale=scale, out_dtype=out_dtype)
    D, I = f64(dy), ids.cpu().numpy()
    D = np.where(((I >= 0) & (I < vocab))[..., None], D, 0.0)
    want = L.embedding_backward(D, I, vocab, scale)
    mag = L.embedding_backward(np.abs(D), I, vocab, abs(scale))
    counts = np.bincount(np.clip(I, -1, vocab).reshape(-1) + 1, minlength=vocab + 2)[1:vocab + 1]
    assert got.dtype == (out_dtype or dy.dtype) and got.shape == (vocab, dy.shape[-1])
    # A row's additions, at most one per token and run, and the product with the scale.
    assert_close(got, want, mag * (counts[:, None] + 2), 0.5, "dtable")
    assert not got[torch.from_numpy(counts == 0).cuda()].any()
    return got


# Tokens up to one block of the sort and beyond, tables of one, two and three digits.
SIZES = [(1, 1, 8), (1, 1000, 16), (5, 3, 1), (31, 40, 24), (33, 1023, 33), (100, 7, 1021), (64, 1024, 256), (300, 70000, 40),
         (4096, 50, 72), (4097, 1025, 64), (9001, 2000, 65), (20000, 300, 128), (700, 1 << 21, 8)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("tokens,vocab,cols", SIZES)
def test_types_and_sizes(gns, tokens, vocab, cols, dtype):
    for k, (pad, id_type, scale) in enumerate([(0, torch.int64, 1.0), (3, torch.int32, 11.5), (8, torch.int64, -0.25)]):
        rng = np.random.default_rng(tokens + 7 * k)
        ids = rng.integers(-2, vocab + 2, tokens)
        if k == 1:  # a few ids, one of them across many runs
            ids = np.where(rng.random(tokens) < 0.7, vocab // 2, ids)
        ids = torch.from_numpy(ids).to(id_type).cuda()
        table = strided(vocab, cols, pad, DTYPES[dtype], rng) if vocab < 1 << 20 else torch.randn(vocab, cols, device="cuda").to(DTYPES[dtype])
        y = gns.gns_embedding(ids, table, scale=scale)
        want = L.embedding(ids.cpu().numpy(), f64(table), scale)
        assert_close(y, want, np.abs(want), 0.5, "y")
        dy = strided(tokens, cols, pad, DTYPES[dtype], rng)
        dy[(ids < 0) | (ids >= vocab)] = float("nan")  # padding
        gradient(gns, dy, ids, vocab, scale)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("out", list(DTYPES))
def test_output_types(gns, dtype, out):
    rng = np.random.default_rng(1)
    for cols in (64, 65):
        ids = torch.from_numpy(rng.integers(0, 30, 500)).cuda()
        gradient(gns, strided(500, cols, 0, DTYPES[dtype], rng), ids, 30, 2.0, DTYPES[out])


@pytest.mark.parametrize("tokens", [32, 33, 64, 1024, 1057, 5000, 70000, 140001])
def test_one_id_everywhere(gns, tokens):
    """Every run of the sorted tokens begins and ends inside one id; with padding, the last ones outside the table."""
    rng = np.random.default_rng(tokens)
    for dy in (strided(tokens, 48, 0, torch.float32, rng), strided(tokens, 33, 0, torch.bfloat16, rng)):
        for share in (0.0, 0.3):
            ids = torch.full((tokens,), 5, device="cuda")
            ids[torch.from_numpy(rng.random(tokens) < share).cuda()] = -1
            gradient(gns, dy, ids, 9, 1.0)


def test_runs_that_end_at_the_chunks(gns):
    """Ids of 31, 32, 33 and 64 tokens in turn: sums that end on, before and behind a chunk's end."""
    rng = np.random.default_rng(5)
    for lengths in ([32] * 9, [31, 33] * 6, [64, 32, 31, 1] * 4, [1, 63, 65, 96] * 3, [16] * 20, [320, 5, 320]):
        ids = np.repeat(np.arange(len(lengths)) * 2 + 1, lengths)
        ids = torch.from_numpy(rng.permutation(ids)).cuda()
        gradient(gns, strided(ids.numel(), 264, 0, torch.bfloat16, rng), ids, 2 * len(lengths) + 1, 1.0, torch.float32)


@pytest.mark.parametrize("lengths", [[64], [63, 65], [128, 64, 1, 63], [1, 127, 129, 191], [4096, 5, 2048]])
def test_long_runs_that_end_at_the_chunks(gns, lengths):
    """The same with tokens enough for the longest runs of 64."""
    rng = np.random.default_rng(sum(lengths))
    ids = np.repeat(np.arange(33000 // sum(lengths) * len(lengths)) * 2 + 1, lengths * (33000 // sum(lengths)))
    ids = torch.from_numpy(rng.permutation(ids)).cuda()
    gradient(gns, strided(ids.numel(), 1024, 0, torch.float32, rng), ids, int(ids.max()) + 2, 1.0)


def test_wide_rows_and_shapes(gns):
    rng = np.random.default_rng(6)
    ids = torch.from_numpy(rng.integers(0, 40, (3, 4, 50))).int().cuda()
    table = strided(40, 4096, 0, torch.bfloat16, rng)
    y = gns.gns_embedding(ids, table)
    assert y.shape == (3, 4, 50, 4096) and torch.equal(y, table[ids.long()])
    dy = torch.randn(3, 4, 50, 4096, device="cuda")
    gradient(gns, dy, ids, 40, 1.0)
    one = gns.gns_embedding(ids[0, 0, 0], table)
    assert one.shape == (4096,) and torch.equal(one, table[ids[0, 0, 0].long()])
    assert torch.equal(gns.gns_embedding_backward(dy[0, 0, 0], ids[0, 0, 0], 40)[ids[0, 0, 0].long()], dy[0, 0, 0])


def test_no_tokens(gns):
    ids = torch.zeros(0, dtype=torch.int64, device="cuda")
    table = torch.ones(7, 12, device="cuda")
    assert gns.gns_embedding(ids, table).shape == (0, 12)
    grad = gns.gns_embedding_backward(torch.zeros(0, 12, device="cuda"), ids, 7)
    assert grad.shape == (7, 12) and not grad.any()


def test_infinities_stay_in_their_rows(gns):
    ids = torch.arange(100, device="cuda") % 10
    dy = torch.ones(100, 16, device="cuda")
    dy[3, 4], dy[25, 7] = float("inf"), float("nan")
    grad = gns.gns_embedding_backward(dy, ids, 10)
    odd = ~torch.isfinite(grad)
    assert odd.sum() == 2 and odd[3, 4] and odd[5, 7]


def test_repeats_bit_for_bit(gns):
    rng = np.random.default_rng(7)
    ids = torch.from_numpy(rng.integers(0, 3000, 30000) * rng.integers(0, 2, 30000)).cuda()
    dy = torch.randn(30000, 200, device="cuda").bfloat16()
    first = gns.gns_embedding_backward(dy, ids, 3000)
    for _ in range(3):
        assert torch.equal(gns.gns_embedding_backward(dy, ids, 3000), first)


def test_a_table_beyond_2_31_elements(gns):
    """Row offsets past 32 bits, forward and backward (8.6 GB a table)."""
    vocab, cols = 1 << 20, 4096 + 8
    table = torch.empty(vocab, cols, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([0, vocab - 1, vocab - 1, 600000, -1, vocab], device="cuda")
    table[ids[:4]] = torch.randn(4, cols, device="cuda").bfloat16()
    y = gns.gns_embedding(ids, table)
    assert torch.equal(y[:4], table[ids[:4]]) and not y[4:].any()
    del table
    dy = torch.randn(6, cols, device="cuda").bfloat16()
    grad = gns.gns_embedding_backward(dy, ids, vocab)
    assert torch.equal(grad[0], dy[0]) and torch.equal(grad[600000], dy[3])
    assert torch.equal(grad[vocab - 1], (dy[1].float() + dy[2].float()).bfloat16())
    assert int((grad != 0).any(1).sum()) == 3


def test_the_most_tokens(gns):
    """2^31 - 4097 tokens of one column (60 GB with the intermediate memory): runs of 2^20,
    whose sums of ones are exact in fp32."""
    tokens, vocab = (1 << 31) - 1 - 4096, 1024
    ids = torch.arange(tokens, dtype=torch.int32, device="cuda").bitwise_and_(vocab - 1)
    grad = gns.gns_embedding_backward(torch.ones(tokens, 1, dtype=torch.bfloat16, device="cuda"), ids, vocab, out_dtype=torch.float32)
    want = torch.full((vocab,), tokens // vocab, dtype=torch.int64, device="cuda")
    want[:tokens % vocab] += 1
    assert torch.equal(grad[:, 0].long(), want)
    del ids
    gns.gns_release()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,cols", [(torch.float32, 2056), (torch.float32, 4104), (torch.bfloat16, 2049), (torch.bfloat16, 8200)])
@pytest.mark.parametrize("shares", [(0.99,), (0.5, 0.45), (0.3, 0.3, 0.3)])
def test_frequent_ids_of_wide_rows(gns, dtype, cols, shares):
    """One id, two and three that each span more than 128 runs, of rows of more than 16 strips:
    their sums are shared among blocks, and joined by the last one of each, strip by strip."""
    rng = np.random.default_rng(cols + len(shares))
    tokens, vocab = 40000, 40
    ids = rng.choice(vocab, tokens, p=[*shares, *[(1 - sum(shares)) / (vocab - len(shares))] * (vocab - len(shares))])
    ids = torch.from_numpy(ids).cuda()
    dy = strided(tokens, cols, 0, dtype, rng)
    first = gns.gns_embedding_backward(dy, ids, vocab, out_dtype=torch.float32)
    D = dy.double()
    want, mag = (torch.zeros(vocab, cols, dtype=torch.float64, device="cuda").index_add_(0, ids, t) for t in (D, D.abs()))
    counts = torch.bincount(ids, minlength=vocab)
    # A run's tokens one after the other, its id's runs by a warp's share of a block's, 16 warps, eight blocks.
    depth = (64 + counts / 64 / 128 + 16 + 8 + 2).cpu().numpy()[:, None]
    assert_close(first, f64(want), f64(mag) * depth, 0.5, "dtable")
    for _ in range(3):
        assert torch.equal(gns.gns_embedding_backward(dy, ids, vocab, out_dtype=torch.float32), first)


@pytest.mark.parametrize("cols", [2056, 2049])
def test_ids_of_many_runs_in_wide_rows(gns, cols):
    """33 to 128 runs, which one block of each strip joins, of more than 16 strips."""
    rng = np.random.default_rng(cols)
    ids = np.repeat(np.arange(6) * 3, [33 * 64, 40 * 64 + 5, 127 * 64, 64, 129 * 64, 100 * 64 + 63])
    ids = torch.from_numpy(rng.permutation(ids)).cuda()
    gradient(gns, strided(ids.numel(), cols, 0, torch.float32, rng), ids, 17, 0.5)
