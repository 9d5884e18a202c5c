"""The layer operators as a program uses them: beside one another on several
streams and threads, captured and replayed, under a cap of the grid, counted, and
in the block of examples/moe_muon_train.py with its norm, its balance loss and its
token rows, whose gradients are those of the same block in fp64 autograd."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.fixture(scope="module")
def gns():
    import newton_schulz_gram_gb300 as m
    from newton_schulz_gram_gb300 import build
    build.build()
    m.load()
    yield m
    assert m.gns_get_status() == 0


def job(gns, seed, dev="cuda"):
    """Inputs, and a function of them and a stream that makes every call with
    intermediate memory, among others."""
    g = torch.Generator(device=dev).manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    rows, cols, experts, vocab = 900 + 64 * seed, 640 + 128 * seed, 40 + 8 * seed, 3000 + 1000 * seed
    wide = normal(330, 12288).bfloat16()  # a row to two blocks
    ww = normal(12288)
    x, dy, w = normal(rows, cols).bfloat16(), normal(rows, cols).bfloat16(), normal(cols)
    logits, dw = normal(5000, experts), normal(5000, 4)
    ids = torch.randint(-1, vocab, (6000,), generator=g, device=dev) * torch.randint(0, 2, (6000,), generator=g, device=dev)
    de = normal(6000, 264)

    def run(scale, s):
        y, stats = gns.gns_layer_norm(x * scale, w, w, stream=s)
        out = [y, stats, *gns.gns_layer_norm_backward(dy, x * scale, stats, w, bias=True, residual=dy, stream=s)]
        y, stats = gns.gns_layer_norm(wide, ww, stream=s)
        out += [y, *gns.gns_layer_norm_backward(y, wide, stats, ww, stream=s)[:2]]
        gate = gns.gns_moe_gate(logits, 4, stream=s)
        loss, counts, probs = gns.gns_moe_balance(logits, gate, 0.1, 0.1, stream=s)
        out += [*gate, loss, counts, probs, gns.gns_moe_gate_backward(dw, logits, gate, counts, 0.1, 0.1, loss.view(1), stream=s)]
        out += [gns.gns_embedding_backward(de, ids, vocab, stream=s), gns.gns_embedding(ids, x[:, :256], stream=s)]
        return out

    return run


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b)) and len(a) == len(b)


def test_several_streams(gns):
    streams = [torch.cuda.Stream() for _ in range(4)]
    jobs = [job(gns, i) for i in range(4)]
    one = torch.ones((), device="cuda")
    want = [f(one, None) for f in jobs]
    torch.cuda.synchronize()
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                torch.cuda._sleep(400000)
        got = []
        for f, s in zip(jobs, streams):
            with torch.cuda.stream(s):  # the products with the scale, too
                got.append(f(one, s))
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))


def test_threads_that_share_a_stream(gns):
    stream = torch.cuda.Stream()
    jobs = [job(gns, i) for i in range(3)]
    one = torch.ones((), device="cuda")
    want = [f(one, None) for f in jobs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        with torch.cuda.stream(stream):
            outs = [jobs[i](one, stream) for _ in range(10)]
        stream.synchronize()
        bad.extend(i for o in outs if not same(o, want[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert bad == []


def test_threads_whose_calls_differ_in_shared_memory(gns):
    """One kernel with much and with little shared memory, and the sort with many and with
    more digits, from two threads at once: neither call takes the other's limit away."""
    wide, narrow = torch.randn(400, 7168, device="cuda").bfloat16(), torch.randn(400, 1024, device="cuda").bfloat16()
    ids = torch.randint(0, 760, (3000, 2), device="cuda")
    bad = []

    def work(x, experts):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(300):
                try:
                    gns.gns_layer_norm(x)
                    gns.gns_moe_sort(ids, experts)
                except gns.GnsError as e:
                    bad.append(str(e))

    threads = [threading.Thread(target=work, args=a) for a in ((wide, 1024), (narrow, 760), (wide, 800), (narrow, 1000))]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert bad == []


def test_two_captured_graphs_outlive_later_calls(gns):
    """Each graph has intermediate memory of its own: replayed in turn, between
    calls that use the library's and others' memory."""
    jobs = [job(gns, i) for i in range(2)]
    scales = [torch.ones((), device="cuda") for _ in jobs]
    two = torch.full((), 2.0, device="cuda")
    want = {(i, v): f(t, None) for i, f in enumerate(jobs) for v, t in ((1, scales[i].clone()), (2, two))}
    torch.cuda.synchronize()
    graphs, outs = [], []
    for f, t in zip(jobs, scales):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(f(t, None))
        graphs.append(graph)
    for order in ((0, 1), (1, 0), (0, 0, 1)):
        for value in (2, 1):
            for t in scales:
                t.fill_(value)
            gns.gns_release()
            filler = [torch.full((1 << 22,), -1, dtype=torch.int32, device="cuda") for _ in range(8)]
            jobs[0](two, None)
            for i in order:
                graphs[i].replay()
            torch.cuda.synchronize()
            for i in set(order):
                assert same(outs[i], want[i, value])
            assert all((f == -1).all() for f in filler)


CHILD = r"""
import sys
import numpy as np
import torch
sys.path.insert(0, sys.argv[1])
sys.path.insert(0, sys.argv[1] + "/tests")
import newton_schulz_gram_gb300 as gns
import test_gpu_layers_together as T
gns.load()
run, one = T.job(gns, 1), torch.ones((), device="cuda")
if sys.argv[3] == "captured":
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(one, None)
    graph.replay()
else:
    out = run(one, None)
torch.cuda.synchronize()
assert gns.gns_get_status() == 0
np.savez(sys.argv[2], *[t.double().cpu().numpy() for t in out])
"""


@pytest.mark.parametrize("how", ["captured", "capped"])
def test_in_a_process_of_its_own(gns, tmp_path, how):
    """The first calls of a process inside a capture: the same results. With every launch
    capped at two processors: those that are sums over the rows (of a norm's weights and
    of the balance loss) in another order, all others the same."""
    want = [t.double().cpu().numpy() for t in job(gns, 1)(torch.ones((), device="cuda"), None)]
    out = tmp_path / "out.npz"
    env = dict(os.environ, **({"GNS_NUM_SMS": "2"} if how == "capped" else {}))
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, str(out), how], env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    got = np.load(out)
    assert len(got.files) == len(want)
    sums = (3, 4, 7, 11, 13, 14) if how == "capped" else ()  # dweight, dbias, dweight, loss, probs, dlogits (by loss)
    for i, a in enumerate(want):
        b = got[f"arr_{i}"]
        if i in sums:
            # fp32 sums of up to 1000 rows or 5000 tokens in two orders, each within 1000 / 2 half steps of
            # the sum of the magnitudes, which is some 30 times a sum of mixed signs.
            assert np.linalg.norm(a - b) <= 30 * 1000 * 2.0 ** -24 * np.linalg.norm(a), i
        else:
            assert np.array_equal(a, b), i


@pytest.mark.parametrize("what,expected,cls", [
    ("norm", 1, "layer_norm"), ("norm rows", 1, "layer_norm"), ("backward", 1, "layer_norm"), ("backward sums", 2, "layer_norm"),
    ("backward of long rows", 3, "layer_norm"), ("gate", 1, "moe"), ("balance", 2, "moe"), ("gate backward", 1, "moe"),
    ("embedding", 1, "embedding"), ("few tokens", 2, "embedding"), ("some tokens", 3, "embedding"), ("tokens", 6, "embedding")])
def test_launches_are_counted(gns, what, expected, cls):
    x, few, long = (torch.randn(*s, device="cuda") for s in ((4000, 512), (4, 512), (3, 70001)))
    w, wl = torch.ones(512, device="cuda"), torch.ones(70001, device="cuda")
    st, sl = gns.gns_layer_norm(x)[1], gns.gns_layer_norm(long)[1]
    logits = torch.randn(4000, 16, device="cuda")
    gate = gns.gns_moe_gate(logits, 2)
    ids = torch.randint(0, 100, (4000,), device="cuda")
    f = {"norm": lambda: gns.gns_layer_norm(few), "norm rows": lambda: gns.gns_layer_norm(x, w),
         "backward": lambda: gns.gns_layer_norm_backward(x, x, st), "backward sums": lambda: gns.gns_layer_norm_backward(x, x, st, w),
         "backward of long rows": lambda: gns.gns_layer_norm_backward(long, long, sl, wl), "gate": lambda: gns.gns_moe_gate(logits, 2),
         "balance": lambda: gns.gns_moe_balance(logits, gate, 0.1),
         "gate backward": lambda: gns.gns_moe_gate_backward(gate.weights, logits, gate), "embedding": lambda: gns.gns_embedding(ids, x),
         "few tokens": lambda: gns.gns_embedding_backward(few, ids[:4], 100),
         "some tokens": lambda: gns.gns_embedding_backward(x[:700], ids[:700], 100),
         "tokens": lambda: gns.gns_embedding_backward(x, ids, 4000)}[what]
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
    assert {k: n for k, (n, _) in read.items() if n} == {cls: expected}


# ------------------------------------------------------------- the example

@pytest.fixture(scope="module")
def example(gns):
    import moe_muon_train
    return moe_muon_train


def test_gradients_of_the_whole_block(example, gns):
    """Token rows, norm, gates, balance loss, experts, dropout and back: each gradient
    near that of fp64 autograd. Two 8-bit products of 2^-4 at worst, 2^-5.8 rms, lie on
    the way to each, as in the block alone: 10 % bounds them, a wrong sign, mask, order
    or scale does not stay below it."""
    vocab, width = 90, 256
    block = example.MoeBlock(width=width, hidden=160, experts=6, topk=2, dropout=0.1, seed=3, norm=True, balance=0.5, z=0.1)
    g = torch.Generator(device="cuda").manual_seed(4)
    block.scale += 0.2 * torch.randn(width, generator=g, device="cuda")
    ids = torch.randint(-1, vocab, (300,), generator=g, device="cuda")
    table = torch.randn(vocab, width, generator=g, device="cuda").bfloat16()
    dz = torch.randn(300, width, generator=g, device="cuda").bfloat16()
    x = gns.gns_embedding(ids, table, scale=2.0)
    z, saved = block.forward(x, 5, 6)
    dx, *grads = block.backward(dz, saved)
    grads = [gns.gns_embedding_backward(dx, ids, vocab, scale=2.0, out_dtype=torch.float32), *grads]
    chosen = saved[1]
    keep = gns.gns_dropout(torch.ones_like(x), 0.1, 5, 6).double()

    leaves = [t.double().requires_grad_() for t in (table, block.router, block.up, block.down, block.scale)]
    tab, router, up, down, scale = leaves
    xd = torch.where((ids >= 0)[:, None], 2.0 * tab[ids.clamp(min=0)], 0.0)
    n = xd * torch.rsqrt(xd.square().mean(1, keepdim=True) + 1e-5) * scale
    logits = n @ router.t()
    gates = torch.softmax(logits.gather(1, chosen), dim=1)
    out = torch.zeros_like(xd)
    for e in range(6):
        y = torch.relu(n @ up[e].t()).square() @ down[e].t()
        out = out + ((chosen == e) * gates).sum(1, keepdim=True) * y
    exact = xd + keep * out
    share = torch.bincount(chosen.reshape(-1), minlength=6).double() / chosen.numel()
    loss = 0.5 * 6 * (share * torch.softmax(logits, 1).mean(0)).sum() + 0.1 * torch.logsumexp(logits, 1).square().mean()
    ((exact * dz.double()).sum() + loss).backward()
    assert abs(block.loss.item() - loss.item()) < 0.02 * abs(loss.item())  # made of bf16 rows alone
    names = ("z", "d_table", "d_router", "d_up", "d_down", "d_scale")
    for name, got, want in zip(names, (z, *grads), (exact.detach(), *(t.grad for t in leaves))):
        rel = ((got.double() - want).norm() / want.norm()).item()
        assert rel < 0.1, (name, rel)


def test_the_example_runs_with_all_of_it(example):
    losses = example.train(steps=6, tokens=512, width=256, hidden=128, experts=8, topk=2, norm=True, balance=0.01, vocab=300)
    assert len(losses) == 6 and all(np.isfinite(losses))
