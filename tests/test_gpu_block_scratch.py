"""Intermediate memory of the training-block operators: calls that overlap on
several streams do not meet in it, and a captured graph keeps its own whatever
the library does between the capture and a replay."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest

from oracle import block as B

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


def ids_of(tokens, topk, experts, seed):
    ids = np.random.default_rng(seed).integers(-1, experts, (tokens, topk))
    return torch.from_numpy(ids).cuda(), B.moe_sort(ids, experts)


def same_route(route, want):
    return all(np.array_equal(a.cpu().numpy().reshape(-1), b.reshape(-1)) for a, b in zip(route, want))


def use_memory(gns):
    """Makes the library replace its workspace and overwrite what it held, and
    other allocations take what that freed."""
    gns.gns_release()
    g = torch.randn(2, 512, 1024, device="cuda")
    gns.gns_orthogonalize_batched(g)
    big = torch.randn(4, 2048, 4096, device="cuda")
    gns.gns_orthogonalize_batched(big)
    filler = [torch.full((1 << 22,), -1, dtype=torch.int32, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    return filler


def test_sorts_on_several_streams(gns):
    """Sorts whose counts lie in intermediate memory, each stream with its own
    ids, queued behind one another so that they run side by side."""
    streams = [torch.cuda.Stream() for _ in range(4)]
    jobs = [ids_of(20000 + 977 * i, 3, 5 + 200 * i, i) for i in range(4)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                torch.cuda._sleep(200000)
        routes = [gns.gns_moe_sort(ids, 5 + 200 * i, stream=s) for i, ((ids, _), s) in enumerate(zip(jobs, streams))]
        torch.cuda.synchronize()
        for route, (_, want) in zip(routes, jobs):
            assert same_route(route, want)


def test_a_captured_sort_outlives_later_calls(gns):
    ids, want = ids_of(30000, 2, 64, 9)
    other, want_other = ids_of(30000, 2, 64, 10)
    gns.gns_moe_sort(ids, 64)
    torch.cuda.synchronize()
    graph, static = torch.cuda.CUDAGraph(), ids.clone()
    with torch.cuda.graph(graph):
        route = gns.gns_moe_sort(static, 64)
    for now, expected in ((ids, want), (other, want_other)):
        filler = use_memory(gns)
        static.copy_(now)
        graph.replay()
        torch.cuda.synchronize()
        assert same_route(route, expected)
        assert all((f == -1).all() for f in filler)


def layers(gns, seed):
    """Products with intermediate memory, as functions of (x, stream): the fused
    layer of many rows, the split product and both split gradients."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, k = 700 + 128 * seed, 4096
    w = gns.gns_fp8_quantize_weight(torch.randn(n, k, generator=g, device="cuda"))
    wt = gns.gns_fp8_quantize_weight(torch.randn(k, n, generator=g, device="cuda"))
    rows = lambda x, s: gns.gns_fp8_quantize(x, cols=False, stream=s)[0]  # noqa: E731
    x = torch.randn(40 + 8 * seed, k, generator=g, device="cuda").bfloat16()
    return x, (lambda x, s: gns.gns_fp8_linear(x, w, out_dtype=torch.float32, stream=s),
               lambda x, s: gns.gns_fp8_matmul(rows(x, s), w, stream=s),
               lambda x, s: gns.gns_fp8_matmul_dgrad(rows(x, s), wt, out_dtype=torch.float32, stream=s))


def test_products_on_several_streams(gns):
    streams = [torch.cuda.Stream() for _ in range(4)]
    jobs = [layers(gns, i) for i in range(4)]
    ids, want_route = ids_of(20000, 3, 70, 4)
    want = [[f(x, None) for f in fs] for x, fs in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                torch.cuda._sleep(400000)
        got = [[] for _ in jobs]
        for k in range(3):
            for out, (x, fs), s in zip(got, jobs, streams):
                out.append(fs[k](x, s))
        route = gns.gns_moe_sort(ids, 70, stream=streams[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for out, exact in zip(got, want) for a, b in zip(out, exact))
        assert same_route(route, want_route)


def test_captured_products_outlive_later_calls(gns):
    x, fs = layers(gns, 2)
    other = torch.randn_like(x)
    want = {id(t): [f(t, None) for f in fs] for t in (x, other)}
    torch.cuda.synchronize()
    graph, static = torch.cuda.CUDAGraph(), x.clone()
    with torch.cuda.graph(graph):
        outs = [f(static, None) for f in fs]
    for t in (other, x):
        filler = use_memory(gns)
        fs[0](torch.randn(4000, 4096, device="cuda"), None)
        static.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want[id(t)]))
        assert all((f == -1).all() for f in filler)


FIRST_CALLS = """
import sys
import threading
import torch
sys.path.insert(0, {root!r})
import newton_schulz_gram_gb300 as gns
gns.load()
x = torch.randn(300, 4096, device="cuda")
ids = torch.randint(0, 6, (5000, 2), device="cuda")
w = torch.randn(200, 4096, device="cuda")

def calls():
    d = gns.gns_dropout(x, 0.3, 1, 2)
    route = gns.gns_moe_sort(ids, 6)
    w8 = gns.gns_fp8_quantize_weight(w)
    return [d, *route, *(gns.gns_fp8_linear(x[:n], w8, out_dtype=torch.float32) for n in (3, 40, 300))]

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = calls()
graph.replay()
torch.cuda.synchronize()
for a, b in zip(captured, calls()):
    assert torch.equal(a, b)
assert gns.gns_get_status() == 0
print("same")
"""


def test_the_first_calls_of_a_process_can_be_captured(gns):
    """What the library sets up on first use (status block, memory pool, kernel
    attributes) does not break a capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(root=root)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stdout + r.stderr


def test_more_streams_than_kept_buffers(gns):
    """Each stream with rows of its own through the same layer, and the buffers
    released in between."""
    gns.gns_release()
    x, fs = layers(gns, 1)
    streams = [torch.cuda.Stream() for _ in range(24)]
    jobs = [x * (1 + i) for i in range(24)]
    want = [fs[0](j, None) for j in jobs]
    for _ in range(3):
        torch.cuda.synchronize()
        got = [fs[0](j, s) for j, s in zip(jobs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert gns.gns_workspace_bytes() > 0
        gns.gns_release()
        assert gns.gns_workspace_bytes() == 0


def test_threads_that_share_a_stream(gns):
    """The kernels of one call stay together although ctypes lets other threads run."""
    stream = torch.cuda.Stream()
    jobs = [layers(gns, i) for i in range(3)]
    want = [fs[0](x, None) for x, fs in jobs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        x, fs = jobs[i]
        outs = [fs[0](x, stream) for _ in range(60)]
        stream.synchronize()
        bad.extend(i for o in outs if not torch.equal(o, want[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert bad == []
