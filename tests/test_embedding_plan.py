"""How the embedding's gradient shares out its tokens and its intermediate memory, up
to the most tokens that its entry takes: host arithmetic, asked from the library by a
small program, since none of it needs a GPU (and a wrong size must not meet one)."""
import subprocess

import pytest

from newton_schulz_gram_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "embedding.cuh"
#include "gns.h"
int main(int, char** a) {
    gns::EmbeddingJob j{};
    j.id_bytes = 8;
    j.tokens = std::atoi(a[1]);
    j.vocab = std::atoi(a[2]);
    j.cols = std::atoi(a[3]);
    j.dtype = GNS_BF16;
    j.out_dtype = GNS_FP32;
    j.lddy = j.lddt = j.cols;
    const gns::EmbeddingPlan p = gns::embedding_plan(j, nullptr);
    const auto at = [](const void* v) { return reinterpret_cast<long long>(v); };
    std::printf("%d %d %d %d %lld %lld %lld %lld %lld %lld %lld %lld %lld\n", p.passes, p.bits, p.chunk, p.chunks, at(p.keys[0]), at(p.order[0]),
                at(p.keys[1]), at(p.order[1]), at(p.ready), at(p.marks), at(p.part), (long long)p.cleared, (long long)p.bytes);
}
"""

MOST = (1 << 31) - 1 - 4096


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    lib = build.build()
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(PROGRAM)
    subprocess.run([build.nvcc(), "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, str(at / "plan.cpp"), lib, "-o", str(at / "plan")],
                   check=True, capture_output=True)

    def ask(*sizes):
        r = subprocess.run([str(at / "plan"), *map(str, sizes)], check=True, capture_output=True, text=True)
        return [int(v) for v in r.stdout.split()]

    return ask


@pytest.mark.parametrize("cols", [1, 1000, 4096])
@pytest.mark.parametrize("tokens", [1, 31, 4097, 131072, 131073, (1 << 30) + 7, MOST - (1 << 20), (1 << 31) - (1 << 20),
                                    (1 << 31) - (1 << 20) + 1, MOST])
def test_runs_and_memory(plan, tokens, cols):
    vocab = 50021
    passes, bits, chunk, chunks, *places, part, cleared, size = plan(tokens, vocab, cols)
    assert passes * bits >= 16 and chunks == -(-tokens // chunk)
    assert chunk == 64 or (chunk < 64 and chunks < 8192) or chunks <= 2048
    keys0, order0, keys1, order1, ready, marks = places
    assert keys0 == 0 and min(order0, keys1 - order0, order1 - keys1, ready - order1) >= 4 * tokens
    assert cleared == marks + vocab - ready and marks - ready >= 4 * (chunks // 128 + 1)
    row = 4 * (cols if cols % 8 == 0 else -(-cols // 128) * 128)
    assert part >= marks + vocab and size - part >= (2 * row * chunks if chunks > 1 else 0)
    assert size < 17 * tokens + 2 * row * chunks + vocab + (1 << 20)
