// Launchers of the embedding lookup and the gradient of its table (embedding.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace gns {

struct EmbeddingJob {
    const void* ids;  // [tokens]; one outside 0 .. vocab - 1 has no row
    int id_bytes;     // 4 or 8
    int tokens, vocab, cols;
    float scale;
    const void* table;  // forward: [vocab][ldt] of dtype
    long long ldt;
    void* y;            // forward: [tokens][ldy]
    long long ldy;
    const void* dy;     // backward: [tokens][lddy] of dtype
    long long lddy;
    void* dtable;       // [vocab][lddt] of out_dtype
    long long lddt;
    int dtype, out_dtype;
};

int launch_embedding(const EmbeddingJob& job, cudaStream_t s);

// The backward pass, once `cleared` bytes from `ready` on are set to zero: `passes` times a count (where the plan has one)
// and a placement, then the sums of runs of sorted tokens, then, of several chunks, the
// ids that span them.
struct EmbeddingPlan {
    int passes, bits;      // of the tokens' sort by id; digits of `bits` bits
    bool counts;           // each pass has a counting kernel
    int chunk;             // sorted tokens that a warp sums
    int chunks;
    size_t bytes;          // intermediate memory
    int *keys[2], *order[2], *hist;  // within it; the sort's result in keys[passes & 1]
    unsigned* ready;       // counts of blocks that share a sum
    unsigned char* marks;  // of each row: whether it has a token
    size_t cleared;
    int hosts;             // kernels that share the rows without
    float* part;
};

EmbeddingPlan embedding_plan(const EmbeddingJob& job, char* scratch);
int launch_embedding_count(const EmbeddingJob& job, const EmbeddingPlan& plan, int pass, cudaStream_t s);
int launch_embedding_place(const EmbeddingJob& job, const EmbeddingPlan& plan, int pass, cudaStream_t s);
int launch_embedding_runs(const EmbeddingJob& job, const EmbeddingPlan& plan, cudaStream_t s);
int launch_embedding_joins(const EmbeddingJob& job, const EmbeddingPlan& plan, cudaStream_t s);

}  // namespace gns
