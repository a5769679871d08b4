// q4_decode.h -- arguments of the decode over a q4_0 pool (decode_q4.cu).
#pragma once

#include <cuda_runtime.h>

#include "ns_paged.h"

namespace ns {

constexpr int kMaxQ4Ctas = 160;  // grid, at most: two records of the workspace for each

struct Q4DecodeArgs {
    const void *q, *k_codes, *k_scales, *v_codes, *v_scales;
    const int32_t *block_tables, *context_lens;
    int num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq;
    long long num_blocks;
    float scale;
    void *out;
    ns_dtype dtype;
    int *counters;   // one a (sequence, kv head, 8 query heads), zero between calls
    float *records;
    unsigned *status;
};
// The line of work of the largest call of these sizes has 32-bit positions.
bool q4_decode_fits(long long num_seqs, long long pairs, long long max_blocks, int block_size);
cudaError_t launch_decode_q4(const Q4DecodeArgs &a, cudaStream_t stream);

}  // namespace ns
