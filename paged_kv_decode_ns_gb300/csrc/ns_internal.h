// ns_internal.h -- host-side launchers shared between the C-ABI file and the
// kernel translation units.
#pragma once

#include <cuda_runtime.h>

#include "ns_paged.h"

namespace ns {

cudaError_t launch_kv_append(const void *k, const void *v, const int64_t *slot_mapping, void *k_pool,
                             void *v_pool, int num_tokens, int num_kv_heads, int head_dim, int block_size,
                             long long num_blocks, unsigned *status, cudaStream_t stream);

// q8_0 append: quantise each new token's K/V rows and scatter codes and scales.
cudaError_t launch_kv_append_q8(const void *k, const void *v, const int64_t *slot_mapping, void *k_codes,
                                void *k_scales, void *v_codes, void *v_scales, int num_tokens, int num_kv_heads,
                                int block_size, long long num_blocks, ns_dtype dtype, unsigned *status,
                                cudaStream_t stream);

// Query spans -> per-row table row and key count (prefill through the decode
// walk).  Rows of spans with at least `tc_min_span` tokens (tc_min_span > 0)
// are marked for the tensor-core kernel: table row -1, key count 0.
cudaError_t launch_span_rows(const int32_t *query_start_loc, const int32_t *context_lens,
                             int num_seqs, int total_rows, int tc_min_span, int32_t *row_seq,
                             int32_t *row_len, unsigned *status, cudaStream_t stream);

// Address of the device status word on device `dev` (current), or nullptr.
unsigned *device_status_word(int dev);

struct DecodeParams;

// Launch the split-KV decode kernel with num_ctas CTAs, or with the resident
// CTAs of device `dev` when num_ctas is 0.
ns_status launch_decode(const DecodeParams &P, ns_dtype dtype, int block_size, int num_ctas,
                        cudaStream_t stream, int dev, bool q8 = false, int head_dim = 64);

// Chunked prefill of every span of two or more tokens on the tcgen05 tensor cores.
// after_walk: the kernel just before it on the stream is this call's span walk
// (whose results it does not read), so it may be launched to overlap it.
bool tc_prefill_supported(int block_size, int group);
cudaError_t launch_tc_prefill(const void *q, const int32_t *query_start_loc, const void *k_pool,
                              const void *v_pool, const int32_t *block_tables,
                              const int32_t *context_lens, int num_seqs, int total_q_tokens,
                              int num_q_heads, int num_kv_heads, int block_size, float scale,
                              void *out, int max_blocks_per_seq, long long num_blocks, ns_dtype dtype,
                              int min_span, int head_dim, unsigned *status, bool after_walk,
                              cudaStream_t stream);

// Attention of query spans over contiguous K/V rows (ns_prompt_attn) or a
// q8_0 pool (ns_paged_attn_prefill_q8_0).
struct SpanAttnArgs {
    const void *q;
    const int32_t *query_start_loc;
    int num_seqs, total_q_tokens, num_q_heads, num_kv_heads, head_dim;
    long long q_row_stride;  // elements
    float scale;
    void *out;
    ns_dtype dtype;
    void *workspace;
    unsigned *status;
    // contiguous rows
    const void *k, *v;
    const int32_t *key_start_loc;
    int total_k_tokens;
    long long k_row_stride, v_row_stride;
    // q8_0 pool
    const void *k_codes, *k_scales, *v_codes, *v_scales;
    const int32_t *block_tables, *context_lens;
    int max_blocks_per_seq;
    long long num_blocks;
};
// SMs of the current device (asked for once a device).
cudaError_t current_sms(int *sms);
constexpr int kMaxSpanGroup = 64;  // query heads per kv head
size_t span_attn_workspace_bytes(int head_dim);
cudaError_t launch_span_attn(const SpanAttnArgs &a, bool q8, cudaStream_t stream);

// Pool rows of the sequences start_loc, packed: 16-bit copies or q8_0 values.
struct GatherArgs {
    const void *k, *v;                // 16-bit pools, or codes
    const void *k_scales, *v_scales;  // q8_0 only
    const int32_t *block_tables, *start_loc;
    int num_seqs, total_tokens, num_kv_heads, head_dim, block_size, max_blocks_per_seq;
    long long num_blocks;
    void *k_out, *v_out;
    ns_dtype dtype;
    unsigned *status;
};
cudaError_t launch_kv_gather(const GatherArgs &a, bool q8, cudaStream_t stream);

struct VerifyArgs {
    const float *target, *draft;
    const int32_t *tokens, *start;
    const float *accept_u, *sample_u;
    int num_seqs, total_drafts, vocab;
    long long target_stride, draft_stride;
    int32_t *out_tokens, *num_accepted;
    unsigned *status;
};
cudaError_t launch_verify_drafts(const VerifyArgs &a, cudaStream_t stream);

}  // namespace ns
