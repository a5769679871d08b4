// ns_span_api.cu -- C ABI of the span attention, cache read-back, draft
// verification, rotary append and 4-bit cache calls: argument checks and dispatch.
#include <cmath>

#include "ns_common.cuh"
#include "ns_internal.h"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool block_size_ok(int bs) { return bs == 4 || bs == 8 || bs == 16 || bs == 32; }

// The current device's status word, or nullptr (then NS_ERR_CUDA).
unsigned *current_status()
{
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess ? ns::device_status_word(dev) : nullptr;
}

ns_status check_heads(int num_q_heads, int num_kv_heads, ns_dtype dtype)
{
    if (num_q_heads <= 0 || num_kv_heads <= 0)
        return NS_ERR_INVALID_ARG;
    if (dtype != NS_F16 && dtype != NS_BF16)
        return NS_ERR_UNSUPPORTED;
    if (num_q_heads % num_kv_heads != 0 || num_q_heads / num_kv_heads > ns::kMaxSpanGroup)
        return NS_ERR_UNSUPPORTED;
    return NS_OK;
}

// Rows `width` elements wide, `stride` apart: 16-byte aligned, and within the
// 2^40 bytes a tensor map's stride may have.
bool stride_ok(int64_t stride, int64_t width)
{
    return stride >= width && stride % 8 == 0 && stride < (int64_t(1) << 38);
}

ns_status done(cudaError_t e) { return e == cudaSuccess ? NS_OK : NS_ERR_CUDA; }

ns_status gather(const ns::GatherArgs &in, int pool, ns_stream_t stream)
{
    ns::GatherArgs a = in;
    if (a.num_seqs < 0 || a.total_tokens < 0 || a.num_kv_heads <= 0 || a.num_blocks < 1 || a.max_blocks_per_seq < 1)
        return NS_ERR_INVALID_ARG;
    if (a.dtype != NS_F16 && a.dtype != NS_BF16)
        return NS_ERR_UNSUPPORTED;
    if ((a.head_dim != 64 && a.head_dim != 128) || !block_size_ok(a.block_size))
        return NS_ERR_UNSUPPORTED;
    if (a.head_dim == 128 && (pool == 8 || a.block_size != 16))
        return NS_ERR_UNSUPPORTED;
    if (a.num_seqs == 0 || a.total_tokens == 0)
        return NS_OK;
    if (!a.k || !a.v || !a.block_tables || !a.start_loc || !a.k_out || !a.v_out || (pool != 16 && (!a.k_scales || !a.v_scales)))
        return NS_ERR_INVALID_ARG;
    if (!aligned16(a.k) || !aligned16(a.v) || !aligned16(a.k_out) || !aligned16(a.v_out) || !aligned16(a.k_scales) ||
        !aligned16(a.v_scales))
        return NS_ERR_INVALID_ARG;
    a.status = current_status();
    if (a.status == nullptr)
        return NS_ERR_CUDA;
    return done(ns::launch_kv_gather(a, pool, reinterpret_cast<cudaStream_t>(stream)));
}

// Attention of query spans over a pool of 8- or 4-bit codes.
ns_status prefill_paged(const void *q, const int32_t *query_start_loc, const void *k_codes,
                        const void *k_scales, const void *v_codes, const void *v_scales,
                        const int32_t *block_tables, const int32_t *context_lens, int num_seqs,
                        int total_q_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                        int block_size, float scale, void *out, ns_stream_t stream,
                        int max_blocks_per_seq, int64_t num_blocks, ns_dtype dtype, void *workspace,
                        size_t workspace_bytes, int pool)
{
    if (num_seqs < 0 || total_q_tokens < 0)
        return NS_ERR_INVALID_ARG;
    const ns_status s = check_heads(num_q_heads, num_kv_heads, dtype);
    if (s != NS_OK)
        return s;
    if (block_size != 16 || (head_dim != 64 && (pool != 4 || head_dim != 128)))
        return NS_ERR_UNSUPPORTED;
    if (max_blocks_per_seq < 1 || num_blocks < 1 || !std::isfinite(scale))
        return NS_ERR_INVALID_ARG;
    if ((long long)max_blocks_per_seq * block_size > 0x7fffffffLL - 1024)  // positions are 32-bit
        return NS_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_q_tokens == 0)
        return NS_OK;
    if (!q || !query_start_loc || !k_codes || !k_scales || !v_codes || !v_scales || !block_tables || !context_lens ||
        !out || !workspace)
        return NS_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_codes) || !aligned16(k_scales) || !aligned16(v_codes) || !aligned16(v_scales) ||
        !aligned16(out) || !aligned16(workspace) || workspace_bytes < ns_span_attn_workspace_bytes(head_dim))
        return NS_ERR_INVALID_ARG;
    ns::SpanAttnArgs a = {};
    a.status = current_status();
    if (a.status == nullptr)
        return NS_ERR_CUDA;
    a.q = q;
    a.query_start_loc = query_start_loc;
    a.num_seqs = num_seqs;
    a.total_q_tokens = total_q_tokens;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.q_row_stride = (long long)num_q_heads * head_dim;
    a.scale = scale;
    a.out = out;
    a.dtype = dtype;
    a.workspace = workspace;
    a.k_codes = k_codes;
    a.k_scales = k_scales;
    a.v_codes = v_codes;
    a.v_scales = v_scales;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    return done(ns::launch_span_attn(a, pool, reinterpret_cast<cudaStream_t>(stream)));
}

constexpr int64_t kMaxRow = int64_t(1) << 30;  // elements of a token's row: offsets within it are 32-bit

// What every append of this file asks of its arguments; NS_OK with no tokens too, then
// without a look at the pointers.
ns_status check_append(const ns::RopeAppendArgs &a, int pool)
{
    if (a.num_tokens < 0 || a.num_kv_heads <= 0 || a.num_blocks < 1)
        return NS_ERR_INVALID_ARG;
    if (a.dtype != NS_F16 && a.dtype != NS_BF16)
        return NS_ERR_UNSUPPORTED;
    if ((a.head_dim != 64 && a.head_dim != 128) || !block_size_ok(a.block_size))
        return NS_ERR_UNSUPPORTED;
    if (a.head_dim == 128 && (pool == 8 || a.block_size != 16))
        return NS_ERR_UNSUPPORTED;
    if ((int64_t)a.num_kv_heads * a.head_dim > kMaxRow || (int64_t)a.num_q_heads * a.head_dim > kMaxRow)
        return NS_ERR_UNSUPPORTED;
    if (a.num_tokens == 0)
        return NS_OK;
    if (!a.k || !a.v || !a.slot_mapping || !a.k_pool || !a.v_pool || (pool != 16 && (!a.k_scales || !a.v_scales)))
        return NS_ERR_INVALID_ARG;
    if (!aligned16(a.k) || !aligned16(a.v) || !aligned16(a.k_pool) || !aligned16(a.v_pool) || !aligned16(a.k_scales) ||
        !aligned16(a.v_scales))
        return NS_ERR_INVALID_ARG;
    return NS_OK;
}

ns_status append(ns::RopeAppendArgs a, int pool, ns_stream_t stream)
{
    a.status = current_status();
    if (a.status == nullptr)
        return NS_ERR_CUDA;
    return done(ns::launch_rope_append(a, pool, reinterpret_cast<cudaStream_t>(stream)));
}

ns_status rope_append(const ns::RopeAppendArgs &a, int pool, ns_stream_t stream)
{
    if (a.num_q_heads <= 0 || a.max_positions < 1)
        return NS_ERR_INVALID_ARG;
    const ns_status s = check_append(a, pool);
    if (s != NS_OK)
        return s;
    if (a.rotary_dim < 16 || a.rotary_dim > a.head_dim || a.rotary_dim % 16 != 0)
        return NS_ERR_UNSUPPORTED;
    const int64_t q_width = (int64_t)a.num_q_heads * a.head_dim, kv_width = (int64_t)a.num_kv_heads * a.head_dim;
    if (!stride_ok(a.q_stride, q_width) || !stride_ok(a.k_stride, kv_width) || !stride_ok(a.v_stride, kv_width) ||
        !stride_ok(a.q_out_stride, q_width) || (a.k_out && !stride_ok(a.k_out_stride, kv_width)))
        return NS_ERR_INVALID_ARG;
    if (a.num_tokens == 0)
        return NS_OK;
    if (!a.q || !a.positions || !a.cos_sin || !a.q_out)
        return NS_ERR_INVALID_ARG;
    if (!aligned16(a.q) || !aligned16(a.cos_sin) || !aligned16(a.q_out) || !aligned16(a.k_out))
        return NS_ERR_INVALID_ARG;
    return append(a, pool, stream);
}

}  // namespace

extern "C" {

size_t ns_span_attn_workspace_bytes(int head_dim)
{
    return head_dim == 64 || head_dim == 128 ? ns::span_attn_workspace_bytes(head_dim) : 0;
}

ns_status ns_prompt_attn(const void *q, const void *k, const void *v, const int32_t *query_start_loc,
                         const int32_t *key_start_loc, int num_seqs, int total_q_tokens, int total_k_tokens,
                         int num_q_heads, int num_kv_heads, int head_dim, int64_t q_row_stride,
                         int64_t k_row_stride, int64_t v_row_stride, float scale, void *out, ns_stream_t stream,
                         ns_dtype dtype, void *workspace, size_t workspace_bytes)
{
    if (num_seqs < 0 || total_q_tokens < 0 || total_k_tokens < 0)
        return NS_ERR_INVALID_ARG;
    const ns_status s = check_heads(num_q_heads, num_kv_heads, dtype);
    if (s != NS_OK)
        return s;
    if (head_dim != 64 && head_dim != 128)
        return NS_ERR_UNSUPPORTED;
    if (!std::isfinite(scale) || (!key_start_loc && total_k_tokens != total_q_tokens))
        return NS_ERR_INVALID_ARG;
    if (!stride_ok(q_row_stride, (int64_t)num_q_heads * head_dim) ||
        !stride_ok(k_row_stride, (int64_t)num_kv_heads * head_dim) ||
        !stride_ok(v_row_stride, (int64_t)num_kv_heads * head_dim))
        return NS_ERR_INVALID_ARG;
    if (num_seqs == 0 || total_q_tokens == 0)
        return NS_OK;
    // without a single key, k and v may be empty tensors
    if (!q || !query_start_loc || !out || !workspace || (total_k_tokens > 0 && (!k || !v)))
        return NS_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(workspace) ||
        workspace_bytes < ns_span_attn_workspace_bytes(head_dim))
        return NS_ERR_INVALID_ARG;
    ns::SpanAttnArgs a = {};
    a.status = current_status();
    if (a.status == nullptr)
        return NS_ERR_CUDA;
    a.q = q;
    a.query_start_loc = query_start_loc;
    a.num_seqs = num_seqs;
    a.total_q_tokens = total_q_tokens;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.q_row_stride = q_row_stride;
    a.scale = scale;
    a.out = out;
    a.dtype = dtype;
    a.workspace = workspace;
    a.k = k;
    a.v = v;
    a.key_start_loc = key_start_loc ? key_start_loc : query_start_loc;
    a.total_k_tokens = total_k_tokens;
    a.k_row_stride = k_row_stride;
    a.v_row_stride = v_row_stride;
    return done(ns::launch_span_attn(a, 0, reinterpret_cast<cudaStream_t>(stream)));
}

ns_status ns_paged_attn_prefill_q8_0(const void *q, const int32_t *query_start_loc, const void *k_codes,
                                     const void *k_scales, const void *v_codes, const void *v_scales,
                                     const int32_t *block_tables, const int32_t *context_lens, int num_seqs,
                                     int total_q_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                     int block_size, float scale, void *out, ns_stream_t stream,
                                     int max_blocks_per_seq, int64_t num_blocks, ns_dtype dtype, void *workspace,
                                     size_t workspace_bytes)
{
    return prefill_paged(q, query_start_loc, k_codes, k_scales, v_codes, v_scales, block_tables, context_lens, num_seqs,
                         total_q_tokens, num_q_heads, num_kv_heads, head_dim, block_size, scale, out, stream,
                         max_blocks_per_seq, num_blocks, dtype, workspace, workspace_bytes, 8);
}

ns_status ns_paged_attn_prefill_q4_0(const void *q, const int32_t *query_start_loc, const void *k_codes,
                                     const void *k_scales, const void *v_codes, const void *v_scales,
                                     const int32_t *block_tables, const int32_t *context_lens, int num_seqs,
                                     int total_q_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                     int block_size, float scale, void *out, ns_stream_t stream,
                                     int max_blocks_per_seq, int64_t num_blocks, ns_dtype dtype, void *workspace,
                                     size_t workspace_bytes)
{
    return prefill_paged(q, query_start_loc, k_codes, k_scales, v_codes, v_scales, block_tables, context_lens, num_seqs,
                         total_q_tokens, num_q_heads, num_kv_heads, head_dim, block_size, scale, out, stream,
                         max_blocks_per_seq, num_blocks, dtype, workspace, workspace_bytes, 4);
}

ns_status ns_kv_gather(const void *k_pool, const void *v_pool, const int32_t *block_tables, const int32_t *start_loc,
                       int num_seqs, int total_tokens, int num_kv_heads, int head_dim, int block_size, void *k_out,
                       void *v_out, ns_stream_t stream, int max_blocks_per_seq, int64_t num_blocks, ns_dtype dtype)
{
    return gather({k_pool, v_pool, nullptr, nullptr, block_tables, start_loc, num_seqs, total_tokens, num_kv_heads,
                   head_dim, block_size, max_blocks_per_seq, num_blocks, k_out, v_out, dtype, nullptr},
                  16, stream);
}

ns_status ns_kv_gather_q8_0(const void *k_codes, const void *k_scales, const void *v_codes, const void *v_scales,
                            const int32_t *block_tables, const int32_t *start_loc, int num_seqs, int total_tokens,
                            int num_kv_heads, int head_dim, int block_size, void *k_out, void *v_out,
                            ns_stream_t stream, int max_blocks_per_seq, int64_t num_blocks, ns_dtype dtype)
{
    return gather({k_codes, v_codes, k_scales, v_scales, block_tables, start_loc, num_seqs, total_tokens, num_kv_heads,
                   head_dim, block_size, max_blocks_per_seq, num_blocks, k_out, v_out, dtype, nullptr},
                  8, stream);
}

ns_status ns_kv_gather_q4_0(const void *k_codes, const void *k_scales, const void *v_codes, const void *v_scales,
                            const int32_t *block_tables, const int32_t *start_loc, int num_seqs, int total_tokens,
                            int num_kv_heads, int head_dim, int block_size, void *k_out, void *v_out,
                            ns_stream_t stream, int max_blocks_per_seq, int64_t num_blocks, ns_dtype dtype)
{
    return gather({k_codes, v_codes, k_scales, v_scales, block_tables, start_loc, num_seqs, total_tokens, num_kv_heads,
                   head_dim, block_size, max_blocks_per_seq, num_blocks, k_out, v_out, dtype, nullptr},
                  4, stream);
}

ns_status ns_kv_append_q4_0(const void *k, const void *v, const int64_t *slot_mapping, void *k_codes, void *k_scales,
                            void *v_codes, void *v_scales, int num_tokens, int num_kv_heads, int head_dim,
                            int block_size, int64_t num_blocks, ns_dtype dtype, ns_stream_t stream)
{
    ns::RopeAppendArgs a = {};
    a.k = k, a.v = v, a.slot_mapping = slot_mapping;
    a.k_pool = k_codes, a.v_pool = v_codes, a.k_scales = k_scales, a.v_scales = v_scales;
    a.num_tokens = num_tokens, a.num_kv_heads = num_kv_heads, a.head_dim = head_dim, a.block_size = block_size;
    a.k_stride = a.v_stride = (long long)num_kv_heads * head_dim;
    a.num_blocks = num_blocks, a.dtype = dtype;
    const ns_status s = check_append(a, 4);
    return s != NS_OK || num_tokens == 0 ? s : append(a, 4, stream);
}

ns_status ns_rope_kv_append(const void *q, const void *k, const void *v, const int32_t *positions, const float *cos_sin,
                            const int64_t *slot_mapping, void *q_out, void *k_out, void *k_pool, void *v_pool,
                            int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim,
                            int interleaved, int max_positions, int64_t q_row_stride, int64_t k_row_stride,
                            int64_t v_row_stride, int64_t q_out_row_stride, int64_t k_out_row_stride, int block_size,
                            int64_t num_blocks, ns_dtype dtype, ns_stream_t stream)
{
    return rope_append({q, k, v, positions, cos_sin, slot_mapping, q_out, k_out, k_pool, v_pool, nullptr, nullptr,
                        num_tokens, num_q_heads, num_kv_heads, head_dim, rotary_dim, interleaved, max_positions,
                        block_size, q_row_stride, k_row_stride, v_row_stride, q_out_row_stride, k_out_row_stride,
                        num_blocks, dtype, nullptr},
                       16, stream);
}

ns_status ns_rope_kv_append_q8_0(const void *q, const void *k, const void *v, const int32_t *positions,
                                 const float *cos_sin, const int64_t *slot_mapping, void *q_out, void *k_out,
                                 void *k_codes, void *k_scales, void *v_codes, void *v_scales, int num_tokens,
                                 int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim, int interleaved,
                                 int max_positions, int64_t q_row_stride, int64_t k_row_stride, int64_t v_row_stride,
                                 int64_t q_out_row_stride, int64_t k_out_row_stride, int block_size, int64_t num_blocks,
                                 ns_dtype dtype, ns_stream_t stream)
{
    return rope_append({q, k, v, positions, cos_sin, slot_mapping, q_out, k_out, k_codes, v_codes, k_scales, v_scales,
                        num_tokens, num_q_heads, num_kv_heads, head_dim, rotary_dim, interleaved, max_positions,
                        block_size, q_row_stride, k_row_stride, v_row_stride, q_out_row_stride, k_out_row_stride,
                        num_blocks, dtype, nullptr},
                       8, stream);
}

ns_status ns_rope_kv_append_q4_0(const void *q, const void *k, const void *v, const int32_t *positions,
                                 const float *cos_sin, const int64_t *slot_mapping, void *q_out, void *k_out,
                                 void *k_codes, void *k_scales, void *v_codes, void *v_scales, int num_tokens,
                                 int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim, int interleaved,
                                 int max_positions, int64_t q_row_stride, int64_t k_row_stride, int64_t v_row_stride,
                                 int64_t q_out_row_stride, int64_t k_out_row_stride, int block_size, int64_t num_blocks,
                                 ns_dtype dtype, ns_stream_t stream)
{
    return rope_append({q, k, v, positions, cos_sin, slot_mapping, q_out, k_out, k_codes, v_codes, k_scales, v_scales,
                        num_tokens, num_q_heads, num_kv_heads, head_dim, rotary_dim, interleaved, max_positions,
                        block_size, q_row_stride, k_row_stride, v_row_stride, q_out_row_stride, k_out_row_stride,
                        num_blocks, dtype, nullptr},
                       4, stream);
}

ns_status ns_verify_drafts(const float *target_probs, const float *draft_probs, const int32_t *draft_tokens,
                           const int32_t *draft_start_loc, const float *accept_uniforms, const float *sample_uniforms,
                           int num_seqs, int total_drafts, int vocab_size, int64_t target_row_stride,
                           int64_t draft_row_stride, int32_t *out_tokens, int32_t *num_accepted, ns_stream_t stream)
{
    if (num_seqs < 0 || total_drafts < 0 || vocab_size < 1 || (long long)num_seqs + total_drafts > 0x7fffffffLL)
        return NS_ERR_INVALID_ARG;
    if (vocab_size > (1 << 30))  // sums of positions are 32-bit
        return NS_ERR_UNSUPPORTED;
    if (target_row_stride < vocab_size || (draft_probs && draft_row_stride < vocab_size))
        return NS_ERR_INVALID_ARG;
    if (num_seqs == 0)
        return NS_OK;
    if (!target_probs || !draft_start_loc || !sample_uniforms || !out_tokens || !num_accepted ||
        (total_drafts > 0 && (!draft_tokens || !accept_uniforms)))
        return NS_ERR_INVALID_ARG;
    if (!aligned16(target_probs) || !aligned16(draft_probs))
        return NS_ERR_INVALID_ARG;
    ns::VerifyArgs a = {target_probs, draft_probs, draft_tokens, draft_start_loc, accept_uniforms, sample_uniforms,
                        num_seqs, total_drafts, vocab_size, target_row_stride, draft_row_stride, out_tokens,
                        num_accepted, current_status()};
    if (a.status == nullptr)
        return NS_ERR_CUDA;
    return done(ns::launch_verify_drafts(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
