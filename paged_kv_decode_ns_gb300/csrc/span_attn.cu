// span_attn.cu -- host side of the span attention: tensor maps, workspace and
// dispatch (the kernels are in span_attn.cuh).
#include "span_attn.cuh"

#include <atomic>
#include <cmath>

namespace ns {

// Headers of the CTAs, then two records for each.
size_t span_attn_workspace_bytes(int head_dim)
{
    return span::header_bytes() + 2 * span::kMaxCtas * span::record_floats(head_dim) * sizeof(float);
}

cudaError_t current_sms(int *sms)
{
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    *sms = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (*sms != 0)
        return cudaSuccess;
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && dev < 64)
        known[dev].store(*sms, std::memory_order_relaxed);
    return e;
}

cudaError_t launch_span_attn(const SpanAttnArgs &a, bool q8, cudaStream_t stream)
{
    int sms = 0;
    const cudaError_t e = current_sms(&sms);
    if (e != cudaSuccess)
        return e;
    span::Params P;
    P.a = a;
    P.group = a.num_q_heads / a.num_kv_heads;
    P.qt = span::kRows / P.group;
    P.scale_log2 = std::max(std::fabs(a.scale) * 1.4426950408889634f, span::kTinyScale);
    P.negate = a.scale < 0.f;
    P.headers = static_cast<span::Header *>(a.workspace);
    P.records = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + span::header_bytes());
    span::Maps tm = {};
    if (span::q_by_tma(a.head_dim, a.dtype == NS_BF16)) {
        // Q: [token][head][element], boxes of a group's heads of a query tile's tokens
        const cuuint64_t dims[3] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.num_q_heads, (cuuint64_t)a.total_q_tokens};
        const cuuint64_t strides[2] = {(cuuint64_t)a.head_dim * 2, (cuuint64_t)a.q_row_stride * 2};
        const cuuint32_t box[3] = {64u, (cuuint32_t)P.group, (cuuint32_t)P.qt};
        if (!encode_tensor_map(&tm.q, a.dtype, 3, a.q, dims, strides, box))
            return cudaErrorInvalidValue;
    }
    if (!q8) {
        // K, V: [token][kv head][element], boxes of one head's 64 elements of a tile of
        // tokens; without a single key nothing is ever copied
        const int kt = a.head_dim == 64 ? span::Geo<64, false>::KT : span::Geo<128, false>::KT;
        const cuuint64_t dims[3] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.num_kv_heads,
                                    (cuuint64_t)std::max(a.total_k_tokens, 1)};
        const cuuint32_t box[3] = {64u, 1u, (cuuint32_t)kt};
        const void *src[2] = {a.total_k_tokens ? a.k : a.q, a.total_k_tokens ? a.v : a.q};
        const long long stride[2] = {a.k_row_stride, a.v_row_stride};
        for (int i = 0; i < 2; ++i) {
            const cuuint64_t strides[2] = {(cuuint64_t)a.head_dim * 2, (cuuint64_t)stride[i] * 2};
            if (!encode_tensor_map(i == 0 ? &tm.k : &tm.v, a.dtype, 3, src[i], dims, strides, box))
                return cudaErrorInvalidValue;
        }
    }
    const int ctas = std::min(sms, span::kMaxCtas);
    const bool bf16 = a.dtype == NS_BF16;
    if (q8)
        return launch_span_q8(bf16, tm, P, ctas, stream);
    return a.head_dim == 64 ? launch_span_d64(bf16, tm, P, ctas, stream)
                            : launch_span_d128(bf16, tm, P, ctas, stream);
}

}  // namespace ns
