// span_attn.cu -- causal attention of query spans over contiguous K/V rows
// (whole prompts) or a q8_0 paged cache.
//
// Row i of a span of n tokens over L keys sits at position L-n+i and sees the
// keys p <= L-n+i: out = sum_p exp(z_p - m) v_p / sum_p exp(z_p - m), one pass
// over the keys with a running maximum m.
//
// One warp per (query row, query head): 32 keys at a time, lane i scoring key
// i, then every lane accumulating its own D / 32 output elements.
#include "ns_common.cuh"
#include "ns_internal.h"

namespace ns {

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;

template <typename T>
__device__ __forceinline__ float load1(const void *p, long long i)
{
    const uint16_t b = __ldg(static_cast<const uint16_t *>(p) + i);
    if (T::code == NS_BF16)
        return __uint_as_float((uint32_t)b << 16);
    return __half2float(__ushort_as_half(b));
}

template <typename T, bool Q8, int D>
__global__ void __launch_bounds__(kThreads) span_attn_kernel(const SpanAttnArgs a)
{
    __shared__ float sq[kWarps][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * kWarps + warp;
    const int t = (int)(unit / a.num_q_heads), j = (int)(unit % a.num_q_heads);
    if (t >= a.total_q_tokens)
        return;
    if (unit == 0)  // a sequence without rows of its own is looked at too
        for (int i = lane; i < a.num_seqs; i += 32)
            if (__ldg(a.query_start_loc + i + 1) < __ldg(a.query_start_loc + i))
                raise_status(a.status, NS_DEV_BAD_QUERY_SPAN);
    // the sequence that owns row t
    const int32_t *start = a.query_start_loc;
    if (__ldg(start) > t)
        return;
    int s = 0, hi = a.num_seqs;
    while (hi - s > 1) {
        const int mid = (s + hi) >> 1;
        if (__ldg(start + mid) <= t)
            s = mid;
        else
            hi = mid;
    }
    const int q0 = __ldg(start + s), q1 = __ldg(start + s + 1);
    if (t >= q1)
        return;
    const int n = q1 - q0;
    int L;
    long long k0 = 0;
    unsigned bad = q0 < 0 || q1 > a.total_q_tokens ? NS_DEV_BAD_QUERY_SPAN : 0u;
    if (Q8) {
        L = __ldg(a.context_lens + s);
        if (L < n)
            bad = NS_DEV_BAD_QUERY_SPAN;
        else if ((long long)L > (long long)a.max_blocks_per_seq * 16)
            bad = NS_DEV_BAD_CONTEXT_LEN;
    } else {
        const int a0 = __ldg(a.key_start_loc + s), a1 = __ldg(a.key_start_loc + s + 1);
        if (a0 < 0 || a1 < a0 || a1 > a.total_k_tokens)
            bad = NS_DEV_BAD_QUERY_SPAN;
        k0 = a0;
        L = a1 - a0;
    }
    if (bad != 0) {
        if (lane == 0)
            raise_status(a.status, bad);
        return;
    }
    const int keys = min(L, L - n + (t - q0) + 1);
    const int h = j / (a.num_q_heads / a.num_kv_heads);
    const float scale = a.scale * 1.4426950408889634f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e)
        sq[warp][e * 32 + lane] = load1<T>(a.q, t * a.q_row_stride + (long long)j * D + e * 32 + lane);
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[D / 32] = {};
    for (int p0 = 0; p0 < keys; p0 += 32) {
        const int p = p0 + lane;
        bool on = p < keys;
        long long row = 0;
        if (Q8) {
            const int blk = on ? __ldg(a.block_tables + (long long)s * a.max_blocks_per_seq + p / 16) : 0;
            if (on && (blk < 0 || blk >= a.num_blocks)) {
                raise_status(a.status, NS_DEV_BAD_BLOCK_ID);
                on = false;
            }
            row = ((long long)blk * a.num_kv_heads + h) * 16 + p % 16;
        } else {
            row = k0 + p;
        }
        float z = -INFINITY;
        if (on) {
            float acc = 0.f;
#pragma unroll
            for (int b = 0; b < D / 32; ++b) {
                float part = 0.f;
                for (int e = 0; e < 32; ++e) {
                    const float kv = Q8 ? (float)__ldg(static_cast<const int8_t *>(a.k_codes) + row * D + b * 32 + e)
                                        : load1<T>(a.k, row * a.k_row_stride + (long long)h * D + b * 32 + e);
                    part = fmaf(sq[warp][b * 32 + e], kv, part);
                }
                acc += Q8 ? part * load1<F16>(a.k_scales, row * 2 + b) : part;
            }
            z = acc * scale;
        }
        float top = z;
#pragma unroll
        for (int x = 16; x; x >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float m_new = fmaxf(m, top);
        if (m_new == -INFINITY)
            continue;
        const float alpha = fast_exp2(m - m_new);
        const float w = on ? fast_exp2(z - m_new) : 0.f;
        m = m_new;
        float sum = w;
#pragma unroll
        for (int x = 16; x; x >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, x);
        l = l * alpha + sum;
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
            o[e] *= alpha;
        const unsigned live = __ballot_sync(0xffffffffu, on);
        for (int i = 0; i < 32; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, i);
            const long long ri = __shfl_sync(0xffffffffu, row, i);
            if (!((live >> i) & 1u))
                continue;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                const float v = Q8 ? (float)__ldg(static_cast<const int8_t *>(a.v_codes) + ri * D + e * 32 + lane) *
                                         load1<F16>(a.v_scales, ri * 2 + e)
                                   : load1<T>(a.v, ri * a.v_row_stride + (long long)h * D + e * 32 + lane);
                o[e] = fmaf(wi, v, o[e]);
            }
        }
    }
    uint16_t *out = static_cast<uint16_t *>(a.out) + ((long long)t * a.num_q_heads + j) * D;
#pragma unroll
    for (int e = 0; e < D / 32; ++e)
        out[e * 32 + lane] = pack1<T>(l > 0.f ? o[e] / l : 0.f);
}

}  // namespace

size_t span_attn_workspace_bytes(int head_dim) { return head_dim == 64 ? 256 : 512; }

cudaError_t launch_span_attn(const SpanAttnArgs &a, bool q8, cudaStream_t stream)
{
    const long long units = (long long)a.total_q_tokens * a.num_q_heads;
    const unsigned grid = (unsigned)((units + kWarps - 1) / kWarps);
    const bool bf = a.dtype == NS_BF16;
    auto kern = q8 ? (bf ? span_attn_kernel<BF16, true, 64> : span_attn_kernel<F16, true, 64>)
                : a.head_dim == 64 ? (bf ? span_attn_kernel<BF16, false, 64> : span_attn_kernel<F16, false, 64>)
                                   : (bf ? span_attn_kernel<BF16, false, 128> : span_attn_kernel<F16, false, 128>);
    kern<<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace ns
