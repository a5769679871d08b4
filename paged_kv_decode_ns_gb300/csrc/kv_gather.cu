// kv_gather.cu -- read sequences back from the pool into packed rows.
//
// k_out[start[s] + p][h][:] = K_s[p][h][:], a copy for 16-bit pools and
// fp16(d) * code rounded once for q8_0 pools.
#include <algorithm>

#include "ns_common.cuh"
#include "ns_internal.h"

namespace ns {

namespace {

constexpr int kThreads = 256;

// The sequence that owns packed row t: the last s with start[s] <= t, when it
// ends behind t; -1 when no sequence does.
__device__ __forceinline__ int owner(const int32_t *start, int num_seqs, int t)
{
    int lo = 0, hi = num_seqs;  // start[lo] <= t < start[hi], once start[0] <= t
    if (*start > t)
        return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    return t < start[lo + 1] ? lo : -1;
}

// Eight codes (x, y) and their scale (z) -> eight elements: fp16(d) * code is exact
// in fp32 and rounds once.
template <typename T>
__device__ __forceinline__ uint4 dequantise(uint4 w)
{
    const float d = __half2float(__ushort_as_half((uint16_t)w.z));
    auto pair = [&](uint32_t x, int i) {
        return pack2<T>(d * (float)(int8_t)(x >> (8 * i)), d * (float)(int8_t)(x >> (8 * i + 8)));
    };
    return make_uint4(pair(w.x, 0), pair(w.x, 2), pair(w.y, 0), pair(w.y, 2));
}

// A CTA copies `tokens` packed rows.  Its first threads look their rows up (owner,
// table entry) once; then a thread moves 16 bytes of K and of V (8 elements) at a
// time, kBatch of them loaded before the first is stored.  Bound by memory once
// the rows fill the GPU: 256 sequences of q8_0 (381 MB) 62.1 us, 6.1 TB/s; 32 of
// 16 bits at head_dim 128 (165 MB) 27.5 us, 6.0 TB/s.  (A thread that looked its own
// row up and divided by the heads for every 16 bytes: 4.1 and 5.0 TB/s.)  Five CTAs an
// SM cap the registers at 48: 66.0 us at four, 90.8 at six, which spills.
constexpr int kBatch = 4;
constexpr int kMaxTokens = 256;

template <typename T, bool Q8>
__global__ void __launch_bounds__(kThreads, 5) kv_gather_kernel(const GatherArgs a, int tokens, int row_chunks, int head_chunks)
{
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ long long src[kMaxTokens];  // first pool row of the token (its kv head 0), or -1
    if (blockIdx.x == 0)  // entries out of order, also those that no row falls between
        for (int s = threadIdx.x; s < a.num_seqs; s += kThreads) {
            const int first = a.start_loc[s], end = a.start_loc[s + 1];
            if (first < 0 || end < first || end > a.total_tokens)
                raise_status(a.status, NS_DEV_BAD_QUERY_SPAN);
        }
    const int t0 = blockIdx.x * tokens, nt = min(tokens, a.total_tokens - t0);
    if ((int)threadIdx.x < nt) {
        const int t = t0 + threadIdx.x;
        long long row = -1;
        const int s = owner(a.start_loc, a.num_seqs, t);
        if (s >= 0) {
            const int first = a.start_loc[s], end = a.start_loc[s + 1], p = t - first;
            if (first < 0 || end > a.total_tokens) {
                // reported above
            } else if ((long long)(end - first) > (long long)a.max_blocks_per_seq * a.block_size) {
                raise_status(a.status, NS_DEV_BAD_CONTEXT_LEN);
            } else {
                const int blk = a.block_tables[(long long)s * a.max_blocks_per_seq + p / a.block_size];
                if (blk < 0 || blk >= a.num_blocks)
                    raise_status(a.status, NS_DEV_BAD_BLOCK_ID);
                else
                    row = (long long)blk * a.num_kv_heads * a.block_size + p % a.block_size;
            }
        }
        src[threadIdx.x] = row;
    }
    __syncthreads();
    const int n = nt * row_chunks;
    const long long out0 = (long long)t0 * row_chunks;
    for (int i0 = threadIdx.x; i0 < n; i0 += kThreads * kBatch) {
        uint4 k[kBatch], v[kBatch];
        bool on[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int i = i0 + b * kThreads;
            const int t = i / row_chunks, c = i - t * row_chunks;
            const int h = c / head_chunks, chunk = c - h * head_chunks;
            const long long row = i < n ? src[t] : -1;
            on[b] = row >= 0;
            if (!on[b])
                continue;
            const long long prow = row + (long long)h * a.block_size;
            if (!Q8) {
                k[b] = static_cast<const uint4 *>(a.k)[prow * head_chunks + chunk];
                v[b] = static_cast<const uint4 *>(a.v)[prow * head_chunks + chunk];
            } else {
                const uint2 kc = static_cast<const uint2 *>(a.k)[prow * 8 + chunk],
                            vc = static_cast<const uint2 *>(a.v)[prow * 8 + chunk];
                k[b] = make_uint4(kc.x, kc.y, static_cast<const uint16_t *>(a.k_scales)[prow * 2 + (chunk >> 2)], 0u);
                v[b] = make_uint4(vc.x, vc.y, static_cast<const uint16_t *>(a.v_scales)[prow * 2 + (chunk >> 2)], 0u);
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (!on[b])
                continue;
            const long long o = out0 + i0 + b * kThreads;
            if (Q8) {
                k[b] = dequantise<T>(k[b]);
                v[b] = dequantise<T>(v[b]);
            }
            static_cast<uint4 *>(a.k_out)[o] = k[b];
            static_cast<uint4 *>(a.v_out)[o] = v[b];
        }
    }
}

}  // namespace

cudaError_t launch_kv_gather(const GatherArgs &a, bool q8, cudaStream_t stream)
{
    const int head_chunks = a.head_dim / 8, row_chunks = a.num_kv_heads * head_chunks;
    // a batch for every thread, two of the smaller reads from q8_0 (71 us with one);
    // at least eight rows, so that the look-ups are shared
    const int tokens = std::min(kMaxTokens, std::max(8, (q8 ? 2 : 1) * kThreads * kBatch / row_chunks));
    const unsigned grid = (unsigned)((a.total_tokens + tokens - 1) / tokens);
    auto kern = !q8 ? kv_gather_kernel<F16, false>
                    : a.dtype == NS_BF16 ? kv_gather_kernel<BF16, true> : kv_gather_kernel<F16, true>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    // its set-up overlaps the end of the kernel before, which it waits for
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, tokens, row_chunks, head_chunks);
}

}  // namespace ns
