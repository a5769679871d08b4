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
    if (__ldg(start) > t)
        return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(start + mid) <= t)
            lo = mid;
        else
            hi = mid;
    }
    return t < __ldg(start + lo + 1) ? lo : -1;
}

// One thread moves 16 bytes of K and 16 of V (8 elements); a row of one head
// is D / 8 threads.
template <typename T, bool Q8>
__global__ void __launch_bounds__(kThreads) kv_gather_kernel(const GatherArgs a, int chunks_per_row, long long n_chunks)
{
    const long long stride = (long long)gridDim.x * kThreads;
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < n_chunks; i += stride) {
        const long long row = i / chunks_per_row;
        const int chunk = (int)(i % chunks_per_row);
        const int t = (int)(row / a.num_kv_heads), h = (int)(row % a.num_kv_heads);
        const int s = owner(a.start_loc, a.num_seqs, t);
        if (s < 0)
            continue;
        const int first = __ldg(a.start_loc + s), end = __ldg(a.start_loc + s + 1);
        const bool lead = t == first && h == 0 && chunk == 0;
        if (first < 0 || end > a.total_tokens) {
            if (lead || (t == 0 && h == 0 && chunk == 0))
                raise_status(a.status, NS_DEV_BAD_QUERY_SPAN);
            continue;
        }
        if ((long long)(end - first) > (long long)a.max_blocks_per_seq * a.block_size) {
            if (lead)
                raise_status(a.status, NS_DEV_BAD_CONTEXT_LEN);
            continue;
        }
        const int p = t - first;
        const int blk = __ldg(a.block_tables + (long long)s * a.max_blocks_per_seq + p / a.block_size);
        if (blk < 0 || blk >= a.num_blocks) {
            if (h == 0 && chunk == 0)
                raise_status(a.status, NS_DEV_BAD_BLOCK_ID);
            continue;
        }
        const long long prow = ((long long)blk * a.num_kv_heads + h) * a.block_size + p % a.block_size;
        uint4 *ko = static_cast<uint4 *>(a.k_out) + i, *vo = static_cast<uint4 *>(a.v_out) + i;
        if (!Q8) {
            *ko = __ldg(static_cast<const uint4 *>(a.k) + prow * chunks_per_row + chunk);
            *vo = __ldg(static_cast<const uint4 *>(a.v) + prow * chunks_per_row + chunk);
        } else {
            auto values = [&](const void *codes, const void *scales) {
                const uint2 c = __ldg(static_cast<const uint2 *>(codes) + prow * chunks_per_row + chunk);
                const float d = __half2float(__ushort_as_half(
                    __ldg(static_cast<const uint16_t *>(scales) + prow * 2 + (chunk >> 2))));
                const int8_t *b = reinterpret_cast<const int8_t *>(&c);
                uint4 w;
                w.x = pack2<T>(d * (float)b[0], d * (float)b[1]);
                w.y = pack2<T>(d * (float)b[2], d * (float)b[3]);
                w.z = pack2<T>(d * (float)b[4], d * (float)b[5]);
                w.w = pack2<T>(d * (float)b[6], d * (float)b[7]);
                return w;
            };
            *ko = values(a.k, a.k_scales);
            *vo = values(a.v, a.v_scales);
        }
    }
}

}  // namespace

cudaError_t launch_kv_gather(const GatherArgs &a, bool q8, cudaStream_t stream)
{
    const int chunks = a.head_dim / 8;
    const long long n = (long long)a.total_tokens * a.num_kv_heads * chunks;
    const unsigned grid = (unsigned)std::min<long long>((n + kThreads - 1) / kThreads, 65535);
    auto kern = !q8 ? kv_gather_kernel<F16, false>
                    : a.dtype == NS_BF16 ? kv_gather_kernel<BF16, true> : kv_gather_kernel<F16, true>;
    kern<<<grid, kThreads, 0, stream>>>(a, chunks, n);
    return cudaGetLastError();
}

}  // namespace ns
