// rope_append.cu -- new tokens' rows into the cache, their queries and keys turned by
// their positions on the way.
//
// A pair (x, y) of a row's elements becomes (x c - y s, y c + x s) with the position's
// cosine and sine of that pair; elements behind rotary_dim and values pass.  The products
// and the sum are rounded to fp32 one by one (no contraction), so that the codes of the 8-
// and 4-bit pools, which are decided from those fp32 values, are determined to the bit.
//
// A warp takes one token, or a part of its rows: 8 elements a lane, 8 or 16 lanes a head row,
// so that the other half of a pair is in a neighbouring lane and a group of 32 elements in
// four of them.  The position's cosines and sines are read once and stay in 16 registers for
// all of the token's heads.  Every lane reads and writes only its own 8 elements (the other
// half of the pairs comes by shuffle), so rows may be turned in place.
#include <algorithm>

#include "ns_internal.h"
#include "quantise.cuh"

namespace ns {

namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 4;  // rows of a lane in flight

template <typename T, int D, int POOL, bool ROPE>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeAppendArgs a, int parts, int part_rows)
{
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int C = D / 8, ROWS = 32 / C;  // lanes of a row, rows of a warp at a time
    const int lane = threadIdx.x & 31, c = lane % C, sub = lane / C;
    const long long item = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const long long t = item / parts;
    const int part = (int)(item - t * parts);
    if (t >= a.num_tokens)
        return;
    const long long slot = a.slot_mapping[t];
    if (slot < 0)
        return;
    const int pos = ROPE ? a.positions[t] : 0;
    const bool bad_slot = slot >= a.num_blocks * a.block_size, bad_pos = ROPE && (pos < 0 || pos >= a.max_positions);
    if (bad_slot || bad_pos) {
        if (part == 0 && lane == 0)
            raise_status(a.status, (bad_slot ? NS_DEV_BAD_SLOT : 0u) | (bad_pos ? NS_DEV_BAD_POSITION : 0u));
        return;
    }
    const long long blk = slot / a.block_size;
    const int off = (int)(slot - blk * a.block_size);

    // this lane's cosines and sines (of the pair's lower element negative), and the lane
    // that holds the other elements of its pairs
    float co[8], si[8];
    const int half = a.rotary_dim / 2, hc = half / 8;  // elements, lanes (halves)
    const bool turned = ROPE && c < 2 * hc;
    const bool pairs = ROPE && a.interleaved;
    int other = lane;
    if (turned) {
        const float *row = a.cos_sin + (long long)pos * a.rotary_dim;
        if (!pairs) {
            const bool low = c < hc;
            other = low ? lane + hc : lane - hc;
            const float *at = row + (low ? c : c - hc) * 8;
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(at + i), y = *reinterpret_cast<const float4 *>(at + half + i);
                co[i] = x.x, co[i + 1] = x.y, co[i + 2] = x.z, co[i + 3] = x.w;
                si[i] = low ? -y.x : y.x, si[i + 1] = low ? -y.y : y.y, si[i + 2] = low ? -y.z : y.z,
                si[i + 3] = low ? -y.w : y.w;
            }
        } else {
            const float4 x = *reinterpret_cast<const float4 *>(row + c * 4), y = *reinterpret_cast<const float4 *>(row + half + c * 4);
            co[0] = co[1] = x.x, co[2] = co[3] = x.y, co[4] = co[5] = x.z, co[6] = co[7] = x.w;
            si[1] = y.x, si[3] = y.y, si[5] = y.z, si[7] = y.w;
            si[0] = -y.x, si[2] = -y.y, si[4] = -y.z, si[6] = -y.w;
        }
    }

    // rows of the token: queries, keys, values
    const int hq = ROPE ? a.num_q_heads : 0, hkv = a.num_kv_heads, rows = hq + 2 * hkv;
    const int first = part * part_rows, last = min(rows, first + part_rows);
    for (int r0 = first; r0 < last; r0 += ROWS * kBatch) {
        uint4 w[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int r = r0 + b * ROWS + sub;
            w[b] = make_uint4(0u, 0u, 0u, 0u);
            if (r < last) {
                const bool is_q = r < hq, is_k = r < hq + hkv;
                const char *src = static_cast<const char *>(is_q ? a.q : is_k ? a.k : a.v);
                const long long row = t * (is_q ? a.q_stride : is_k ? a.k_stride : a.v_stride);
                const int h = is_q ? r : is_k ? r - hq : r - hq - hkv;
                w[b] = *reinterpret_cast<const uint4 *>(src + (row + (long long)h * D + c * 8) * 2);
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int top = r0 + b * ROWS;  // the warp's first row: the same in all lanes
            if (top >= last)
                break;
            const int r = top + sub;
            const bool on = r < last, is_q = r < hq, is_v = r >= hq + hkv;
            float x[8];
            {
                const float2 p0 = unpack2<T>(w[b].x), p1 = unpack2<T>(w[b].y), p2 = unpack2<T>(w[b].z), p3 = unpack2<T>(w[b].w);
                x[0] = p0.x, x[1] = p0.y, x[2] = p1.x, x[3] = p1.y, x[4] = p2.x, x[5] = p2.y, x[6] = p3.x, x[7] = p3.y;
            }
            if (ROPE && top < hq + hkv) {
                uint4 o;
                if (pairs) {  // the other element of a pair is in the same word
                    o = make_uint4(__byte_perm(w[b].x, 0u, 0x1032), __byte_perm(w[b].y, 0u, 0x1032),
                                   __byte_perm(w[b].z, 0u, 0x1032), __byte_perm(w[b].w, 0u, 0x1032));
                } else {
                    o.x = __shfl_sync(0xffffffffu, w[b].x, other);
                    o.y = __shfl_sync(0xffffffffu, w[b].y, other);
                    o.z = __shfl_sync(0xffffffffu, w[b].z, other);
                    o.w = __shfl_sync(0xffffffffu, w[b].w, other);
                }
                if (turned && !is_v) {
                    const float2 q0 = unpack2<T>(o.x), q1 = unpack2<T>(o.y), q2 = unpack2<T>(o.z), q3 = unpack2<T>(o.w);
                    const float y[8] = {q0.x, q0.y, q1.x, q1.y, q2.x, q2.y, q3.x, q3.y};
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        x[i] = __fadd_rn(__fmul_rn(x[i], co[i]), __fmul_rn(y[i], si[i]));
                    w[b] = make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
                }
            }
            if (on && is_q)
                *reinterpret_cast<uint4 *>(static_cast<char *>(a.q_out) + (t * a.q_out_stride + (long long)r * D + c * 8) * 2) = w[b];
            if (top + ROWS <= hq)  // no lane of the warp has a row for the cache
                continue;
            const int h = is_v ? r - hq - hkv : r - hq;
            const bool store = on && !is_q;
            if (ROPE && store && !is_v && a.k_out != nullptr)
                *reinterpret_cast<uint4 *>(static_cast<char *>(a.k_out) + (t * a.k_out_stride + (long long)h * D + c * 8) * 2) = w[b];
            const long long prow = (blk * hkv + (store ? h : 0)) * a.block_size + off;
            void *pool = is_v ? a.v_pool : a.k_pool, *scales = is_v ? a.v_scales : a.k_scales;
            if constexpr (POOL == 16) {
                if (store)
                    static_cast<uint4 *>(pool)[prow * C + c] = w[b];
            } else {
                uint16_t d16;
                if constexpr (POOL == 8) {
                    uint2 codes;
                    q8_quantize8(x, codes, d16);
                    if (store)
                        static_cast<uint2 *>(pool)[prow * C + c] = codes;
                } else {
                    uint32_t codes;
                    q4_quantize8(x, codes, d16);
                    if (store)
                        static_cast<uint32_t *>(pool)[prow * C + c] = codes;
                }
                if (store && (c & 3) == 0)
                    static_cast<uint16_t *>(scales)[prow * (C / 4) + (c >> 2)] = d16;
            }
        }
    }
}

template <typename T, int D>
const void *kernel_of(int pool, bool rope)
{
    if (pool == 16)
        return (const void *)rope_append_kernel<T, D, 16, true>;
    if (pool == 4)
        return rope ? (const void *)rope_append_kernel<T, D, 4, true> : (const void *)rope_append_kernel<T, D, 4, false>;
    return D == 64 ? (const void *)rope_append_kernel<T, 64, 8, true> : nullptr;
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendArgs &in, int pool, cudaStream_t stream)
{
    RopeAppendArgs a = in;
    const bool rope = a.positions != nullptr;
    const void *kern = a.dtype == NS_BF16 ? (a.head_dim == 64 ? kernel_of<BF16, 64>(pool, rope) : kernel_of<BF16, 128>(pool, rope))
                                          : (a.head_dim == 64 ? kernel_of<F16, 64>(pool, rope) : kernel_of<F16, 128>(pool, rope));
    int sms = 0;
    const cudaError_t e = current_sms(&sms);
    if (e != cudaSuccess)
        return e;
    // A batch of rows is the least a warp takes; a token's batches are shared by as many
    // warps as the GPU has room for (16 an SM), so that few tokens spread over it.
    const int warp_rows = 32 / (a.head_dim / 8) * kBatch, rows = (rope ? a.num_q_heads : 0) + 2 * a.num_kv_heads;
    const long long batches = (rows + warp_rows - 1) / warp_rows;
    const long long room = std::max<long long>(1, (long long)sms * 16 / a.num_tokens);
    const int per = (int)((batches + std::min(batches, room) - 1) / std::min(batches, room));
    int part_rows = per * warp_rows, parts = (rows + part_rows - 1) / part_rows;
    const long long warps = (long long)a.num_tokens * parts, grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (grid > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    void *args[] = {&a, &parts, &part_rows};
    return launch_early(kern, dim3((unsigned)grid), kThreads, 0, stream, args);
}

}  // namespace ns
