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

// What a warp does is a run of steps, 32 / (D / 8) head rows each: a token's query rows, then its
// key and value rows.
template <int D>
constexpr int step_rows() { return 32 / (D / 8); }
constexpr int kBatch = 4;  // query steps in flight
constexpr int kLeast = 2;  // steps of a warp, at least

// TURN: 0 no rotation, 1 pairs of halves, 2 neighbours.
template <typename T, int D, int POOL, int TURN>
__global__ void __launch_bounds__(kThreads, 7) rope_append_kernel(const RopeAppendArgs a, int part_steps)
{
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr bool ROPE = TURN != 0, pairs = TURN == 2;
    constexpr int C = D / 8, ROWS = step_rows<D>();  // lanes of a row, rows of a step
    const int lane = threadIdx.x & 31, c = lane % C, sub = lane / C;
    const long long t = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int part = blockIdx.y;
    if (t >= a.num_tokens)
        return;
    const int hq = ROPE ? a.num_q_heads : 0, hkv = a.num_kv_heads;
    const int q_steps = (hq + ROWS - 1) / ROWS, steps = q_steps + (2 * hkv + ROWS - 1) / ROWS;
    const int first = part * part_steps, last = min(steps, first + part_steps);

    // the first rows are on their way before the slot and the position are known
    const long long slot = a.slot_mapping[t];
    const int pos = ROPE ? a.positions[t] : 0;
    const uint16_t *q_row = static_cast<const uint16_t *>(a.q) + t * a.q_stride + (sub * D + c * 8);
    const uint16_t *k_row = static_cast<const uint16_t *>(a.k) + t * a.k_stride + c * 8,
                   *v_row = static_cast<const uint16_t *>(a.v) + t * a.v_stride + c * 8;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    uint4 qw[kBatch], kw;
    auto load_q = [&](int step) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            qw[b] = step + b < last && (step + b) * ROWS + sub < hq
                        ? *reinterpret_cast<const uint4 *>(q_row + (step + b) * (ROWS * D))
                        : none;
    };
    auto load_kv = [&](int step) {  // keys, then values
        const int r = (step - q_steps) * ROWS + sub;
        return step < last && r < 2 * hkv ? *reinterpret_cast<const uint4 *>(r < hkv ? k_row + r * D : v_row + (r - hkv) * D) : none;
    };
    if (first < q_steps)
        load_q(first);
    kw = load_kv(max(first, q_steps));

    if (slot < 0)
        return;
    const bool bad_slot = slot >= a.num_blocks * a.block_size, bad_pos = ROPE && (pos < 0 || pos >= a.max_positions);
    if (bad_slot || bad_pos) {
        if (part == 0 && lane == 0)
            raise_status(a.status, (bad_slot ? NS_DEV_BAD_SLOT : 0u) | (bad_pos ? NS_DEV_BAD_POSITION : 0u));
        return;
    }

    // this lane's cosines and sines (of the pair's lower element negative), and the lane
    // that holds the other elements of its pairs
    float2 co[4], si[4];
    const int half = a.rotary_dim / 2, hc = half / 8;  // elements, lanes (halves)
    const bool turned = ROPE && c < 2 * hc;
    int other = lane;
    if (turned) {
        const float *row = a.cos_sin + (long long)pos * a.rotary_dim;
        if (!pairs) {
            const bool low = c < hc;
            other = low ? lane + hc : lane - hc;
            const float *at = row + (low ? c : c - hc) * 8;
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float4 x = *reinterpret_cast<const float4 *>(at + 2 * i), y = *reinterpret_cast<const float4 *>(at + half + 2 * i);
                co[i] = make_float2(x.x, x.y), co[i + 1] = make_float2(x.z, x.w);
                si[i] = low ? make_float2(-y.x, -y.y) : make_float2(y.x, y.y);
                si[i + 1] = low ? make_float2(-y.z, -y.w) : make_float2(y.z, y.w);
            }
        } else {
            const float4 x = *reinterpret_cast<const float4 *>(row + c * 4), y = *reinterpret_cast<const float4 *>(row + half + c * 4);
            co[0] = make_float2(x.x, x.x), co[1] = make_float2(x.y, x.y), co[2] = make_float2(x.z, x.z), co[3] = make_float2(x.w, x.w);
            si[0] = make_float2(-y.x, y.x), si[1] = make_float2(-y.y, y.y), si[2] = make_float2(-y.z, y.z), si[3] = make_float2(-y.w, y.w);
        }
    }
    // x: this lane's elements, turned where `turn` says so; all lanes take part
    auto rotate = [&](const uint4 &w, bool turn, float2 (&x)[4]) {
        uint4 o;
        if (pairs) {  // the other element of a pair is in the same word
            o = make_uint4(__byte_perm(w.x, 0u, 0x1032), __byte_perm(w.y, 0u, 0x1032), __byte_perm(w.z, 0u, 0x1032),
                           __byte_perm(w.w, 0u, 0x1032));
        } else {
            o.x = __shfl_sync(0xffffffffu, w.x, other);
            o.y = __shfl_sync(0xffffffffu, w.y, other);
            o.z = __shfl_sync(0xffffffffu, w.z, other);
            o.w = __shfl_sync(0xffffffffu, w.w, other);
        }
        const uint32_t mine[4] = {w.x, w.y, w.z, w.w}, others[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = unpack2<T>(mine[i]);
            if (turn) {  // (with the sum of pairs too they come out contracted)
                const float2 y = fmul2(unpack2<T>(others[i]), si[i]);
                x[i] = fmul2(x[i], co[i]);
                x[i] = make_float2(__fadd_rn(x[i].x, y.x), __fadd_rn(x[i].y, y.y));
            }
        }
    };
    auto packed = [](const float2 (&x)[4]) {
        return make_uint4(pack2<T>(x[0].x, x[0].y), pack2<T>(x[1].x, x[1].y), pack2<T>(x[2].x, x[2].y), pack2<T>(x[3].x, x[3].y));
    };

    if (ROPE) {
        uint16_t *to = static_cast<uint16_t *>(a.q_out) + t * a.q_out_stride + (sub * D + c * 8);
        for (int s0 = first; s0 < min(last, q_steps); s0 += kBatch) {
            if (s0 > first)
                load_q(s0);
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (s0 + b >= min(last, q_steps))
                    break;
                float2 x[4];
                rotate(qw[b], turned, x);
                if ((s0 + b) * ROWS + sub < hq)
                    *reinterpret_cast<uint4 *>(to + (s0 + b) * (ROWS * D)) = turned ? packed(x) : qw[b];
            }
        }
    }
    if (last <= q_steps)
        return;
    const int shift = __ffs(a.block_size) - 1;  // a power of two
    const long long row0 = (((slot >> shift) * hkv) << shift) + ((int)slot & (a.block_size - 1));  // of kv head 0
    for (int step = max(first, q_steps); step < last; ++step) {
        const int r = (step - q_steps) * ROWS + sub;
        const bool on = r < 2 * hkv, is_v = r >= hkv;
        const int h = is_v ? r - hkv : r;
        uint4 w = kw;
        kw = load_kv(step + 1);
        float2 x[4];
        if (ROPE) {
            rotate(w, turned && !is_v, x);
            if (turned && !is_v)
                w = packed(x);
        } else {
            x[0] = unpack2<T>(w.x), x[1] = unpack2<T>(w.y), x[2] = unpack2<T>(w.z), x[3] = unpack2<T>(w.w);
        }
        if (ROPE && on && !is_v && a.k_out != nullptr)
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.k_out) + t * a.k_out_stride + (h * D + c * 8)) = w;
        const long long prow = row0 + ((long long)h << shift);
        void *pool = is_v ? a.v_pool : a.k_pool;
        if constexpr (POOL == 16) {
            if (on)
                static_cast<uint4 *>(pool)[prow * C + c] = w;
        } else {
            const float y[8] = {x[0].x, x[0].y, x[1].x, x[1].y, x[2].x, x[2].y, x[3].x, x[3].y};
            uint16_t d16;
            if constexpr (POOL == 8) {
                uint2 codes;
                q8_quantize8(y, codes, d16);
                if (on)
                    static_cast<uint2 *>(pool)[prow * C + c] = codes;
            } else {
                uint32_t codes;
                q4_quantize8(y, codes, d16);
                if (on)
                    static_cast<uint32_t *>(pool)[prow * C + c] = codes;
            }
            if (on && (c & 3) == 0)
                static_cast<uint16_t *>(is_v ? a.v_scales : a.k_scales)[prow * (C / 4) + (c >> 2)] = d16;
        }
    }
}

template <typename T, int D, int TURN>
const void *kernel_of(int pool)
{
    if constexpr (TURN == 0)
        return (const void *)rope_append_kernel<T, D, 4, 0>;
    else if (pool == 8)
        return D == 64 ? (const void *)rope_append_kernel<T, 64, 8, TURN> : nullptr;
    else
        return pool == 16 ? (const void *)rope_append_kernel<T, D, 16, TURN> : (const void *)rope_append_kernel<T, D, 4, TURN>;
}

template <typename T, int D>
const void *kernel_of(int pool, int turn)
{
    return turn == 0 ? kernel_of<T, D, 0>(pool) : turn == 1 ? kernel_of<T, D, 1>(pool) : kernel_of<T, D, 2>(pool);
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendArgs &in, int pool, cudaStream_t stream)
{
    RopeAppendArgs a = in;
    const bool rope = a.positions != nullptr;
    const int turn = !rope ? 0 : a.interleaved ? 2 : 1;
    const void *kern = a.dtype == NS_BF16 ? (a.head_dim == 64 ? kernel_of<BF16, 64>(pool, turn) : kernel_of<BF16, 128>(pool, turn))
                                          : (a.head_dim == 64 ? kernel_of<F16, 64>(pool, turn) : kernel_of<F16, 128>(pool, turn));
    int sms = 0;
    const cudaError_t e = current_sms(&sms);
    if (e != cudaSuccess)
        return e;
    // A token's steps are shared by as many warps as the GPU has room for (32 an SM), so that few
    // tokens spread over it.
    const int rows = a.head_dim == 64 ? step_rows<64>() : step_rows<128>();
    const int steps = ((rope ? a.num_q_heads : 0) + rows - 1) / rows + (2 * a.num_kv_heads + rows - 1) / rows;
    const long long shares = (steps + kLeast - 1) / kLeast;
    const long long room = std::max<long long>(1, (long long)sms * 32 / a.num_tokens);
    const int per = (int)((shares + std::min(shares, room) - 1) / std::min(shares, room));
    int part_steps = per * kLeast;
    const int parts = (steps + part_steps - 1) / part_steps;  // at most 32 sms
    void *args[] = {&a, &part_steps};
    return launch_early(kern, dim3((unsigned)((a.num_tokens - 1) / (kThreads / 32) + 1), (unsigned)parts), kThreads, 0, stream, args);
}

}  // namespace ns
