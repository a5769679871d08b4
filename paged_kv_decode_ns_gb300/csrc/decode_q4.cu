// decode_q4.cu -- decode attention over a q4_0 (4-bit) paged cache.
//
// out = sum_p 2^(z_p - m) v_p / sum_p 2^(z_p - m), z in log2 units, in one pass over the
// keys with a running reference m.  K_p = dk_p (c - 8) and V_p = dv_p (c - 8) by group of 32
// elements, so that with integer codes c
//   z_p = scale sum_g dk_pg (q_g . c_pg - 8 sum q_g),   out_g = sum_p (w_p dv_pg) (c_pg - 8):
// the steps are applied to the scores and to the weights, 8 heads wide, instead of to 64 or 128
// elements, and the 8 of K once for a row of q.  A code is used as it lies: four bits at the
// bottom of an fp16 word are the (subnormal) number c 2^-24, or c 2^-20 one place higher, so one
// AND makes two operands.  (A sum of w_p dv_pg for V's 8 would cancel against a much larger
// one, and a product for it took as long as the subtraction.)  Both sums are small matrix
// products (mma.m16n8k16: 16 tokens or elements by the 8 query heads of a group, fp32 sums).  A tcgen05
// product has 128 rows at least and its operands in shared memory, where each code would
// be four times as large as in the cache; here they go from the codes to the product in registers.
//
// Only two factors are rounded: q to fp16, scaled by a power of two (exact down to 2^-24 of the
// row's largest element, off by 2^-35 of that below) and w dv to fp16 (2^-11 of itself, or 2^-32
// of the largest weight times the largest step so far).
//
// Work.  The pairs (sequence, kv head, 8 query heads) lie end to end on a line, in chunks of
// 32 tokens and two more for a pair's own cost, and each warp of a persistent grid takes an
// equal run of it.  A pair cut by warps of one CTA is joined in shared memory, one cut by
// CTAs through records in the workspace, by the CTA that arrives last; in the order of the
// keys, so results do not depend on timing.
#include <algorithm>
#include <cmath>

#include "ns_internal.h"
#include "q4_decode.h"
#include "quantise.cuh"

namespace ns {

namespace {

constexpr int kChunk = 32;     // tokens of a step: one a lane
constexpr int kPairCost = 2;   // chunks that a pair counts besides its own (batch 256 21.9 us; 0: 23.7, 1 and 3: 22.4)
constexpr float kNone = -3.402823466e38f;
constexpr float kLeastUnit = 1.17549435e-38f, kMostUnit = 1.2676506e30f;  // 2^-126, 2^100
// The largest w dv is set just below 2^kLift, and again when one would pass that by
// 2^kSlack: fp16 has room up to 2^16 and steps of 2^-24.
constexpr float kLift = 7.0f, kSlack = 8.0f;

template <int D>
struct Geo {
    static constexpr int R = D / 32;                       // groups of 32 elements
    static constexpr int WARPS = D == 64 ? 16 : 12;
    static constexpr int STAGES = 3;                       // chunks of a warp, one of them in use
    static constexpr int CODES = kChunk * D / 2;           // bytes of a chunk's K or V
    static constexpr int SCALES = kChunk * R * 2;
    static constexpr int STAGE = 2 * (CODES + SCALES);
    static constexpr int RECORD = 8 * (D + 2);             // floats: m, l, O of 8 heads
    static constexpr int THREADS = WARPS * 32;
    static constexpr int SLOTS = 2 * D;                    // float4s of 8 heads' O
};

template <int D>
struct alignas(16) Smem {
    using GG = Geo<D>;
    uint8_t ring[GG::WARPS][GG::STAGES][GG::STAGE];  // afterwards a warp's last record
    float first[GG::WARPS][GG::RECORD];              // its first one
    int before[GG::THREADS];                         // chunks in front of a thread's sequences
    int scan[GG::WARPS];
    // what a warp left: the pair of its first and last record (-1: none) and whether the first
    // one goes to its pair's end
    int first_pair[GG::WARPS], first_ends[GG::WARPS], last_pair[GG::WARPS];
    // the pair that came from a CTA before and the one that goes on in the next: the CTAs that
    // have parts of it, and the pair again when it is left to the whole CTA to join
    int first_cta[2], pieces[2], to_join[2];
    static_assert(GG::STAGES * GG::STAGE >= GG::RECORD * 4, "a record fits a warp's ring");
};

struct Params {
    Q4DecodeArgs a;
    int heads;      // pairs of a sequence
    int subs;       // of a kv head
    int group;      // query heads of a kv head
    int shift;      // log2 of the block size
    uint32_t blocks;  // of the pool (entries have 31 bits)
    float scale_log2, sign;  // of the scale
    int *counters;
    float *records;

    __device__ __forceinline__ float *record(int i, int floats) const { return records + (size_t)i * floats; }
};

// ---------------------------------------------------------------------------
__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four 8 x 8 matrices of 16-bit elements.
__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void load_matrices_turned(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t turn_matrix(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void product(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight codes of a word -> fp16 pairs, code i beside code i + 4: c 2^-24 for i = 0 and 2,
// c 2^-20 for i = 1 and 3.
__device__ __forceinline__ void codes_in_place(uint32_t (&p)[4], uint32_t w)
{
    const uint32_t v = w >> 8;
    p[0] = w & 0x000f000fu;
    p[1] = w & 0x00f000f0u;
    p[2] = v & 0x000f000fu;
    p[3] = v & 0x00f000f0u;
}
// Those of codes less 8 (subnormal too, or 0).
__device__ __forceinline__ void less_8(uint32_t (&p)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __hadd2(*reinterpret_cast<__half2 *>(&p[i]), __half2half2(__ushort_as_half(i & 1 ? 0x8080 : 0x8008)));
        p[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
}
constexpr float kCode = 16777216.f, kCodeHigh = 1048576.f;  // 2^24, 2^20

__device__ __forceinline__ float unit_of(float x) { return fminf(fmaxf(x * kCode, kLeastUnit), kMostUnit); }

__device__ __forceinline__ uint32_t larger_f16(uint32_t a, uint32_t b)  // magnitudes, signs of no meaning
{
    uint32_t r;
    asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The same with a sum that starts elsewhere.
__device__ __forceinline__ void product(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, float c0, float c1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %10, %11};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}

__device__ __forceinline__ float2 halves(uint32_t w) { return unpack2<F16>(w); }

// ---------------------------------------------------------------------------
// Walk over the pieces of a warp's run.
// ---------------------------------------------------------------------------
struct Piece {
    int s, h;       // sequence, pair of it
    int L;          // keys of the sequence
    int c, c1;      // chunks
    int whole;      // the piece is its whole pair
    int ends;       // it goes to the pair's end
};

struct Walk {
    int s, h, off;  // where the next piece starts
    int left;       // chunks of the run still to come
};

__device__ __forceinline__ int keys_of(const Q4DecodeArgs &a, int shift, int s)
{
    const int L = a.context_lens[s];
    const long long cap = (long long)a.max_blocks_per_seq << shift;
    return L < 0 ? 0 : L > cap ? (int)cap : L;
}

__device__ __forceinline__ int length_of(int L) { return (L + kChunk - 1) / kChunk + kPairCost; }

// The next piece of a run that is not over.
__device__ __forceinline__ Piece next_piece(const Params &P, Walk &w)
{
    Piece p;
    p.s = w.s;
    p.h = w.h;
    p.L = keys_of(P.a, P.shift, w.s);
    const int len = length_of(p.L), take = min(w.left, len - w.off);
    p.c = max(w.off - kPairCost, 0);
    p.c1 = max(w.off + take - kPairCost, 0);
    p.ends = w.off + take == len;
    p.whole = p.ends && w.off == 0;
    w.left -= take;
    w.off = 0;
    if (p.ends && ++w.h == P.heads) {
        w.h = 0;
        ++w.s;
    }
    return p;
}

// ---------------------------------------------------------------------------
// A pair's parts, joined by a warp: lane i has float4s i, i + 32, .. of O, with the reference and
// the sum of their heads.  Loops of little code, since every warp runs them once and has to
// fetch it (batch 256 21.4 us; unrolled over all 16 records 21.8, not at all 21.8).
template <int D>
struct Joined {
    static constexpr int F = D / 16, PER = D / 4;  // float4s of a lane, of a head
    float4 acc[F];
    float top[F], sum[F];

    // n records of this CTA, in the order of the keys
    template <typename Record>
    __device__ __forceinline__ void join(int n, int lane, const Record &record)
    {
#pragma unroll
        for (int f = 0; f < F; ++f) {
            acc[f] = make_float4(0.f, 0.f, 0.f, 0.f);
            top[f] = kNone;
            sum[f] = 0.f;
        }
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const float *r = record(i);
#pragma unroll
            for (int f = 0; f < F; ++f)
                top[f] = fmaxf(top[f], r[(32 * f + lane) / PER]);
        }
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const float *r = record(i);
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const int at = 32 * f + lane, h = at / PER;
                const float c = fast_exp2(r[h] - top[f]);
                const float4 y = reinterpret_cast<const float4 *>(r + 16)[at];
                sum[f] = fmaf(c, r[8 + h], sum[f]);
                acc[f].x = fmaf(c, y.x, acc[f].x), acc[f].y = fmaf(c, y.y, acc[f].y);
                acc[f].z = fmaf(c, y.z, acc[f].z), acc[f].w = fmaf(c, y.w, acc[f].w);
            }
        }
    }

    // A record of another CTA.
    __device__ __forceinline__ void load(const float *rec, int lane)
    {
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int at = 32 * f + lane;
            top[f] = __ldcg(rec + at / PER);
            sum[f] = __ldcg(rec + 8 + at / PER);
            acc[f] = __ldcg(reinterpret_cast<const float4 *>(rec + 16) + at);
        }
    }

    // The part behind this one in the order of the keys.
    __device__ __forceinline__ void add(const Joined &next)
    {
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const float higher = fmaxf(top[f], next.top[f]);
            const float a = fast_exp2(top[f] - higher), b = fast_exp2(next.top[f] - higher);
            top[f] = higher;
            sum[f] = fmaf(b, next.sum[f], a * sum[f]);
            acc[f].x = fmaf(b, next.acc[f].x, a * acc[f].x), acc[f].y = fmaf(b, next.acc[f].y, a * acc[f].y);
            acc[f].z = fmaf(b, next.acc[f].z, a * acc[f].z), acc[f].w = fmaf(b, next.acc[f].w, a * acc[f].w);
        }
    }

    __device__ __forceinline__ void keep(float *rec, int lane) const
    {
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int at = 32 * f + lane;
            if (at % PER == 0) {
                rec[at / PER] = top[f];
                rec[8 + at / PER] = sum[f];
            }
            reinterpret_cast<float4 *>(rec + 16)[at] = acc[f];
        }
    }

    template <typename T>
    __device__ __forceinline__ void put(const Params &P, int pair, int lane) const
    {
        const int s = pair / P.heads, ph = pair - s * P.heads, kv = ph / P.subs, sub = ph - kv * P.subs;
        uint8_t *row = static_cast<uint8_t *>(P.a.out) + ((long long)s * P.a.num_q_heads + kv * P.group + sub * 8) * (D * 2);
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int at = 32 * f + lane;
            const float c = sum[f] == 0.f ? 0.f : __fdividef(1.f, sum[f]);
            if (at / PER < P.group - sub * 8)
                reinterpret_cast<uint2 *>(row)[at] = make_uint2(pack2<T>(acc[f].x * c, acc[f].y * c), pack2<T>(acc[f].z * c, acc[f].w * c));
        }
    }
};

// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(Geo<D>::THREADS, 1) decode_q4_kernel(const __grid_constant__ Params P)
{
    using GG = Geo<D>;
    constexpr int R = GG::R, ST = GG::STAGES, W = GG::WARPS;
    constexpr int PARTS = R;                    // 16-byte parts of a token's codes: one a group
    constexpr int SPAN = 16 / (2 * R);          // tokens whose scales are 16 bytes
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>(smem_raw);
    const Q4DecodeArgs &a = P.a;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;  // row and column pair of the products' fragments
    if (lane == 0) {  // by the lane that writes them later: no barrier lies between (up to 32 sequences)
        sm.first_pair[warp] = -1;
        sm.last_pair[warp] = -1;
    }
    if (tid < 2)
        sm.to_join[tid] = -1;
    grid_dependency_wait();
    grid_launch_dependents();

    // ---- the line: each lane of a warp, or with more of them each thread of the CTA, measures a
    // share of the sequences
    const bool few = a.num_seqs <= 32;
    const int per = few ? 1 : (a.num_seqs + GG::THREADS - 1) / GG::THREADS, who = few ? lane : tid;
    const int s0 = min(a.num_seqs, who * per), s1 = min(a.num_seqs, s0 + per);
    int mine = 0;
    for (int s = s0; s < s1; ++s) {
        const int L = a.context_lens[s];
        if (blockIdx.x == 0 && (L < 0 || L > ((long long)a.max_blocks_per_seq << P.shift)))
            raise_status(a.status, NS_DEV_BAD_CONTEXT_LEN);
        mine += length_of(keys_of(a, P.shift, s));
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += y;
    }
    int total = __shfl_sync(0xffffffffu, incl, 31), ahead = 0;
    if (!few) {
        if (lane == 31)
            sm.scan[warp] = incl;
        __syncthreads();
        total = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int x = sm.scan[i];
            ahead += i < warp ? x : 0;
            total += x;
        }
        sm.before[tid] = ahead + incl - mine;
        __syncthreads();
    }
    total *= P.heads;
    // Runs: the first `rest` of `runs` warps take share + 1 chunks, the others share.  What one CTA
    // can do with three chunks a warp stays in one (four short sequences 6.4 us, 7.2 by single chunks
    // in three CTAs; 8 x 4096 tokens by two chunks 10.0, by one 9.0).
    const int runs = min((int)gridDim.x * W, total <= 3 * W ? min(W, (total + 1) / 2) : total);
    const int share = quotient(total, runs), rest = total - share * runs;
    const int me = blockIdx.x * W + warp;
    if ((int)blockIdx.x * W >= runs)
        return;
    auto cta_of = [&](int x) {  // of the warp whose run has position x
        const int y = x - rest * (share + 1);
        return (y < 0 ? quotient(x, share + 1) : rest + quotient(y, share)) / W;
    };
    Walk next;
    next.s = next.h = next.off = 0;
    next.left = me < runs ? share + (me < rest ? 1 : 0) : 0;
    const int x0 = me * share + min(me, rest);
    if (me < runs) {
        // the last lane or thread whose sequences start at x0 or before
        int lo, y;
        if (few) {
            lo = __popc(__ballot_sync(0xffffffffu, lane < a.num_seqs && (incl - mine) * P.heads <= x0)) - 1;
            y = x0 - __shfl_sync(0xffffffffu, incl - mine, lo) * P.heads;
        } else {  // of every `step`th, then of each
            auto starts = [&](int i) { return i < GG::THREADS && (long long)i * per < a.num_seqs && sm.before[i] * P.heads <= x0; };
            constexpr int step = GG::THREADS / 32;
            lo = (__popc(__ballot_sync(0xffffffffu, starts(lane * step))) - 1) * step;
            lo += __popc(__ballot_sync(0xffffffffu, lane < step && starts(lo + lane))) - 1;
            y = x0 - sm.before[lo] * P.heads;
        }
        for (int s = lo * per;; ++s) {
            const int len = length_of(keys_of(a, P.shift, s));
            if (y < len * P.heads || s + 1 >= a.num_seqs) {
                next.s = s;
                next.h = quotient(y, len);
                next.off = y - next.h * len;
                break;
            }
            y -= len * P.heads;
        }
    }
    Walk ahead_walk = next;  // the copies' walk, up to ST - 1 chunks ahead of the arithmetic

    // ---- copies: a chunk's codes and scales of K and V by 16 bytes a lane.  A lane's places in
    // its tokens' blocks are the same in every chunk, so an address is one multiplication of
    // the block's number.
    const uint32_t ring = smem_addr(sm.ring[warp][0]);
    constexpr uint32_t row_bytes = D / 2;
    constexpr int N = kChunk / SPAN;          // lanes that copy the scales of K, and again of V
    constexpr int TOKENS = 32 / PARTS;        // of a copy of all lanes
    const int bs1 = (1 << P.shift) - 1;
    const uint32_t block_rows = (uint32_t)a.num_kv_heads << P.shift;  // of all heads
    const int part = lane % PARTS, tau0 = lane / PARTS, tau_s = lane % N * SPAN;
    // eight rows of one part are eight different banks of 16 bytes
    const uint32_t place = tau0 * row_bytes + (D == 64 ? part ^ ((tau0 >> 2) & 1) : part ^ ((tau0 >> 1) & 3)) * 16;
    const uint32_t lane_at = (tau0 & bs1) * row_bytes + part * 16, lane_at_s = (tau_s & bs1) * (2 * R);
    // blocks of 32: the second 16 tokens are further on in the same block (head_dim 64)
    const uint32_t hop = D == 64 && P.shift == 5 ? 16 * row_bytes : 0u;
    Piece ip;
    ip.c = ip.c1 = 0;
    ip.s = ip.h = ip.L = 0;
    int entry = -1;  // the block of this lane's token in the next chunk to copy
    const uint8_t *k_from = nullptr, *v_from = nullptr, *s_from = nullptr;  // of the piece's head in block 0
    const int32_t *row_of = nullptr;  // its sequence's table row
    uint32_t to = ring, in_flight[ST - 1] = {};  // tokens that count of the chunks on their way
    auto look_up = [&]() {  // the next chunk's blocks, whose piece may be another one
        if (ip.c == ip.c1) {
            while (ip.c == ip.c1 && ahead_walk.left > 0)
                ip = next_piece(P, ahead_walk);
            if (ip.c < ip.c1) {
                const int kv = P.subs == 1 ? ip.h : ip.h / P.subs;
                const uint32_t head = (uint32_t)kv << P.shift;
                k_from = static_cast<const uint8_t *>(a.k_codes) + (head * row_bytes + lane_at);
                v_from = static_cast<const uint8_t *>(a.v_codes) + (head * row_bytes + lane_at);
                s_from = static_cast<const uint8_t *>(lane < N ? a.k_scales : a.v_scales) + (head * (2 * R) + lane_at_s);
                row_of = a.block_tables + (long long)ip.s * a.max_blocks_per_seq;
            }
        }
        entry = -1;
        const int tok = ip.c * kChunk + lane;
        if (ip.c < ip.c1 && tok < ip.L)
            entry = row_of[tok >> P.shift];
    };
    auto issue = [&]() {
#pragma unroll
        for (int i = 0; i < ST - 2; ++i)
            in_flight[i] = in_flight[i + 1];
        if (ip.c < ip.c1) {
            const bool ok = (uint32_t)entry < P.blocks;
            const int block = ok ? entry : -1;
            const uint32_t live = __ballot_sync(0xffffffffu, ok);
            in_flight[ST - 2] = live;
            if (live != 0xffffffffu && !ok && ip.c * kChunk + lane < ip.L)
                raise_status(a.status, NS_DEV_BAD_BLOCK_ID);
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // 16 tokens each
                const int id = __shfl_sync(0xffffffffu, block, tau0 + 16 * i);
                if (id >= 0) {
                    const unsigned long long at = (unsigned long long)((uint32_t)id) * (block_rows * row_bytes) + i * hop;
                    const uint8_t *k = k_from + at, *v = v_from + at;
                    const uint32_t dst = to + place + i * 16 * row_bytes;
#pragma unroll
                    for (int x = 0; x < 16 / TOKENS; ++x) {
                        copy16(dst + x * TOKENS * row_bytes, k + x * TOKENS * row_bytes);
                        copy16(dst + x * TOKENS * row_bytes + GG::CODES, v + x * TOKENS * row_bytes);
                    }
                }
            }
            {
                const int id = __shfl_sync(0xffffffffu, block, tau_s);
                if (id >= 0 && lane < 2 * N)
                    copy16(to + 2 * GG::CODES + lane * 16, s_from + (unsigned long long)((uint32_t)id) * (block_rows * (2 * R)));
            }
            ++ip.c;
            to = to == ring + (ST - 1) * GG::STAGE ? ring : to + GG::STAGE;
            look_up();
        }
        copies_commit();
    };

    look_up();
#pragma unroll 1  // (less code to fetch: batch 256 22.6 -> 22.3 us)
    for (int i = 0; i < ST - 1; ++i)
        issue();

    // ---- arithmetic
    int used = 0;  // chunks, modulo ST
    while (next.left > 0) {
        const int off0 = next.off, x = x0 + (share + (me < rest ? 1 : 0)) - next.left;  // the piece's position
        const Piece p = next_piece(P, next);
        if (lane == 0 && (warp == 0 ? off0 > 0 : warp == W - 1 && !p.ends)) {
            const int slot = warp == 0 ? 0 : 1, begin = x - off0, c0 = cta_of(begin);
            sm.first_cta[slot] = c0;
            sm.pieces[slot] = cta_of(begin + length_of(p.L) - 1) - c0 + 1;
        }
        const int kv = P.subs == 1 ? p.h : p.h / P.subs, sub = p.h - kv * P.subs;
        const int head0 = kv * P.group + sub * 8, heads = min(8, P.group - sub * 8);
        // q of head g, elements 8 t .. 8 t + 7 of each group, as the products' second operand
        uint32_t q[R][4];
        float q_unit;      // 2^-e: what a unit of q is worth
        float q_sum[R];    // -8 times the sum of a group, as the products count
        {
            uint4 w[R];
            float top = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                w[r] = make_uint4(0u, 0u, 0u, 0u);
                if (g < heads)
                    w[r] = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.q) +
                                                            (((long long)p.s * a.num_q_heads + head0 + g) * D + 32 * r + 8 * t) * 2);
                const uint32_t x[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = unpack2<T>(x[i]);
                    top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // the row's largest goes to [2^14, 2^15); the factor stays a normal number
            const int e = top > 0.f && top < INFINITY ? min(max(141 - (int)(__float_as_uint(top) >> 23), -113), 113) : 0;
            const float f = P.sign * __uint_as_float((uint32_t)(127 + e) << 23), f_high = f * 0.0625f;
            q_unit = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint32_t x[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
                // elements i and i + 4, less four binary places where the code is that much higher
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 a0 = unpack2<T>(x[i >> 1]), a1 = unpack2<T>(x[(i >> 1) + 2]);
                    q[r][i] = i & 1 ? pack2<F16>(a0.y * f_high, a1.y * f_high) : pack2<F16>(a0.x * f, a1.x * f);
                    const float2 y = halves(q[r][i]);
                    sum = fmaf(y.x + y.y, i & 1 ? 16.f : 1.f, sum);
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                q_sum[r] = sum * (-8.f / kCode);
            }
        }
        // of the two heads of this lane's columns: a unit of the products, and where they start.  The
        // unit stays above 0, which the -infinity of a token that is not there must not meet, and at 2^100:
        // different products are 2^-72 apart at least, so that their scores still differ by 2^28 there.
        const float2 unit = make_float2(unit_of(P.scale_log2 * __shfl_sync(0xffffffffu, q_unit, 8 * t)),
                                        unit_of(P.scale_log2 * __shfl_sync(0xffffffffu, q_unit, 8 * t + 4)));
        float2 base[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
            base[r] = make_float2(__shfl_sync(0xffffffffu, q_sum[r], 8 * t), __shfl_sync(0xffffffffu, q_sum[r], 8 * t + 4));

        float O[R][2][4];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    O[r][u][i] = 0.f;
        // Weights are 2^((z - z0) unit + lift): the reference z0 and the limit of the scores are in units of the
        // products, and the difference of scores of any size is exact before it is scaled.  (As z unit - m
        // in one step, scores from 2^24 on met the rounding of m; batch 256 21.3 us then, 21.7 so.)
        float2 l = make_float2(0.f, 0.f), z0 = make_float2(kNone, kNone), limit = z0;
        const float2 slack = make_float2(kSlack * __fdividef(1.f, unit.x), kSlack * __fdividef(1.f, unit.y));
        uint32_t step_limit = 0u;  // the largest fp16 with the exponent of the largest V step so far
        float lift = 0.f;          // kLift less what those steps are below, in log2

        for (int c = p.c; c < p.c1; ++c) {
            copies_wait<ST - 2>();
            __syncwarp();
            const uint32_t live = in_flight[0];
            issue();  // into the stage that the last turn has read
            const uint32_t from = ring + used * GG::STAGE;
            const uint8_t *stage = sm.ring[warp][used];
            used = used + 1 == ST ? 0 : used + 1;

            // ---- scores: 16 tokens at a time, by group
            float2 z[2][2];  // [tile][token g or g + 8] of the two heads, in units of the products
            uint32_t dv[2][2][R / 2];
#pragma unroll
            for (int tile = 0; tile < 2; ++tile) {
                uint32_t dk[2][R / 2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint8_t *at = stage + 2 * GG::CODES + (tile * 16 + i * 8 + g) * (2 * R);
                    if constexpr (R == 2) {
                        dk[i][0] = *reinterpret_cast<const uint32_t *>(at);
                        dv[tile][i][0] = *reinterpret_cast<const uint32_t *>(at + GG::SCALES);
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2 *>(at), y = *reinterpret_cast<const uint2 *>(at + GG::SCALES);
                        dk[i][0] = x.x, dk[i][1] = x.y;
                        dv[tile][i][0] = y.x, dv[tile][i][1] = y.y;
                    }
                }
#pragma unroll
                for (int r2 = 0; r2 < R; r2 += 2) {
                    uint32_t w[4];
                    {
                        const int tau = tile * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), part = r2 + (lane >> 4);
                        const int turned = D == 64 ? part ^ ((tau >> 2) & 1) : part ^ ((tau >> 1) & 3);
                        load_matrices(w, from + tau * row_bytes + turned * 16);
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int r = r2 + j;
                        uint32_t lo[4], hi[4];
                        codes_in_place(lo, w[2 * j]);
                        codes_in_place(hi, w[2 * j + 1]);
                        float s[4];
                        product(s, lo[0], hi[0], lo[1], hi[1], q[r][0], q[r][1], base[r].x, base[r].y);
                        product(s, lo[2], hi[2], lo[3], hi[3], q[r][2], q[r][3]);
                        const float2 d0 = halves(dk[0][r2 / 2]), d1 = halves(dk[1][r2 / 2]);
                        const float e0 = j == 0 ? d0.x : d0.y, e1 = j == 0 ? d1.x : d1.y;
                        const float2 y0 = make_float2(s[0], s[1]), y1 = make_float2(s[2], s[3]);
                        z[tile][0] = r == 0 ? fmul2(y0, make_float2(e0, e0)) : ffma2(y0, make_float2(e0, e0), z[tile][0]);
                        z[tile][1] = r == 0 ? fmul2(y1, make_float2(e1, e1)) : ffma2(y1, make_float2(e1, e1), z[tile][1]);
                    }
                }
            }
            if (live != 0xffffffffu)  // a token that is not there has neither a weight nor a step
#pragma unroll
                for (int tile = 0; tile < 2; ++tile)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (!((live >> (tile * 16 + i * 8 + g)) & 1u)) {
                            z[tile][i] = make_float2(-INFINITY, -INFINITY);
#pragma unroll
                            for (int j = 0; j < R / 2; ++j)
                                dv[tile][i][j] = 0u;
                        }
            uint32_t largest = dv[0][0][0];
#pragma unroll
            for (int x = 1; x < 4 * (R / 2); ++x)
                largest = larger_f16(largest, dv[x / (R / 2) / 2][x / (R / 2) % 2][x % (R / 2)]);

            // ---- the reference moves, or the lift falls, when a weight times a step would leave fp16's range
            const float za = fmaxf(fmaxf(z[0][0].x, z[0][1].x), fmaxf(z[1][0].x, z[1][1].x));
            const float zb = fmaxf(fmaxf(z[0][0].y, z[0][1].y), fmaxf(z[1][0].y, z[1][1].y));
            const uint32_t big = max(largest & 0x7fffu, (largest >> 16) & 0x7fffu);
            if (__any_sync(0xffffffffu, za > limit.x || zb > limit.y || big > step_limit)) {
                float2 top = make_float2(za, zb);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    top.x = fmaxf(top.x, __shfl_xor_sync(0xffffffffu, top.x, o));
                    top.y = fmaxf(top.y, __shfl_xor_sync(0xffffffffu, top.y, o));
                }
                const int top_e = (int)((step_limit + 1u) >> 10) - 1;  // the field of that exponent, or -1
                const int e = max(top_e, (int)(__reduce_max_sync(0xffffffffu, big) >> 10));
                const float higher = kLift - (float)(e - 14), fall = higher - lift;  // steps are below 2^(e - 14)
                lift = higher;
                step_limit = ((uint32_t)(e + 1) << 10) - 1u;
                // a head's reference follows its own scores alone, whatever the heads beside it hold
                const float2 to = make_float2(top.x > limit.x ? top.x : z0.x, top.y > limit.y ? top.y : z0.y);
                const float2 f = make_float2(fast_exp2(fmaf(z0.x - to.x, unit.x, fall)), fast_exp2(fmaf(z0.y - to.y, unit.y, fall)));
                z0 = to;
                limit = fadd2(z0, slack);
                l = fmul2(l, f);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        O[r][u][0] *= f.x;
                        O[r][u][1] *= f.y;
                        O[r][u][2] *= f.x;
                        O[r][u][3] *= f.y;
                    }
            }

            // ---- weights, and the values' product
#pragma unroll
            for (int tile = 0; tile < 2; ++tile) {
                float2 w[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 x = ffma2(fadd2(z[tile][i], make_float2(-z0.x, -z0.y)), unit, make_float2(lift, lift));
                    w[i] = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                    l = fadd2(l, w[i]);
                }
#pragma unroll
                for (int r2 = 0; r2 < R; r2 += 2) {
                    uint32_t v[4];
                    {
                        const int tau = tile * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), part = r2 + (lane >> 4);
                        const int turned = D == 64 ? part ^ ((tau >> 2) & 1) : part ^ ((tau >> 1) & 3);
                        load_matrices_turned(v, from + GG::CODES + tau * row_bytes + turned * 16);
                    }
                    const float2 d0 = halves(dv[tile][0][r2 / 2]), d1 = halves(dv[tile][1][r2 / 2]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float e0 = j == 0 ? d0.x : d0.y, e1 = j == 0 ? d1.x : d1.y;
                        const float2 w0 = fmul2(w[0], make_float2(e0, e0)), w1 = fmul2(w[1], make_float2(e1, e1));
                        const uint32_t b0 = turn_matrix(pack2<F16>(w0.x, w0.y)), b1 = turn_matrix(pack2<F16>(w1.x, w1.y));
                        uint32_t lo[4], hi[4];
                        codes_in_place(lo, v[2 * j]);
                        codes_in_place(hi, v[2 * j + 1]);
                        less_8(lo);
                        less_8(hi);
                        product(O[r2 + j][0], lo[0], lo[1], hi[0], hi[1], b0, b1);
                        product(O[r2 + j][1], lo[2], lo[3], hi[2], hi[3], b0, b1);
                    }
                }
            }
        }

        // ---- the piece's end: this lane has elements 4 g .. 4 g + 3 of each group, heads 2 t, 2 t + 1
        // (the lift out again, exactly: pieces of a pair have lifts of their own)
        const float drop = __uint_as_float((uint32_t)(127 - (int)lift) << 23);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            l.x += __shfl_xor_sync(0xffffffffu, l.x, o);
            l.y += __shfl_xor_sync(0xffffffffu, l.y, o);
        }
        l = fmul2(l, make_float2(drop, drop));
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    O[r][u][i] *= (i < 2 ? kCode : kCodeHigh) * drop;
        if (p.whole) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float sum = i == 0 ? l.x : l.y, inv = sum == 0.f ? 0.f : __fdividef(1.f, sum);
                if (2 * t + i < heads)
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const uint2 y = make_uint2(pack2<T>(O[r][0][i] * inv, O[r][0][i + 2] * inv),
                                                   pack2<T>(O[r][1][i] * inv, O[r][1][i + 2] * inv));
                        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) +
                                                   (((long long)p.s * a.num_q_heads + head0 + 2 * t + i) * D + 32 * r + 4 * g) * 2) = y;
                    }
            }
        } else {
            const bool is_first = off0 > 0;
            if (!is_first) {  // the last piece of the run: its copies are all in, and the ring is free
                copies_wait<0>();
                __syncwarp();
            }
            // (a pair that the CTA's last warp leaves open goes on in the next CTA)
            float *rec = is_first        ? sm.first[warp]
                         : warp == W - 1 ? P.record(2 * blockIdx.x + 1, GG::RECORD)
                                         : reinterpret_cast<float *>(sm.ring[warp][0]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int h = 2 * t + i;
                if (g == 0) {
                    const float sum = i == 0 ? l.x : l.y;
                    rec[h] = sum != 0.f ? fmaxf(i == 0 ? z0.x * unit.x : z0.y * unit.y, kNone) : kNone;
                    rec[8 + h] = sum;
                }
#pragma unroll
                for (int r = 0; r < R; ++r)
                    *reinterpret_cast<float4 *>(rec + 16 + h * D + 32 * r + 4 * g) =
                        make_float4(O[r][0][i], O[r][0][i + 2], O[r][1][i], O[r][1][i + 2]);
            }
            if (lane == 0) {
                const int pair = p.s * P.heads + p.h;
                if (is_first) {
                    sm.first_pair[warp] = pair;
                    sm.first_ends[warp] = p.ends;
                } else {
                    sm.last_pair[warp] = pair;
                }
            }
        }
    }
    copies_wait<0>();
    __syncthreads();

    // ---- join the CTA's cut pairs.  Chain -1 starts with warp 0's first record (a pair that
    // began in a CTA before), chain w with warp w's last one; the first records of the warps
    // behind it follow, up to one that goes to the pair's end.  Warp w joins chain w - 1.
    const bool has_first = lane < W && sm.first_pair[lane < W ? lane : 0] >= 0;
    const uint32_t open = __ballot_sync(0xffffffffu, lane < W && sm.last_pair[lane < W ? lane : 0] >= 0),
                   enders = __ballot_sync(0xffffffffu, has_first && sm.first_ends[lane]);
    const bool from_before = sm.first_pair[0] >= 0;
    const int opener = 31 - __clz(open);  // the last warp that leaves a pair open, or -1
    const bool goes_on = opener >= 0 && (enders >> (opener + 1)) == 0u;
    const uint32_t chains = open << 1 | (from_before ? 1u : 0u);  // bit w + 1: chain w
    const int chain = warp - 1;
    auto of_cta = [&](int slot, int i) {  // record i of a pair of several CTAs
        const int c0 = sm.first_cta[slot];
        return P.record(i == 0 ? 2 * c0 + 1 : 2 * (c0 + i), GG::RECORD);
    };
    // This CTA's record of the pair is written.  Each CTA counts itself, and the last to do so joins
    // them: a warp two of them, more the whole CTA.
    auto finish = [&](int slot, int pair) {
        const int n = sm.pieces[slot];
        __syncwarp();
        int last = 0;
        if (lane == 0) {  // what the warp wrote is out before its count, what others wrote is read behind theirs
            asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(last) : "l"(P.counters + pair) : "memory");
            last = last == n - 1;
            if (last)
                P.counters[pair] = 0;
        }
        last = __shfl_sync(0xffffffffu, last, 0);
        __syncwarp();
        if (!last)
            return;
        if (n > 2) {
            if (lane == 0)
                sm.to_join[slot] = pair;
            return;
        }
        Joined<D> r, behind;
        r.load(of_cta(slot, 0), lane);
        behind.load(of_cta(slot, 1), lane);
        r.add(behind);
        r.template put<T>(P, pair, lane);
    };
    if ((chains >> warp) & 1u) {
        const int pair = chain < 0 ? sm.first_pair[0] : sm.last_pair[chain];
        const uint32_t behind = chain < 0 ? enders : enders >> (chain + 1) << (chain + 1);
        const bool ends = behind != 0u;
        const int n = (ends ? __ffs(behind) - 1 : W - 1) - chain + (chain < 0 ? 0 : 1);
        Joined<D> r;
        r.join(n, lane, [&](int i) -> const float * {
            return chain < 0 ? sm.first[i] : i == 0 ? reinterpret_cast<const float *>(sm.ring[chain][0]) : sm.first[chain + i];
        });
        if (chain >= 0 && ends) {
            r.template put<T>(P, pair, lane);
        } else {
            const int slot = chain < 0 ? 0 : 1;
            r.keep(P.record(2 * blockIdx.x + slot, GG::RECORD), lane);
            finish(slot, pair);
        }
    }
    // the record that the last warp wrote itself is finished by a warp without a chain, if there is one
    const uint32_t idle = ~chains & ((1u << W) - 1u);
    if (opener == W - 1 && warp == (idle != 0u ? __ffs(idle) - 1 : W - 1))
        finish(1, sm.last_pair[W - 1]);
    if (!(from_before && sm.pieces[0] > 2) && !(goes_on && sm.pieces[1] > 2))
        return;

    // ---- pairs of more CTAs: the whole CTA joins them
    __syncthreads();
#pragma unroll 1
    for (int slot = 0; slot < 2; ++slot) {
        const int pair = sm.to_join[slot];
        if (pair < 0)
            continue;
        const int n = sm.pieces[slot], c0 = sm.first_cta[slot];
        // A thread merges four elements over every LANESth record as they come, four at a
        // time.  Record i: the first CTA's last slot, then the others' first ones.
        constexpr int LANES = GG::THREADS / GG::SLOTS;
        const int at = tid % GG::SLOTS, first = tid / GG::SLOTS, h = at / (D / 4);
        float top = kNone, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (first < LANES)
            for (int i = first; i < n; i += 4 * LANES) {
                float4 x[4];
                float mi[4], li[4], higher = top;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = i + k * LANES;
                    const float *rec = P.record(r == 0 ? 2 * c0 + 1 : 2 * (c0 + r), GG::RECORD);
                    const bool on = r < n;
                    mi[k] = on ? __ldcg(rec + h) : kNone;
                    li[k] = on ? __ldcg(rec + 8 + h) : 0.f;
                    x[k] = on ? __ldcg(reinterpret_cast<const float4 *>(rec + 16) + at) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    higher = fmaxf(higher, mi[k]);
                const float f0 = fast_exp2(top - higher);
                top = higher;
                sum *= f0;
                acc.x *= f0, acc.y *= f0, acc.z *= f0, acc.w *= f0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float f = fast_exp2(mi[k] - top);
                    sum = fmaf(f, li[k], sum);
                    acc.x = fmaf(f, x[k].x, acc.x), acc.y = fmaf(f, x[k].y, acc.y);
                    acc.z = fmaf(f, x[k].z, acc.z), acc.w = fmaf(f, x[k].w, acc.w);
                }
            }
        if constexpr (LANES > 1) {
            float4 *part = reinterpret_cast<float4 *>(sm.ring[0][0]);
            float2 *part_top = reinterpret_cast<float2 *>(part + (LANES - 1) * GG::SLOTS);
            if (first > 0) {
                part[(first - 1) * GG::SLOTS + at] = acc;
                part_top[(first - 1) * GG::SLOTS + at] = make_float2(top, sum);
            }
            __syncthreads();
            if (first == 0) {
                float higher = top;
#pragma unroll
                for (int k = 0; k < LANES - 1; ++k)
                    higher = fmaxf(higher, part_top[k * GG::SLOTS + at].x);
                const float f0 = fast_exp2(top - higher);
                sum *= f0;
                acc.x *= f0, acc.y *= f0, acc.z *= f0, acc.w *= f0;
#pragma unroll
                for (int k = 0; k < LANES - 1; ++k) {
                    const float2 y = part_top[k * GG::SLOTS + at];
                    const float4 x = part[k * GG::SLOTS + at];
                    const float f = fast_exp2(y.x - higher);
                    sum = fmaf(f, y.y, sum);
                    acc.x = fmaf(f, x.x, acc.x), acc.y = fmaf(f, x.y, acc.y);
                    acc.z = fmaf(f, x.z, acc.z), acc.w = fmaf(f, x.w, acc.w);
                }
            }
        }
        if (first == 0) {
            const int s = pair / P.heads, ph = pair - s * P.heads, kv = ph / P.subs, sub = ph - kv * P.subs;
            if (h < P.group - sub * 8) {
                const float inv = sum == 0.f ? 0.f : __fdividef(1.f, sum);
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) +
                                           (((long long)s * a.num_q_heads + kv * P.group + sub * 8 + h) * D + (at % (D / 4)) * 4) * 2) =
                    make_uint2(pack2<T>(acc.x * inv, acc.y * inv), pack2<T>(acc.z * inv, acc.w * inv));
            }
        }
        __syncthreads();
    }
}

template <typename T, int D>
cudaError_t launch(const Params &P, cudaStream_t stream)
{
    int sms = 0;
    cudaError_t e = current_sms(&sms);
    if (e != cudaSuccess)
        return e;
    const void *kern = (const void *)decode_q4_kernel<T, D>;
    static unsigned long long ready = 0;  // devices whose kernel has its shared memory
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !((__atomic_load_n(&ready, __ATOMIC_RELAXED) >> dev) & 1ull)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<D>));
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            __atomic_fetch_or(&ready, 1ull << dev, __ATOMIC_RELAXED);
    }
    // no more CTAs than the tables' rows could fill
    const long long most = (long long)P.a.num_seqs * P.heads *
                           ((((long long)P.a.max_blocks_per_seq << P.shift) + kChunk - 1) / kChunk + kPairCost);
    const int ctas = (int)std::min<long long>(std::min(sms, kMaxQ4Ctas), (most + Geo<D>::WARPS - 1) / Geo<D>::WARPS);
    Params p = P;
    void *args[] = {&p};
    return launch_early(kern, dim3(ctas), Geo<D>::THREADS, sizeof(Smem<D>), stream, args);
}

}  // namespace

bool q4_decode_fits(long long num_seqs, long long pairs, long long max_blocks, int block_size)
{
    return num_seqs * pairs * ((max_blocks * block_size + kChunk - 1) / kChunk + kPairCost) <= 0x7fffffffLL;
}

cudaError_t launch_decode_q4(const Q4DecodeArgs &a, cudaStream_t stream)
{
    Params P;
    P.a = a;
    P.group = a.num_q_heads / a.num_kv_heads;
    P.subs = (P.group + 7) / 8;
    P.heads = a.num_kv_heads * P.subs;
    P.shift = a.block_size == 4 ? 2 : a.block_size == 8 ? 3 : a.block_size == 16 ? 4 : 5;
    // a unit of the products has to be positive: q takes the scale's sign
    P.blocks = (uint32_t)std::min<long long>(a.num_blocks, 0x80000000LL);
    P.scale_log2 = std::fabs(a.scale) * 1.4426950408889634f;
    P.sign = a.scale < 0.f ? -1.f : 1.f;
    P.counters = a.counters;
    P.records = a.records;
    if (a.head_dim == 64)
        return a.dtype == NS_BF16 ? launch<BF16, 64>(P, stream) : launch<F16, 64>(P, stream);
    return a.dtype == NS_BF16 ? launch<BF16, 128>(P, stream) : launch<F16, 128>(P, stream);
}

}  // namespace ns
