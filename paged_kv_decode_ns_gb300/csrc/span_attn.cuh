// span_attn.cuh -- causal attention of query spans on the tcgen05 tensor cores:
// whole packed prompts over contiguous K/V rows, or new tokens over a q8_0
// paged cache.
//
// Row i of a span of n tokens over L keys sits at position L-n+i and sees the
// keys p <= L-n+i: out = sum_p 2^(z_p - m) v_p / sum_p 2^(z_p - m) with z in
// log2 units, one pass over the keys with a running reference m.
//
// Unit of work: (sequence, kv head, 2 QT query tokens), QT = 128 / G for groups
// of G query heads.  A unit is two query tiles of QT tokens x G heads (row r of a
// tile: token r / G, head r % G), so every K/V tile is loaded once for up to 256
// rows.  The units of a call are laid end to end, each as long as the keys it
// sees, and every CTA of a persistent grid takes an equal run of that line: long
// and short sequences, prompts and single tokens share the SMs evenly.  A unit
// that a cut falls into leaves its parts in fp32 records, and a second small
// kernel joins them.
//
// Warps of a CTA (512 threads):
//   0-3, 4-7  softmax of query tile 0 and 1: a thread owns a row.  It reads its row
//             of S from TMEM, and writes P (fp16) back to TMEM;
//   8-11      conversion: K and V tiles into the form that the products take;
//   12        producer: TMA copies of K and V tiles;
//   13, 14    issue S = Q K^T and O += P V of query tile 0 and 1;
//   15        walks the CTA's run of units, and copies their Q (fp16, or head_dim 128).
// The two tiles' softmax and products alternate by themselves: while one tile's
// scores are exponentiated, the other's products run.
//
// P is rounded to fp16 (11 bits) for both types: the products of a bf16 call
// would need P in two bf16 parts for the same accuracy, twice the value products.
// So V is fp16 too: a tile of bf16 values is scaled by a power of two, 2^-Ev.  Ev only
// rises along a unit, to 2^3 above what puts the largest value so far just below 2^15,
// and O is rescaled when it does (seldom, thanks to the 2^3): every value is off by at
// most 2^-36 of the largest so far, and P, 2^(z - m), does not depend on the size of the
// values.  (With exponents of 32 keys each in the exponent of P, one value 2^12 above the
// others took 12 bits of the weights of all keys but those 32.)
// q8_0 tiles are dequantised to fp16 in the same way, with Ek for K, by group of keys, in
// the score's scale: code times scale has up to 18 bits, so K, V and P each lose up to
// 2^-11 of themselves there.  An fp16 call over a q8_0 cache is then off by 4.2e-4 of its output,
// half of it the output's own rounding; two products for each would undo that at
// twice the tensor work.  Everything else (scores, sums, O) is fp32.
//
// What bounds it.  At head_dim 128 the tensor cores: 8192 fp16 tokens, 32 / 8 heads, 397 us,
// 1.38 PFLOP/s, 75% of the measured peak (394 to 411 us on different GPUs); bf16 470 us, its
// conversion of V on top.  At head_dim 64 the softmax: a pair of 128 x
// 128 tiles takes ~2370 clocks, against 1050 of products and 1024 of exponentials; two
// softmax warps a scheduler issue half of the time and wait on TMEM, barriers and
// each other's use of the exponential unit for the rest (135 us for 8192 fp16 tokens of
// 14 / 2 heads, 0.90 PFLOP/s; bf16 148 us, its conversion on top).  Short
// calls: launch, the plan, one unit's chain of copy, product, softmax, product and
// the join (four prompts of up to 200 tokens 10 us; 32 spans of drafts 19 us).
//
// Two softmax warpgroups a query tile (96 registers a thread) take 155 us where one
// takes 136: the row no longer fits the registers.  Tiles read from TMEM 32 columns at a
// time, the exponentials of the two tiles in turns (whole or half of them), a sleep
// between polls, a head start for one tile, and the first weights before the maximum
// were slower too or made no difference.
#pragma once

#include <algorithm>
#include <cstddef>

#include "ns_internal.h"
#include "tcgen05.cuh"

namespace ns {
namespace span {

constexpr int kRows = 128;       // rows of a query tile (MMA M)
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kRegs = 128;       // registers a thread at launch; the warpgroups then share them out:
constexpr int kSoftmaxRegs = 184, kConvertRegs = 72, kOtherRegs = 72;
static_assert(2 * kSoftmaxRegs + kConvertRegs + kOtherRegs <= 4 * kRegs, "the shares fit the launch's registers");
constexpr int kTileWarps = 4;    // softmax warps of a query tile
constexpr int kConvertWarp = 8, kProducerWarp = 12, kProductWarp = 13, kPlanWarp = 15;  // 13, 14: query tiles 0, 1
constexpr int kPanel = 128;      // bytes of a row of a panel: 64 elements, one swizzle span
constexpr int kUnits = 4;        // units announced ahead
constexpr int kMeta = 8;
constexpr int kMaxCtas = 160;    // grid, at most: the workspace has two records for each
constexpr float kTinyScale = 1.17549435e-38f;  // a score of -infinity times a scale of 0 would be NaN
// The reference m of a row is set kLift below a score (log2 units), and moves when a
// score passes that by more than kSlack: weights 2^(z - m) of up to 2^15 use fp16's range
// down to 2^-32 of the largest weight (half of its least step 2^-24, beside a weight of
// 2^7 or more).
constexpr float kLift = 7.0f, kSlack = 8.0f;
constexpr int kRoom = 3;   // the exponent of bf16 and q8_0 values is set for values 2^3 larger
constexpr int kLeast = 54; // and not below this field: a sum times 2^84 stays in fp32

template <int D, bool Q8>
struct Geo {
    static constexpr int KT = D == 64 ? 128 : 64;  // keys of a tile
    static constexpr int REG = D / 64;             // panels of a row
    static constexpr int TILE = REG * KT * kPanel; // bytes of a K or V tile
    static constexpr int GROUP = KT / 4;           // keys of a conversion warp
    static constexpr int STAGES = Q8 ? 3 : 4;
    static constexpr int RAW = Q8 ? 3 : 1;         // q8_0 tiles in flight (4 measured 2 to 4 % slower)
    // TMEM columns: S of tile t at KT t, O at 2 KT + D t, P at 2 KT + 2 D + KT / 2 t
    static constexpr int O = 2 * KT, P = 2 * KT + 2 * D;
    static_assert(P + KT <= 512, "tensor memory");
    // cost of a unit besides its keys (laying out Q, filling the pipe, the epilogue)
    // and the least cost that a CTA is given, in keys
    static constexpr int OVERHEAD = D == 128 ? 11 * KT / 2 : Q8 ? 5 * KT / 2 : 3 * KT;
    static constexpr int SHARE = OVERHEAD;  // at most one short unit a CTA while there are CTAs
    static constexpr int WHOLE = 4;  // units of so few key tiles are not cut
};

// Q comes by TMA as soon as the scores of the unit before are out, or by the softmax
// threads, a row each, between two units (1100 to 3500 clocks, of 2400 a tile).  The
// first against the second, in one run: head_dim 128, fp16, packed prompts 177 against 198
// us, 8192 tokens 407 against 422, four short prompts 13.8 against 15.4, bf16 packed 214
// against 222 and 8192 tokens 492 against 485; head_dim 64, fp16, packed 66.9 against 69.4,
// four short ones 9.4 against 10.3, mixed chunks over q8_0 32.1 against 32.4, 8192 tokens
// 134.8 against 134.2; bf16 at 64, packed 81.0 against 77.0, four short ones 10.7 against
// 10.4, 8192 tokens 146.7 against 149.1: many units gain there from the threads, since the
// two query tiles' softmax bounds the call and the later Q of one keeps them out of step.
constexpr bool q_by_tma(int D, bool bf16) { return D == 128 || !bf16; }

// A CTA's part of a unit: key tiles [t0, t1).
struct Unit {
    int s, h, i0, n, L;  // sequence, kv head, first token, span, keys
    int q0, k0;          // first rows of the sequence
    int t0, t1;          // t1 < 0: no more units
    int rec;             // record of a cut unit, or -1
};

// What a CTA tells the joining kernel.
struct alignas(16) Header {
    int own;               // it holds the first part of a cut unit (record 2 c + 1)
    int row0, tokens, h;   // that unit's first query row, its tokens, its kv head
    int last;              // and the last CTA with a part of it
    int head;              // it holds a later part of a unit (record 2 c)
    int pad[2];
};

constexpr size_t record_floats(int D) { return (size_t)2 * kRows * (D + 2); }
constexpr size_t header_bytes() { return kMaxCtas * sizeof(Header); }

struct Params {
    SpanAttnArgs a;
    int group, qt;
    float scale_log2;  // of |scale|
    int negate;        // scale < 0: the products take -Q
    Header *headers;
    float *records;
};

struct Maps {
    CUtensorMap q, k, v;  // k, v: contiguous rows only
};

template <int D, bool Q8>
struct alignas(1024) Smem {
    using GG = Geo<D, Q8>;
    uint8_t q[2][GG::REG * kRows * kPanel];
    uint8_t k[GG::STAGES][GG::TILE];
    uint8_t v[GG::STAGES][GG::TILE];
    uint8_t raw[GG::RAW][Q8 ? 2 * GG::KT * 64 + 2 * GG::KT * 4 : 16];  // codes of K, of V, scales of K, of V
    uint64_t raw_full[GG::RAW], raw_empty[GG::RAW];
    uint64_t v_full[GG::STAGES];
    uint64_t k_ready[GG::STAGES], v_ready[GG::STAGES], k_empty[GG::STAGES], v_empty[GG::STAGES];
    uint64_t q_ready[2], q_empty[2], s_full[2], s_free[2], p_full[2], pv_done[2];
    uint64_t u_full[kUnits], u_empty[kUnits];
    uint64_t top_full[2];
    Unit unit[kUnits], no_unit;
    float ev[GG::STAGES];                  // Ev of a stage's V
    alignas(16) uint32_t top[2][4];        // largest bf16 value of a tile, by conversion warp
    // q8_0: 2^Ek of a tile's K, by group of keys, and its blocks that were read.  A K
    // stage is free before the softmax has looked here; a ring of more than STAGES + 1 is not
    alignas(16) float ek[kMeta][4];
    uint32_t loaded[kMeta];
    uint32_t raw_loaded[GG::RAW];
    long long scan[kWarps];
    long long start_x, x0, x1, share, rest;
    int start_s;
    uint32_t tmem_base;
};

template <int D, bool Q8>
constexpr size_t smem_bytes()
{
    return sizeof(Smem<D, Q8>) + 1024;
}

// ---------------------------------------------------------------------------
// The line of work
// ---------------------------------------------------------------------------
struct Seq {
    int q0, n, k0, L;  // n = 0: nothing to do
};

template <bool Q8>
__device__ __forceinline__ Seq read_seq(const SpanAttnArgs &a, int s, unsigned *status)
{
    Seq r;
    r.q0 = a.query_start_loc[s];
    const int q1 = a.query_start_loc[s + 1];
    r.n = q1 - r.q0;
    unsigned bad = r.q0 < 0 || q1 < r.q0 || q1 > a.total_q_tokens ? NS_DEV_BAD_QUERY_SPAN : 0u;
    if (Q8) {
        r.k0 = 0;
        r.L = a.context_lens[s];
        if (r.L < r.n)
            bad |= NS_DEV_BAD_QUERY_SPAN;
        else if ((long long)r.L > (long long)a.max_blocks_per_seq * 16)
            bad |= NS_DEV_BAD_CONTEXT_LEN;
    } else {
        r.k0 = a.key_start_loc[s];
        const int k1 = a.key_start_loc[s + 1];
        r.L = k1 - r.k0;
        if (r.k0 < 0 || k1 < r.k0 || k1 > a.total_k_tokens)
            bad |= NS_DEV_BAD_QUERY_SPAN;
    }
    if (bad != 0) {
        if (status != nullptr)
            raise_status(status, bad);
        r.n = 0;
    }
    return r;
}

__device__ __forceinline__ long long quotient(long long a, long long b)  // a >= 0, b > 0
{
    return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Cost of the first u units of one kv head of a sequence (u < its units): unit v
// sees b + (v + 1) R keys.
__device__ __forceinline__ long long cost_before(long long u, long long each, long long R)
{
    return u * each + R * (u * (u + 1) / 2);
}

// The unit that position x of a kv head's line falls into, of `units`.
__device__ __forceinline__ int unit_at(long long x, int units, long long each, long long R)
{
    // u each + R u (u + 1) / 2 <= x, solved in fp32 and put right
    const float p = (float)each + 0.5f * (float)R, r = (float)R;
    const float g = 2.f * (float)x / (p + sqrtf(fmaf(2.f * r, (float)x, p * p)));
    int u = min(max((int)g, 0), units - 1);
    while (u > 0 && cost_before(u, each, R) > x)
        --u;
    while (u + 1 < units && cost_before(u + 1, each, R) <= x)
        ++u;
    return u;
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Key tiles that query tile t of a unit needs (keys up to its last token's own).
template <int KT>
__device__ __forceinline__ int tiles_of(const Unit &u, int t, int qt)
{
    const int first = u.i0 + t * qt;
    if (first >= u.n)
        return 0;
    const int keys = u.L - u.n + min(u.n, first + qt);
    return keys > 0 ? ceil_div(keys, KT) : 0;
}

// ---------------------------------------------------------------------------
// Helpers
// ---------------------------------------------------------------------------
__device__ __forceinline__ float pow2(int e)  // 2^e, -126 <= e <= 127
{
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Waits and arrivals of a whole warp, with as few branches as possible: a taken branch
// costs a lone warp some 25 clocks, and these are in everyone's inner loop.

// Bounded wait; the warp's lanes go on together, `ok` falls when the time is up.
__device__ __forceinline__ void warp_wait(uint64_t *bar, uint32_t parity, bool &ok)
{
    const bool done = mbar_try_wait(bar, parity);
    if (__builtin_expect(__any_sync(0xffffffffu, !done), 0))
        ok = __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0 && ok;
}

// Two or three waits at the price of one while all of them are over.
__device__ __forceinline__ void warp_wait(uint64_t *a, uint32_t pa, uint64_t *b, uint32_t pb, bool &ok)
{
    const bool da = mbar_try_wait(a, pa), db = mbar_try_wait(b, pb);
    if (__builtin_expect(__any_sync(0xffffffffu, !(da && db)), 0))
        ok = __all_sync(0xffffffffu, mbar_wait(a, pa) && mbar_wait(b, pb)) != 0 && ok;
}

// One arrival for the warp, through an elected lane.  What the lanes wrote to shared
// memory needs a __syncwarp before.
__device__ __forceinline__ void warp_arrive(uint64_t *bar)
{
    asm volatile(
        "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
        " @q mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(smem_addr(bar))
        : "memory");
}

// x 2^d, d <= 0: also where 2^d alone leaves fp32 (references of values 2^-60 and 2^60
// in size differ by that much).
__device__ __forceinline__ float times_pow2(float x, float d)
{
    return x * fast_exp2(fmaxf(d, -100.f)) * fast_exp2(fminf(d + 100.f, 0.f));
}

// The registers are read behind this point (after a wait for a TMEM load).
__device__ __forceinline__ void hold32(float *v)
{
    asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]));
    asm volatile("" : "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                 "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                 "+f"(v[30]), "+f"(v[31]));
}

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// The larger magnitudes of two pairs of values, with signs of no meaning; a NaN beside
// a number is left out.
__device__ __forceinline__ uint32_t larger_bf16(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t larger_f16(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t larger_bf16(uint4 w, uint32_t t)
{
    return larger_bf16(larger_bf16(larger_bf16(w.x, w.y), larger_bf16(w.z, w.w)), t);
}

// Largest magnitude of a pair.
__device__ __forceinline__ uint32_t top_of(uint32_t pair)
{
    return max(pair & 0x7fffu, (pair >> 16) & 0x7fffu);
}

// bf16 pair -> fp16 pair of the value times f.
__device__ __forceinline__ uint32_t bf16_to_f16(uint32_t w, float2 f)
{
    const float2 x = fmul2(unpack2<BF16>(w), f);
    return pack2<F16>(x.x, x.y);
}

__device__ __forceinline__ uint4 bf16_to_f16(uint4 w, float f)
{
    const float2 ff = make_float2(f, f);
    return make_uint4(bf16_to_f16(w.x, ff), bf16_to_f16(w.y, ff), bf16_to_f16(w.z, ff), bf16_to_f16(w.w, ff));
}

// Four q8_0 codes (a word) -> two fp16 pairs of code * d.  A code plus 128 is the
// low byte of the fp16 1024 + code + 128; the product rounds once.
__device__ __forceinline__ uint2 codes_to_f16(uint32_t w, __half2 d)
{
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    uint2 r;
    r.x = __byte_perm(u, 0x64646464u, 0x4140);
    r.y = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 *h = reinterpret_cast<__half2 *>(&r);
    h[0] = __hmul2(__hsub2(h[0], off), d);
    h[1] = __hmul2(__hsub2(h[1], off), d);
    return r;
}

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
template <typename T, int D, bool Q8>
__global__ void __launch_bounds__(kThreads, 1)
    span_attn_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params P)
{
    using GG = Geo<D, Q8>;
    constexpr int KT = GG::KT, REG = GG::REG, ST = GG::STAGES;
    constexpr bool BF = T::code == NS_BF16;
    constexpr bool SCALED = Q8 || BF;  // V tiles carry an exponent
    // The softmax reads that exponent with the scores, which then wait for the tile's V, or
    // only before it touches O.  The second is faster at head_dim 128, where the conversion
    // is behind (8192 bf16 tokens 480 us against 488, packed prompts 209 against 214), the
    // first at 64 (149 against 150, packed 76.9 against 77.1; drafts over q8_0 18.5 against 19.2).
    constexpr bool LATE = BF && D == 128;
    constexpr bool Q_TMA = q_by_tma(D, BF);
    extern __shared__ unsigned char smem_raw[];
    Smem<D, Q8> &sm = *reinterpret_cast<Smem<D, Q8> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const SpanAttnArgs &a = P.a;
    const int qt = P.qt, R = 2 * P.qt;

    if (!Q8 && threadIdx.x == kProducerWarp * 32) {
        tc::prefetch_tensormap(&maps.k);
        tc::prefetch_tensormap(&maps.v);
    }
    if (Q_TMA && threadIdx.x == kPlanWarp * 32)
        tc::prefetch_tensormap(&maps.q);
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&sm.k_ready[i], Q8 ? 4 : 1);
            mbar_init(&sm.v_full[i], 1);
            mbar_init(&sm.v_ready[i], 4);
            mbar_init(&sm.k_empty[i], 2);  // both tiles' products
            mbar_init(&sm.v_empty[i], 2);
        }
        for (int i = 0; i < GG::RAW; ++i) {
            mbar_init(&sm.raw_full[i], 1);
            mbar_init(&sm.raw_empty[i], 4);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sm.q_ready[t], Q_TMA ? 1 : kTileWarps);
            mbar_init(&sm.q_empty[t], 1);
            mbar_init(&sm.s_full[t], LATE ? 1 : SCALED ? 2 : 1);
            mbar_init(&sm.s_free[t], kTileWarps);
            mbar_init(&sm.p_full[t], kTileWarps);
            mbar_init(&sm.pv_done[t], 1);
        }
        for (int i = 0; i < 2; ++i)
            mbar_init(&sm.top_full[i], 4);
        for (int i = 0; i < kUnits; ++i) {
            mbar_init(&sm.u_full[i], 1);
            mbar_init(&sm.u_empty[i], kWarps - 1);  // one arrival a warp, but the walk's
        }
        sm.no_unit.t1 = -1;
        mbar_init_fence();
    }
    if (warp == kProductWarp) {
        tc::tmem_alloc(&sm.tmem_base, 512);
        tc::tmem_relinquish();
    }
    grid_dependency_wait();
    grid_launch_dependents();  // the joining kernel may be set up; it waits for this grid's end

    // ---- this CTA's run of the line: one warp costs up to 32 sequences, the whole
    // CTA more of them, a share for every thread
    {
        auto cost = [&](int s, unsigned *status) -> long long {
            const Seq q = read_seq<Q8>(a, s, status);
            if (q.n == 0)
                return 0;
            const long long units = ceil_div(q.n, R), each = GG::OVERHEAD + max(q.L - q.n, 0);
            return (cost_before(units - 1, each, R) + each + q.n) * a.num_kv_heads;
        };
        const bool few = a.num_seqs <= 32;
        const int per = few ? 1 : ceil_div(a.num_seqs, kThreads), who = few ? lane : (int)threadIdx.x;
        if (!few || warp == kPlanWarp) {
            const int s0 = min(a.num_seqs, who * per), s1 = min(a.num_seqs, s0 + per);
            long long mine = 0;
            for (int s = s0; s < s1; ++s)
                mine += cost(s, blockIdx.x == 0 ? a.status : nullptr);
            long long incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o)
                    incl += y;
            }
            long long before = incl - mine, total = __shfl_sync(0xffffffffu, incl, 31);
            if (!few) {
                if (lane == 31)
                    sm.scan[warp] = incl;
                __syncthreads();
                total = 0;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const long long x = sm.scan[w];
                    if (w < warp)
                        before += x;
                    total += x;
                }
            }
            const int ctas = (int)min((long long)gridDim.x, max(1LL, quotient(total, GG::SHARE)));
            const long long share = quotient(total, ctas), rest = total - share * ctas;
            const long long c = min((int)blockIdx.x, ctas), x0 = share * c + min(c, rest),
                            x1 = c < ctas ? x0 + share + (c < rest ? 1 : 0) : x0;
            if (who == 0) {
                sm.x0 = x0;
                sm.x1 = x1;
                sm.share = share;
                sm.rest = rest;
            }
            if (x0 < x1 && x0 >= before && x0 < before + mine) {
                long long x = before;
                int s = s0;
                for (;; ++s) {
                    const long long w = cost(s, nullptr);
                    if (x0 < x + w)
                        break;
                    x += w;
                }
                sm.start_s = s;
                sm.start_x = x;
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sm.tmem_base;
    bool ok = true;

    // The next announced unit (t1 < 0 at the end), in registers, or left in shared
    // memory until the warp hands it back.
    int unit_no = 0;
    auto wait_unit = [&]() -> const Unit & {
        const int i = unit_no % kUnits;
        warp_wait(&sm.u_full[i], (uint32_t)(unit_no / kUnits) & 1u, ok);
        if (!ok)
            return sm.no_unit;
        ++unit_no;
        return sm.unit[i];
    };
    auto release_unit = [&](int no) {
        __syncwarp();
        warp_arrive(&sm.u_empty[no % kUnits]);
    };
    auto next_unit = [&]() -> Unit {
        const Unit u = wait_unit();
        if (ok)
            release_unit(unit_no - 1);
        return u;
    };

    if (warp < 8) {
        // ------------------------------------------------------------ softmax
        regs_grow<kSoftmaxRegs>();
        const int t = warp >> 2;                        // query tile
        const int r = threadIdx.x & (kRows - 1);        // row == TMEM lane
        const int G = P.group;
        const int rt = r / G, rg = r - rt * G;          // token and head of the row
        const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_addr = lane_addr + t * KT, o_addr = lane_addr + GG::O + t * D,
                       p_addr = lane_addr + GG::P + t * (KT / 2);
        uint8_t *qs = sm.q[t] + r * kPanel;
        int count = 0;   // key tiles of this query tile so far
        int vtile = 0;   // key tiles of the CTA before this unit
        float row_scale = P.scale_log2;
        // Lay row r of the unit's query tile into shared memory.
        auto lay_q = [&](const Unit &u) {
            if (Q_TMA || min(u.t1, tiles_of<KT>(u, t, qt)) <= u.t0)
                return;
            const int tok = u.i0 + t * qt + rt;
            const bool on = rt < qt && tok < u.n;
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) +
                                                               (long long)(u.q0 + tok) * a.q_row_stride +
                                                               (long long)(u.h * G + rg) * D);
            uint4 w[D / 8];
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
                w[c] = on ? src[c] : make_uint4(0u, 0u, 0u, 0u);
            if (Q8 && BF) {
                // fp16 for the product with fp16 keys: the row's largest value goes
                // just below 2^15, its power of two into the score's scale
                uint32_t m = 0;
#pragma unroll
                for (int c = 0; c < D / 8; ++c)
                    m = larger_bf16(w[c], m);
                const int e = max((int)(top_of(m) >> 7), 15);
                const float f = pow2(141 - e);
#pragma unroll
                for (int c = 0; c < D / 8; ++c)
                    w[c] = bf16_to_f16(w[c], f);
                row_scale = P.scale_log2 * pow2(max(e - 141, -126));
            }
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
                *reinterpret_cast<uint4 *>(qs + (c >> 3) * (kRows * kPanel) + (((c & 7) ^ (r & 7)) << 4)) = w[c];
            fence_async_smem();
            __syncwarp();
            warp_arrive(&sm.q_ready[t]);
        };

        const Unit *now = &wait_unit();
        lay_q(*now);
        while (now->t1 >= 0) {
            const int t0 = now->t0, end = min(now->t1, tiles_of<KT>(*now, t, qt));
            // last key of the row, of the tile's first row
            const int low = now->L - now->n + now->i0 + t * qt;
            const int pos = rt < qt && now->i0 + t * qt + rt < now->n ? low + rt : -1;
            // rows are independent: 32 rows without a token need no weights
            const bool busy = __any_sync(0xffffffffu, pos >= 0 || (rt < qt && now->i0 + t * qt + rt < now->n));
            float m = -INFINITY, l = 0.f, o_ev = 0.f;  // O is in units of 2^(m + o_ev)
            for (int j = t0; ok && !busy && j < end; ++j, ++count) {
                warp_wait(&sm.s_full[t], (uint32_t)count & 1u, ok);
                warp_arrive(&sm.s_free[t]);
                warp_wait(&sm.pv_done[t], (uint32_t)(count - 1) & 1u, ok);
                warp_arrive(&sm.p_full[t]);
            }
            for (int j = t0; ok && busy && j < end; ++j, ++count) {
                warp_wait(&sm.s_full[t], (uint32_t)count & 1u, ok);
                tc::fence_after_sync();
                float sv[KT];
#pragma unroll
                for (int c = 0; c < KT; c += 32)
                    tc::tmem_ld32(s_addr + c, *reinterpret_cast<float(*)[32]>(&sv[c]));
                // scale of the scores, by group of keys, and exponent of the values; the
                // weights are summed by groups of four for all but fp16 values (bf16 packed
                // prompts 78.9 us, 80.2 in one)
                constexpr int NG = Q8 ? 4 : 1, NS = SCALED ? 4 : 1, GK = KT / NS;
                const int tile = vtile + j - t0;
                float sc[NG];
                float ev = SCALED && !LATE ? sm.ev[tile % ST] : 0.f;
                uint32_t loaded = 0xffffffffu;
                sc[0] = row_scale;
                if (Q8) {
                    const float4 k4 = *reinterpret_cast<const float4 *>(sm.ek[tile % kMeta]);
                    const float k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                    for (int g = 0; g < NG; ++g)
                        sc[g] = fmaxf(row_scale * k[g], kTinyScale);
                    loaded = sm.loaded[tile % kMeta];
                }
                tc::tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < KT; c += 32)
                    hold32(&sv[c]);
                tc::fence_before_sync();
                warp_arrive(&sm.s_free[t]);

                const int base = j * KT;
                if (base + KT - 1 > low) {
                    const int lim = pos - base;
#pragma unroll
                    for (int c = 0; c < KT; ++c)
                        sv[c] = c <= lim ? sv[c] : -INFINITY;
                }
                if (Q8 && (loaded & 0xffu) != 0xffu) {  // blocks that are not in the pool count for nothing
#pragma unroll
                    for (int c = 0; c < KT; ++c)
                        sv[c] = (loaded >> (c / 16)) & 1u ? sv[c] : -INFINITY;
                }
                float top = -INFINITY;
                {
                    float tm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < KT / 4; c += 2)
#pragma unroll
                        for (int e = 0; e < 4; ++e)  // a quarter of the columns each
                            tm[e] = max3(tm[e], sv[e * (KT / 4) + c], sv[e * (KT / 4) + c + 1]);
                    if (Q8) {
#pragma unroll
                        for (int g = 0; g < NG; ++g)
                            top = fmaxf(top, tm[g] * sc[g]);
                    } else {
                        top = fmaxf(fmaxf(tm[0], tm[1]), fmaxf(tm[2], tm[3])) * sc[0];
                    }
                }
                // the reference moves to a score that passes it by more than the slack
                const bool up = top > m + (kLift + kSlack);
                const float drop = up ? m - (top - kLift) : 0.f;
                l *= fast_exp2(drop);  // 0 at the first tile
                m = up ? top - kLift : m;
                const float ref = m > -INFINITY ? m : 0.f;
                uint32_t pk[KT / 2];
#pragma unroll
                for (int g = 0; g < NS; ++g) {
                    const float2 sc2 = make_float2(sc[g * NG / NS], sc[g * NG / NS]), nm2 = make_float2(-ref, -ref);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int c = g * GK; c < (g + 1) * GK; c += 2) {
                        const float2 z = ffma2(make_float2(sv[c], sv[c + 1]), sc2, nm2);
                        const float2 p = make_float2(fast_exp2(z.x), fast_exp2(z.y));
                        sum[(c >> 1) & 1] = fadd2(sum[(c >> 1) & 1], p);
                        pk[c >> 1] = pack2<F16>(p.x, p.y);
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                }

                // P is free, and O at rest, once the previous tile's value products are done
                if (LATE) {
                    warp_wait(&sm.pv_done[t], (uint32_t)(count - 1) & 1u, &sm.v_ready[tile % ST],
                              (uint32_t)(tile / ST) & 1u, ok);
                    ev = sm.ev[tile % ST];
                } else {
                    warp_wait(&sm.pv_done[t], (uint32_t)(count - 1) & 1u, ok);
                }
                tc::fence_after_sync();
                const bool moved = j > t0 && (up || (SCALED && ev != o_ev));
                const float fall = SCALED ? drop + (o_ev - ev) : drop;
                o_ev = ev;
                if (__any_sync(0xffffffffu, moved)) {
                    const float f = moved ? fast_exp2(fall) : 1.f;
#pragma unroll
                    for (int c = 0; c < D; c += 32) {
                        float ov[32];
                        tc::tmem_ld32(o_addr + c, ov);
                        tc::tmem_ld_wait();
                        hold32(ov);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            ov[e] *= f;
                        tc::tmem_st32(o_addr + c, ov);
                    }
                }
#pragma unroll
                for (int c = 0; c < KT / 2; c += 32)
                    tc::tmem_st32(p_addr + c, *reinterpret_cast<const uint32_t(*)[32]>(&pk[c]));
                tc::tmem_st_wait();
                tc::fence_before_sync();
                warp_arrive(&sm.p_full[t]);
            }
            const Unit &u = *now;
            vtile += u.t1 - t0;

            // the next unit's Q first, so that its scores are under way during the epilogue
            const int this_no = unit_no - 1;
            const Unit *next = &wait_unit();
            lay_q(*next);

            // ---- epilogue
            const int tok = u.i0 + t * qt + rt;
            const bool on = rt < qt && tok < u.n;
            const bool any = end > t0;
            if (any)
                warp_wait(&sm.pv_done[t], (uint32_t)(count - 1) & 1u, ok);
            tc::fence_after_sync();
            if (u.rec < 0) {
                // no weight: the row sees nothing; a NaN is passed on
                const float inv = SCALED ? pow2((int)o_ev) / l : 1.f / l;
                uint16_t *out = static_cast<uint16_t *>(a.out) +
                                ((long long)(u.q0 + tok) * a.num_q_heads + (long long)u.h * G + rg) * D;
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    float ov[32];
                    tc::tmem_ld32(o_addr + c, ov);
                    tc::tmem_ld_wait();
                    hold32(ov);
                    if (on && ok) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint4 w;
                            uint32_t *ww = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                ww[x] = any && l != 0.f ? pack2<T>(ov[e + 2 * x] * inv, ov[e + 2 * x + 1] * inv) : 0u;
                            *reinterpret_cast<uint4 *>(out + c + e) = w;
                        }
                    }
                }
            } else {
                // a part: unnormalised row, [D / 4][256 rows][4], and its reference and sum, which
                // take the exponent of the values in
                float *rec = P.records + (size_t)u.rec * record_floats(D);
                const int row = t * kRows + r;
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    float ov[32];
                    tc::tmem_ld32(o_addr + c, ov);
                    tc::tmem_ld_wait();
                    hold32(ov);
                    if (on && any) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(rec + ((size_t)((c + e) >> 2) * (2 * kRows) + row) * 4) =
                                make_float4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
                    }
                }
                if (on) {
                    rec[(size_t)D * 2 * kRows + row] = any ? m + o_ev : -INFINITY;
                    rec[(size_t)(D + 1) * 2 * kRows + row] = any ? (SCALED ? l * pow2(-(int)o_ev) : l) : 0.f;
                }
            }
            tc::fence_before_sync();
            release_unit(this_no);
            now = next;
        }
        if (!ok)
            raise_status(a.status, NS_DEV_WAIT_TIMEOUT);
    } else if (warp < kProducerWarp) {
        // ------------------------------------------------------------ conversion
        regs_shrink<kConvertRegs>();
        // a warp a group of keys; a lane a key (D 64) or one panel of a key
        const int group = warp - kConvertWarp;
        const int key = group * GG::GROUP + lane / REG, pan = lane % REG;
        const int panel = pan * (KT * kPanel) + key * kPanel;
        const int turn = (key & 7) ^ (pan << 2);  // order of the chunks: no two of eight lanes share a bank
        int tile = 0;
        for (Unit u = next_unit(); ok && u.t1 >= 0; u = next_unit()) {
            int most = 0;  // exponent field that the unit's values are laid out for
            auto raise = [&](int e) { most = e > most ? e + kRoom : most; };
            for (int j = u.t0; ok && j < u.t1; ++j, ++tile) {
                const int stage = tile % ST;
                const uint32_t par = (uint32_t)(tile / ST) & 1u;
                const bool live = j * KT + key < u.L;  // a row behind the last key is zero
                if (!Q8) {
                    warp_wait(&sm.v_full[stage], par, ok);
                    uint8_t *row = sm.v[stage] + panel;
                    if (BF) {
                        uint4 x[8];
                        uint32_t top = 0;
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            x[c] = live ? lds128(row + ((c ^ turn) << 4)) : make_uint4(0u, 0u, 0u, 0u);
                            top = larger_bf16(x[c], top);
                        }
                        top = __reduce_max_sync(0xffffffffu, top_of(top));
                        // the tile's largest value: the warps' own, exchanged
                        if (lane == 0)
                            sm.top[tile & 1][group] = top;
                        __syncwarp();
                        warp_arrive(&sm.top_full[tile & 1]);
                        warp_wait(&sm.top_full[tile & 1], (uint32_t)(tile >> 1) & 1u, ok);
                        const uint4 tops = lds128(sm.top[tile & 1]);
                        raise(max((int)(max(max(tops.x, tops.y), max(tops.z, tops.w)) >> 7), kLeast));
                        const float f = pow2(141 - most);
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            *reinterpret_cast<uint4 *>(row + ((c ^ turn) << 4)) = bf16_to_f16(x[c], f);
                        if (lane == 0 && group == 0)
                            sm.ev[stage] = (float)(most - 141);
                        fence_async_smem();
                    } else if (!live) {
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            *reinterpret_cast<uint4 *>(row + c * 16) = make_uint4(0u, 0u, 0u, 0u);
                        fence_async_smem();
                    }
                    __syncwarp();
                    warp_arrive(&sm.v_ready[stage]);
                } else {
                    const int rs = tile % GG::RAW;
                    warp_wait(&sm.raw_full[rs], (uint32_t)(tile / GG::RAW) & 1u, ok);
                    const uint8_t *raw = sm.raw[rs];
                    const uint32_t loaded = sm.raw_loaded[rs];
                    const bool have = live && ((loaded >> (key / 16)) & 1u);
                    const uint32_t *scales = reinterpret_cast<const uint32_t *>(raw + 2 * KT * 64);
                    const uint32_t d[2] = {have ? scales[key] : 0u, have ? scales[KT + key] : 0u};
                    // the tile's largest scale of V, four keys a lane (those that are there)
                    const int key4 = 4 * lane;
                    const int there = (loaded >> (key4 / 16)) & 1u ? u.L - j * KT - key4 : 0;
                    uint4 w4 = lds128(scales + KT + key4);
                    if (there < 4) {
                        w4.w = 0u;
                        w4.z = there > 2 ? w4.z : 0u;
                        w4.y = there > 1 ? w4.y : 0u;
                        w4.x = there > 0 ? w4.x : 0u;
                    }
                    const uint32_t vmag = larger_f16(larger_f16(w4.x, w4.y), larger_f16(w4.z, w4.w));
                    // code chunks in an order in which neither the reads (64-byte rows) nor the
                    // writes (swizzled 128-byte rows) of eight lanes share a bank
                    const int half = (key >> 1) & 3, first = (half << 1) ^ ((half >> 1) * 7);
                    uint4 code[2][4];
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            code[x][c] = lds128(raw + x * KT * 64 + key * 64 + ((c ^ first) << 4));
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        // the largest scale of these keys' K goes just below 2^8, its codes below
                        // 2^15; the unit's largest of V so far there or up to 2^kRoom lower
                        if (x == 1)
                            raise((int)(__reduce_max_sync(0xffffffffu, top_of(vmag)) >> 10));
                        const int e = x == 0 ? (int)(__reduce_max_sync(0xffffffffu, top_of(d[0])) >> 10) : most;
                        const float2 ds = unpack2<F16>(d[x]);
                        const float f = pow2(22 - e);
                        const __half2 dd[2] = {__float2half2_rn(ds.x * f), __float2half2_rn(ds.y * f)};
                        warp_wait(x == 0 ? &sm.k_empty[stage] : &sm.v_empty[stage], par ^ 1u, ok);
                        if (lane == 0) {
                            if (x == 0)
                                sm.ek[tile % kMeta][group] = pow2(e - 22);
                            else if (group == 0)
                                sm.ev[stage] = (float)(e - 22);
                            if (x == 0 && group == 0)
                                sm.loaded[tile % kMeta] = loaded;
                        }
                        uint8_t *row = (x == 0 ? sm.k[stage] : sm.v[stage]) + panel;
#pragma unroll
                        for (int c0 = 0; c0 < 4; ++c0) {
                            const int c = c0 ^ first;
                            const uint4 q = code[x][c0];
                            const __half2 s2 = c < 2 ? dd[0] : dd[1];
                            const uint2 e0 = codes_to_f16(q.x, s2), e1 = codes_to_f16(q.y, s2),
                                        e2 = codes_to_f16(q.z, s2), e3 = codes_to_f16(q.w, s2);
                            *reinterpret_cast<uint4 *>(row + (((2 * c) ^ (key & 7)) << 4)) = make_uint4(e0.x, e0.y, e1.x, e1.y);
                            *reinterpret_cast<uint4 *>(row + (((2 * c + 1) ^ (key & 7)) << 4)) = make_uint4(e2.x, e2.y, e3.x, e3.y);
                        }
                        fence_async_smem();
                        __syncwarp();
                        warp_arrive(x == 0 ? &sm.k_ready[stage] : &sm.v_ready[stage]);
                    }
                    warp_arrive(&sm.raw_empty[rs]);
                }
            }
        }
        if (!ok)
            raise_status(a.status, NS_DEV_WAIT_TIMEOUT);
    } else {
        regs_shrink<kOtherRegs>();
        if (warp == kProducerWarp) {
            // ------------------------------------------------------------ producer
            int tile = 0;
            for (Unit u = next_unit(); ok && u.t1 >= 0; u = next_unit()) {
                const int blocks = Q8 ? ceil_div(u.L, 16) : 0;
                for (int j = u.t0; ok && j < u.t1; ++j, ++tile) {
                    const int stage = tile % ST;
                    const uint32_t par = ((uint32_t)(tile / ST) & 1u) ^ 1u;
                    if (!Q8) {
                        if (lane == 0) {
                            const int row = u.k0 + j * KT;
                            ok = mbar_wait(&sm.k_empty[stage], par);
                            if (ok) {
                                mbar_arrive_expect_tx(&sm.k_ready[stage], GG::TILE);
#pragma unroll
                                for (int g = 0; g < REG; ++g)
                                    tc::tma_load_3d(sm.k[stage] + g * KT * kPanel, &maps.k, g * 64, u.h, row,
                                                    &sm.k_ready[stage]);
                                ok = mbar_wait(&sm.v_empty[stage], par);
                            }
                            if (ok) {
                                mbar_arrive_expect_tx(&sm.v_full[stage], GG::TILE);
#pragma unroll
                                for (int g = 0; g < REG; ++g)
                                    tc::tma_load_3d(sm.v[stage] + g * KT * kPanel, &maps.v, g * 64, u.h, row,
                                                    &sm.v_full[stage]);
                            }
                        }
                        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                    } else {
                        // lane i: block i / 4 of the tile, its codes of K, of V, scales of K, of V
                        const int rs = tile % GG::RAW;
                        const int b = lane >> 2, what = lane & 3, blk = j * (KT / 16) + b;
                        int phys = -1;
                        if (blk < blocks) {
                            phys = a.block_tables[(long long)u.s * a.max_blocks_per_seq + blk];
                            if (phys < 0 || (long long)phys >= a.num_blocks) {
                                raise_status(a.status, NS_DEV_BAD_BLOCK_ID);
                                phys = -1;
                            }
                        }
                        // blocks behind the last key are neither read nor missed
                        const uint32_t have = __ballot_sync(0xffffffffu, phys >= 0),
                                       fine = __ballot_sync(0xffffffffu, phys >= 0 || blk >= blocks);
                        if (lane == 0) {
                            ok = mbar_wait(&sm.raw_empty[rs], ((uint32_t)(tile / GG::RAW) & 1u) ^ 1u);
                            if (ok) {
                                uint32_t mask = 0;
                                for (int i = 0; i < KT / 16; ++i)
                                    mask |= ((fine >> (4 * i)) & 1u) << i;
                                sm.raw_loaded[rs] = mask;
                                mbar_arrive_expect_tx(&sm.raw_full[rs],
                                                      (uint32_t)(__popc(have) / 4) * 2u * (16u * 64u + 16u * 4u));
                            }
                        }
                        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                        if (ok && phys >= 0) {
                            const long long row = ((long long)phys * a.num_kv_heads + u.h) * 16;
                            uint8_t *raw = sm.raw[rs];
                            if (what < 2)
                                bulk_load(raw + what * KT * 64 + b * 1024,
                                          static_cast<const uint8_t *>(what == 0 ? a.k_codes : a.v_codes) + row * 64, 1024u,
                                          &sm.raw_full[rs]);
                            else
                                bulk_load(raw + 2 * KT * 64 + (what - 2) * KT * 4 + b * 64,
                                          static_cast<const uint8_t *>(what == 2 ? a.k_scales : a.v_scales) + row * 4, 64u,
                                          &sm.raw_full[rs]);
                        }
                    }
                }
            }
            // Never leave while copies may still land in this CTA's shared memory:
            // the last tile of every stage has arrived.
            if (lane == 0) {
                bool drained = true;
                const int depth = Q8 ? GG::RAW : ST;
                for (int i = 1; drained && i <= depth && i <= tile; ++i) {
                    const int x = tile - i;
                    if (Q8)
                        drained = mbar_wait(&sm.raw_full[x % GG::RAW], (uint32_t)(x / GG::RAW) & 1u);
                    else
                        drained = mbar_wait(&sm.k_ready[x % ST], (uint32_t)(x / ST) & 1u) &&
                                  mbar_wait(&sm.v_full[x % ST], (uint32_t)(x / ST) & 1u);
                }
                if (!drained || !ok)
                    raise_status(a.status, NS_DEV_WAIT_TIMEOUT);
            }
            __syncwarp();
        } else if (warp == kProductWarp || warp == kProductWarp + 1) {
            // ------------------------------------------------------------ products
            // One warp for each query tile: the scores of key tile j + 1 as soon as those
            // of j were read, then the values of j as soon as its weights are there.  The
            // whole warp walks the tiles; operands are warp-uniform.
            const int t = warp - kProductWarp;
            const uint32_t idesc_s = tc::idesc_f16(kRows, KT, BF && !Q8 ? 1 : 0, false) | (P.negate ? tc::kNegateA : 0u);
            const uint32_t idesc_o = tc::idesc_f16(kRows, D, 0, true);
            const uint64_t dk = tc::desc_sw128(0), dv = tc::desc_sw128_panels(0, KT * kPanel);
            auto uniform = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
            const uint32_t tm = uniform(tmem), q_lo = uniform((uint32_t)dk + (smem_addr(sm.q[t]) >> 4)),
                           k_lo = uniform((uint32_t)dk + (smem_addr(sm.k[0]) >> 4)),
                           v_lo = uniform((uint32_t)dv + (smem_addr(sm.v[0]) >> 4));
            uint32_t units = 0, count = 0;                // units and scores so far
            uint32_t ks = 0, kpar = 0, vs = 0, vpar = 0;  // stages of K and V
            auto next_stage = [](uint32_t &stage, uint32_t &parity) {
                const bool wrap = stage == ST - 1;
                stage = wrap ? 0 : stage + 1;
                parity ^= wrap ? 1u : 0u;
            };
            for (Unit u = next_unit(); ok && u.t1 >= 0; u = next_unit()) {
                const int n = uniform(u.t1 - u.t0),
                          mine = uniform(max(0, min(u.t1, tiles_of<KT>(u, t, qt)) - u.t0));
                if (mine > 0)
                    warp_wait(&sm.q_ready[t], units++ & 1u, ok);
                for (int i = 0; ok && i <= mine && mine > 0; ++i) {
                    if (i < mine) {
                        // S of tile i, once the scores before were read
                        warp_wait(&sm.k_ready[ks], kpar, &sm.s_free[t], (count - 1) & 1u, ok);
                        tc::fence_after_sync();
                        const uint32_t b_lo = uniform(k_lo + ks * (GG::TILE >> 4));
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            tc::mma_ss_warp(tm + t * KT, q_lo + (((kk >> 2) * (kRows * kPanel) + (kk & 3) * 32) >> 4),
                                            b_lo + (((kk >> 2) * (KT * kPanel) + (kk & 3) * 32) >> 4),
                                            (uint32_t)(dk >> 32), idesc_s, kk > 0);
                        tc::mma_commit_warp(&sm.s_full[t]);
                        tc::mma_commit_warp(&sm.k_empty[ks]);
                        if (Q_TMA && i == mine - 1)
                            tc::mma_commit_warp(&sm.q_empty[t]);
                        ++count;
                        if (SCALED && !LATE) {
                            // the softmax reads the exponents of this tile, too: they are in
                            // place when its V is
                            warp_wait(&sm.v_ready[ks], kpar, ok);
                            warp_arrive(&sm.s_full[t]);
                        }
                        next_stage(ks, kpar);
                    }
                    if (i > 0) {
                        // the values of tile i - 1, once its weights are there
                        const uint32_t done = (i < mine ? count - 2 : count - 1) & 1u;
                        warp_wait(&sm.v_ready[vs], vpar, &sm.p_full[t], done, ok);
                        tc::fence_after_sync();
                        const uint32_t b_lo = uniform(v_lo + vs * (GG::TILE >> 4));
                        const bool more = uniform(i > 1 ? 1u : 0u) != 0;
#pragma unroll
                        for (int kk = 0; kk < KT / 16; ++kk)
                            tc::mma_ts_warp(tm + GG::O + t * D, tm + GG::P + t * (KT / 2) + kk * 8,
                                            b_lo + ((kk * 16 * kPanel) >> 4), (uint32_t)(dv >> 32), idesc_o,
                                            kk > 0 || more);
                        tc::mma_commit_warp(&sm.pv_done[t]);
                        tc::mma_commit_warp(&sm.v_empty[vs]);
                        next_stage(vs, vpar);
                    }
                }
                // key tiles that this query tile has no rows for: their stages go back once
                // they are held, so that both query tiles count the same uses
                for (int i = mine; ok && i < n; ++i) {
                    warp_wait(&sm.k_ready[ks], kpar, &sm.v_ready[vs], vpar, ok);
                    warp_arrive(&sm.k_empty[ks]);
                    warp_arrive(&sm.v_empty[vs]);
                    next_stage(ks, kpar);
                    next_stage(vs, vpar);
                }
            }
            if (!ok && lane == 0)
                raise_status(a.status, NS_DEV_WAIT_TIMEOUT);
        } else {
            // ------------------------------------------------------------ the walk
            const long long x0 = sm.x0, x1 = sm.x1;
            auto owner = [&](long long x) {  // the CTA whose run position x falls into
                const long long wide = (sm.share + 1) * sm.rest;
                return (int)(x < wide ? quotient(x, sm.share + 1) : sm.rest + quotient(x - wide, sm.share));
            };
            Header head = {};
            int no = 0;
            auto announce = [&](const Unit &u) {
                const int i = no % kUnits;
                warp_wait(&sm.u_empty[i], ((uint32_t)(no / kUnits) & 1u) ^ 1u, ok);
                if (lane == 0 && ok) {
                    sm.unit[i] = u;
                    mbar_arrive(&sm.u_full[i]);
                }
                ++no;
            };
            // Q of both query tiles, each once the scores of the unit before are out.  The next
            // unit is announced first, so that its keys are not held up.
            int loads[2] = {0, 0};
            auto load_q = [&](const Unit &u) {
                if (lane == 0 && ok) {
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (min(u.t1, tiles_of<KT>(u, t, qt)) <= u.t0)
                            continue;
                        ok = ok && mbar_wait(&sm.q_empty[t], (uint32_t)(loads[t] - 1) & 1u);
                        if (!ok)
                            break;
                        ++loads[t];
                        mbar_arrive_expect_tx(&sm.q_ready[t], (uint32_t)(REG * P.group * qt * kPanel));
#pragma unroll
                        for (int g = 0; g < REG; ++g)
                            tc::tma_load_3d(sm.q[t] + g * kRows * kPanel, &maps.q, g * 64, u.h * P.group,
                                            u.q0 + u.i0 + t * qt, &sm.q_ready[t]);
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            };
            Unit behind = {};  // announced, its Q not yet asked for
            bool pending = false;
            if (x0 < x1) {
                int s = sm.start_s, h = 0, v = 0;
                long long xs = sm.start_x;  // of the sequence
                int held = -1;              // lane i holds sequence held + i
                Seq mine = {0, 0, 0, 0};
                bool first = true;
                for (; ok && s < a.num_seqs; ++s) {
                    if (held < 0 || s >= held + 32) {
                        held = s;
                        if (s + lane < a.num_seqs)
                            mine = read_seq<Q8>(a, s + lane, nullptr);
                        else
                            mine.n = 0;
                    }
                    Seq q;
                    q.q0 = __shfl_sync(0xffffffffu, mine.q0, s - held);
                    q.n = __shfl_sync(0xffffffffu, mine.n, s - held);
                    q.k0 = __shfl_sync(0xffffffffu, mine.k0, s - held);
                    q.L = __shfl_sync(0xffffffffu, mine.L, s - held);
                    if (q.n == 0)
                        continue;
                    if (xs >= x1)
                        break;
                    const int units = ceil_div(q.n, R);
                    const long long each = GG::OVERHEAD + max(q.L - q.n, 0);
                    const long long per_head = cost_before(units - 1, each, R) + each + q.n;
                    h = v = 0;
                    if (first) {
                        h = (int)quotient(x0 - xs, per_head);
                        v = unit_at(x0 - xs - h * per_head, units, each, R);
                        first = false;
                    }
                    for (; ok && h < a.num_kv_heads; ++h, v = 0)
                        for (; ok && v < units; ++v) {
                            const long long us = xs + h * per_head + cost_before(v, each, R);
                            if (us >= x1) {
                                h = a.num_kv_heads;
                                break;
                            }
                            const long long ue = us + each + (v + 1 < units ? (v + 1) * R : q.n);
                            Unit u;
                            u.s = s;
                            u.h = h;
                            u.i0 = v * R;
                            u.n = q.n;
                            u.L = q.L;
                            u.q0 = q.q0;
                            u.k0 = q.k0;
                            const int keys = q.L - q.n + min(q.n, u.i0 + R);
                            const int all = keys > 0 ? ceil_div(keys, KT) : 0;
                            auto cut = [&](long long x) {  // the key tile that position x falls before
                                if (all <= GG::WHOLE)
                                    return 2 * (x - us) > ue - us ? all : 0;
                                const long long d = (x - us - GG::OVERHEAD) / KT;
                                return (int)min(max(d, 0LL), (long long)all);
                            };
                            u.t0 = us >= x0 ? 0 : cut(x0);
                            u.t1 = ue <= x1 ? all : cut(x1);
                            if (u.t1 <= u.t0 && !(all == 0 && us >= x0))
                                continue;
                            u.rec = -1;
                            if (u.t0 > 0) {
                                u.rec = 2 * blockIdx.x;
                                head.head = 1;
                            } else if (u.t1 < all) {
                                u.rec = 2 * blockIdx.x + 1;
                                head.own = 1;
                                head.row0 = q.q0 + u.i0;
                                head.tokens = min(R, q.n - u.i0);
                                head.h = h;
                                head.last = owner(ue - 1);
                            }
                            announce(u);
                            if (Q_TMA && (no == 1 || pending))
                                load_q(pending ? behind : u);
                            pending = no > 1;
                            behind = u;
                        }
                    xs += per_head * a.num_kv_heads;
                }
            }
            Unit stop = {};
            stop.t1 = -1;
            if (ok)
                announce(stop);
            if (Q_TMA && pending)
                load_q(behind);
            if (lane == 0) {
                // the copies have landed before the CTA leaves
                for (int t = 0; t < 2; ++t)
                    if (loads[t] > 0)
                        ok = mbar_wait(&sm.q_ready[t], (uint32_t)(loads[t] - 1) & 1u) && ok;
                P.headers[blockIdx.x] = head;
                if (!ok)
                    raise_status(a.status, NS_DEV_WAIT_TIMEOUT);
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kProductWarp) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

// Joins the parts of cut units: 32 rows of one unit a block, a warp an eighth of
// the columns.  Parts come in the order of the keys, so results do not depend on
// which CTA ended first.  The header says which CTAs hold parts, so that everything
// else is read at once: two round trips to L2.
template <typename T, int D>
__global__ void __launch_bounds__(256) span_join_kernel(const __grid_constant__ Params P)
{
    constexpr int kPer = D / 32;  // float4 columns a thread
    constexpr int kBatch = 4;     // parts read at once
    grid_dependency_wait();
    grid_launch_dependents();
    const int c = blockIdx.x / 8, row = (blockIdx.x % 8) * 32 + (threadIdx.x & 31), warp = threadIdx.x >> 5;
    const Header hd = P.headers[c];
    const int t = row / kRows, r = row % kRows, rt = r / P.group;
    const int tok = t * P.qt + rt;
    if (!hd.own || rt >= P.qt || tok >= hd.tokens)
        return;
    float4 acc[kPer] = {};
    float sum = 0.f, top = -INFINITY;
    for (int i0 = c; i0 <= hd.last; i0 += kBatch) {
        float m[kBatch], l[kBatch];
        float4 o[kBatch][kPer];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int i = min(i0 + b, hd.last);
            const float *rec = P.records + (size_t)(i == c ? 2 * c + 1 : 2 * i) * record_floats(D);
            const bool part = i0 + b <= hd.last && (i == c || P.headers[i].head);
            m[b] = rec[(size_t)D * 2 * kRows + row];
            l[b] = rec[(size_t)(D + 1) * 2 * kRows + row];
#pragma unroll
            for (int x = 0; x < kPer; ++x)
                o[b][x] = *reinterpret_cast<const float4 *>(rec + ((size_t)(warp * kPer + x) * (2 * kRows) + row) * 4);
            if (!part)
                l[b] = 0.f;
        }
        float most = top;
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            most = l[b] != 0.f ? fmaxf(most, m[b]) : most;
        const float drop = top > -INFINITY ? top - most : 0.f, f0 = fast_exp2(drop);
        top = most;
        sum = times_pow2(sum, drop);
#pragma unroll
        for (int x = 0; x < kPer; ++x)
            acc[x] = make_float4(acc[x].x * f0, acc[x].y * f0, acc[x].z * f0, acc[x].w * f0);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (l[b] == 0.f)
                continue;
            const float f = fast_exp2(m[b] - top);
            sum += times_pow2(l[b], m[b] - top);
#pragma unroll
            for (int x = 0; x < kPer; ++x) {
                acc[x].x = fmaf(f, o[b][x].x, acc[x].x);
                acc[x].y = fmaf(f, o[b][x].y, acc[x].y);
                acc[x].z = fmaf(f, o[b][x].z, acc[x].z);
                acc[x].w = fmaf(f, o[b][x].w, acc[x].w);
            }
        }
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    uint16_t *out = static_cast<uint16_t *>(P.a.out) +
                    ((long long)(hd.row0 + tok) * P.a.num_q_heads + (long long)hd.h * P.group + (r - rt * P.group)) * D +
                    warp * kPer * 4;
#pragma unroll
    for (int x = 0; x < kPer; ++x)
        *reinterpret_cast<uint2 *>(out + 4 * x) =
            make_uint2(pack2<T>(acc[x].x * inv, acc[x].y * inv), pack2<T>(acc[x].z * inv, acc[x].w * inv));
}

// ---------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------
template <typename T, int D, bool Q8>
cudaError_t launch(const Maps &tm, const Params &P, int ctas, cudaStream_t stream)
{
    const long long max_keys = Q8 ? (long long)P.a.max_blocks_per_seq * 16 : P.a.total_k_tokens;
    // once for each device: the shared memory, and that the kernel has the registers
    // that its warpgroups share out (with fewer they would wait for ever)
    static unsigned long long ready = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !((__atomic_load_n(&ready, __ATOMIC_RELAXED) >> dev) & 1ull)) {
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, span_attn_kernel<T, D, Q8>);
        if (e == cudaSuccess && fa.numRegs != kRegs)
            e = cudaErrorInvalidValue;
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(span_attn_kernel<T, D, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)smem_bytes<D, Q8>());
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            __atomic_fetch_or(&ready, 1ull << dev, __ATOMIC_RELAXED);
    }
    // Programmatic dependents: the set-up of a kernel runs while the one before it on
    // the stream ends, and each waits for that one before it reads anything.
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes<D, Q8>();
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, span_attn_kernel<T, D, Q8>, tm, P);
    // no sequence has the keys of a unit that may be cut (the second launch costs
    // 3 us of a small call)
    if (e != cudaSuccess || max_keys <= Geo<D, Q8>::WHOLE * Geo<D, Q8>::KT)
        return e;
    cfg.gridDim = dim3(ctas * 8);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, span_join_kernel<T, D>, P);
}

}  // namespace span

cudaError_t launch_span_d64(bool bf16, const span::Maps &tm, const span::Params &P, int ctas, cudaStream_t stream);
cudaError_t launch_span_d128(bool bf16, const span::Maps &tm, const span::Params &P, int ctas, cudaStream_t stream);
cudaError_t launch_span_q8(bool bf16, const span::Maps &tm, const span::Params &P, int ctas, cudaStream_t stream);

}  // namespace ns
