// quantise.cuh -- the cache's 8- and 4-bit formats: 32 elements of a head row and
// one fp16 scale.  A thread holds eight consecutive elements, four neighbouring
// lanes a group; all lanes of a warp take part.
#pragma once

#include "ns_common.cuh"

namespace ns {

// q8_0: the scale d = max|x| / 127 and every code rint(x * (1/d)) (ties to even,
// clamped to +-127) are rounded to fp32 at each step, and d is stored as fp16
// (nearest even, saturating): the decisions the CPU oracle takes.
__device__ __forceinline__ void q8_quantize8(const float *x, uint2 &codes, uint16_t &d16)
{
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        amax = fmaxf(amax, fabsf(x[i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const float d = __fdiv_rn(amax, 127.f);
    const float inv = d > 0.f ? __fdiv_rn(1.f, d) : 0.f;
    uint32_t packed[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int code = max(-127, min(127, __float2int_rn(__fmul_rn(x[i], inv))));
        packed[i >> 2] |= (uint32_t)(code & 0xff) << (8 * (i & 3));
    }
    codes = make_uint2(packed[0], packed[1]);
    d16 = __half_as_ushort(__float2half_rn(fminf(d, 65504.f)));
}

// q4_0: with m the element of largest magnitude (of +a and -a the positive one), the
// step is d = -m / 8, stored as fp16 (nearest even, saturating); code = min(15,
// floor(x * (1/d) + 8.5)), rounded to fp32 at each step, stands for fp16(d) * (code - 8).
// So m itself is code 0, and the range reaches 7 steps on the other side.  A step that
// fp16 rounds to 0 makes every code 8 (value 0; 1/d would leave fp32); a group that holds
// an infinity or NaN gets the scale NaN, so that it shows wherever the group is read.
// Eight codes are a word, element i in bits 4 i .. 4 i + 3.
__device__ __forceinline__ void q4_quantize8(const float *x, uint32_t &codes, uint16_t &d16)
{
    float hi = -INFINITY, lo = INFINITY;
    bool fine = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        hi = fmaxf(hi, x[i]);
        lo = fminf(lo, x[i]);
        fine = fine && fabsf(x[i]) < INFINITY;  // false for NaN
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    }
    const uint32_t all = __ballot_sync(0xffffffffu, fine);
    fine = ((all >> (threadIdx.x & 28u)) & 15u) == 15u;
    const float d = -0.125f * (hi >= -lo ? hi : lo);
    const __half s = __float2half_rn(fminf(fmaxf(d, -65504.f), 65504.f));
    d16 = fine ? __half_as_ushort(s) : (uint16_t)0x7fffu;
    const bool zero = !fine || __heq(s, __ushort_as_half(0));
    const float inv = zero ? 0.f : __fdiv_rn(1.f, d);
    codes = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float y = zero ? 8.f : __fadd_rn(__fmul_rn(x[i], inv), 8.5f);
        codes |= (uint32_t)min(15, max(0, __float2int_rd(y))) << (4 * i);
    }
}

// Eight q4_0 codes (a word) times d, as fp16.  code - 8 is exact in either type that the product
// is taken in, so it rounds once: a code in the low bits of an fp16 1024 (an fp32 2^23), less that and
// 8, is code - 8.
__device__ __forceinline__ uint4 q4_halves(uint32_t w, __half2 d)
{
    const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
    const uint32_t a = __byte_perm(even, odd, 0x5140), b = __byte_perm(even, odd, 0x7362);  // elements 0-3, 4-7
    const __half2 off = __half2half2(__ushort_as_half(0x6408));  // 1032
    uint4 r = make_uint4(__byte_perm(a, 0x64646464u, 0x4140), __byte_perm(a, 0x64646464u, 0x4342),
                         __byte_perm(b, 0x64646464u, 0x4140), __byte_perm(b, 0x64646464u, 0x4342));
    __half2 *h = reinterpret_cast<__half2 *>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = __hmul2(__hsub2(h[i], off), d);
    return r;
}

// Eight codes and their step (fp16 bits) -> eight elements.
template <typename T>
__device__ __forceinline__ uint4 q4_elements(uint32_t w, uint16_t d16);

template <>
__device__ __forceinline__ uint4 q4_elements<F16>(uint32_t w, uint16_t d16)
{
    return q4_halves(w, __half2half2(__ushort_as_half(d16)));
}

template <>
__device__ __forceinline__ uint4 q4_elements<BF16>(uint32_t w, uint16_t d16)
{
    const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
    const float d = __half2float(__ushort_as_half(d16));
    auto element = [&](uint32_t codes, int i) {
        uint32_t x;
        asm("prmt.b32 %0, %1, %2, %3;" : "=r"(x) : "r"(codes), "r"(0x4b000000u), "r"(0x7550u + i));
        return d * (__uint_as_float(x) - 8388616.f);
    };
    return make_uint4(pack2<BF16>(element(even, 0), element(odd, 0)), pack2<BF16>(element(even, 1), element(odd, 1)),
                      pack2<BF16>(element(even, 2), element(odd, 2)), pack2<BF16>(element(even, 3), element(odd, 3)));
}

}  // namespace ns
