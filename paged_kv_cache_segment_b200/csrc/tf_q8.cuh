// tf_q8.cuh - the 8-bit cache's number format on the device: codes (e4m3 or
// signed bytes) to f16 and bf16, scale bytes to floats, and a row's scale.
//
// An element is code * 2^(e - 127).  A code has at most 8 significant bits,
// so it is exact in f16, and code * 2^(e - 127) is exact in bf16 for every
// scale byte an append writes (27 to 249).
#pragma once

#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/tfserve.h"
#include "tf_common.cuh"

namespace tfp {

constexpr int kE8Bias = 127;
constexpr int kE8MinExp = -100;   // the smallest exponent an append writes
constexpr uint32_t kE8Nan = 255;  // the scale byte of a row that held a NaN or an infinity

// References of the softmax over an 8-bit cache, in base 2: one is set to
// kRefLift below the largest exponent seen and stays until an exponent passes
// kRefTop above it.  So a weight is at most 2^15, inside f16, and the largest at
// least 2^7: f16 hi + f16 lo hold 22 bits of a weight down to 2^-10 of the largest
// and, as f16 ends at 2^-24, 2^-32 of the largest below that.  (With the references
// at the largest exponent that floor is 2^-25: 32,000 keys just below it, behind one
// that weighs 1, lost 8e-4 of an output whose sum counted them.  A lift of 11 would
// put it at 2^-36, but the references then move oftener: a verify round of 1-16
// rows took 58.5 us a call instead of 54.8, a decode step 32.8 with either.)
constexpr float kRefLift = 7.f, kRefTop = 15.f;

// 2^(e - 127) (e = 0: the subnormal 2^-127), NaN for 255.
__device__ __forceinline__ float e8m0_f32(uint32_t e) {
    return __uint_as_float(e == kE8Nan ? 0x7fc00000u : (e == 0 ? 0x00400000u : e << 23));
}

// Four codes (a 32-bit word, lowest byte first) to f16 pairs (0, 1) and (2, 3).
template <int TYPE>
__device__ __forceinline__ void q8_to_f16(uint32_t w, uint32_t &p01, uint32_t &p23) {
    if constexpr (TYPE == TF_KV_E4M3) {
        asm("{\n\t.reg .b16 a, b;\n\t"
            "mov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(p01), "=r"(p23)
            : "r"(w));
    } else {
        // u = code + 128 as a byte under the exponent of 1,024: f16 1,024 + u, less 1,152
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p01) : "r"(a), "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p23) : "r"(b), "r"(0x64806480u));
    }
}

// Two keys' code pairs as a transposing ldmatrix leaves them (bytes: key a
// column d, key a column d + 1, key b column d, key b column d + 1) to the f16
// pairs (key a, key b) of column d and of column d + 1.
template <int TYPE>
__device__ __forceinline__ void q8_to_f16_pairs(uint32_t w, uint32_t &d0, uint32_t &d1) {
    if constexpr (TYPE == TF_KV_E4M3) {
        q8_to_f16<TYPE>(__byte_perm(w, 0u, 0x3120), d0, d1);
    } else {
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4240), b = __byte_perm(u, 0x64646464u, 0x4341);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d0) : "r"(a), "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d1) : "r"(b), "r"(0x64806480u));
    }
}

// Two floats -> packed f16x2 (round to nearest even); `lo` lands in bits 0..15.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// D = A * B + D, f16 inputs, fp32 accumulators (m16n8k16, row.col).
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with a D that starts at 0.
__device__ __forceinline__ void mma_f16_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t p) {
    __half2 h;
    *reinterpret_cast<uint32_t *>(&h) = p;
    return __half22float2(h);
}

// Eight codes times s (a power of two) as bf16: exact (see above).
template <int TYPE>
__device__ __forceinline__ uint4 q8_to_bf16x8(uint2 w, float s) {
    uint32_t p[4];
    q8_to_f16<TYPE>(w.x, p[0], p[1]);
    q8_to_f16<TYPE>(w.y, p[2], p[3]);
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = f16x2_to_f32(p[i]);
        r[i] = pack_bf16x2(f.x * s, f.y * s);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// The scale exponent of a row whose largest magnitude has these bf16 bits
// (finite, sign cleared): the smallest k >= -100 with amax <= Q * 2^k.  With
// amax = 1.f * 2^(E - 127) and Q = 1.75 * 2^8 (448) or 1.984375 * 2^6 (127),
// k is E - 127 less Q's exponent, and one more when 1.f is above Q's mantissa.
template <int TYPE>
__device__ __forceinline__ int q8_exponent(uint32_t amax) {
    const int E = (int)(amax >> 7), man = (int)(amax & 0x7fu);
    const int k = TYPE == TF_KV_E4M3 ? E - 127 - 8 + (man > 0x60 ? 1 : 0) : E - 127 - 6 + (man > 0x7e ? 1 : 0);
    return k > kE8MinExp ? k : kE8MinExp;
}

// Four values times s (a power of two that brings them into the code range), to
// codes (nearest, ties to even; lowest byte first).
template <int TYPE>
__device__ __forceinline__ uint32_t q8_encode4(float a, float b, float c, float d, float s) {
    if constexpr (TYPE == TF_KV_E4M3) {
        uint32_t r;
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
            "mov.b32 %0, {lo, hi};\n\t}"
            : "=r"(r)
            : "f"(a * s), "f"(b * s), "f"(c * s), "f"(d * s));
        return r;
    } else {
        // a * s is exact; adding 1.5 * 2^23 rounds it to an integer, whose low
        // byte is the sum's
        const float big = 12582912.f;
        const uint32_t x = __float_as_uint(fmaf(a, s, big)), y = __float_as_uint(fmaf(b, s, big));
        const uint32_t z = __float_as_uint(fmaf(c, s, big)), w = __float_as_uint(fmaf(d, s, big));
        return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
    }
}

}  // namespace tfp
