// act8.cuh -- the 8-bit form of kept activations (gg.h, "activations kept in 8 bits"):
// blocks of 32 columns of a row share a power-of-two scale 2^(s - 127), codes are int8
// or e4m3.  Scaling by a power of two is exact, so every routine here gives the same
// bits for the same values, whichever kernel it runs in.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace gg {

constexpr int kActBlock = 32;  // columns that share a scale
constexpr int kActNaN = 255;   // scale byte of a block that is not finite

__host__ __device__ constexpr int64_t act8_blocks(int64_t cols) { return (cols + kActBlock - 1) / kActBlock; }
__host__ __device__ constexpr int64_t act8_code_pitch(int64_t cols) { return kActBlock * act8_blocks(cols); }
__host__ __device__ constexpr int64_t act8_scale_pitch(int64_t cols) { return 4 * ((act8_blocks(cols) + 3) / 4); }

// Largest |x| so far and another; a NaN stays (as the pattern 0x7fffffff, above infinity's).
__device__ __forceinline__ float amax_nan(float m, float x) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(x)));
    return r;
}

// Scale byte of a block: e = exponent of amax / M rounded up to a power of two.  The
// mantissas of M = 127 (1.984375 2^6) and 448 (1.75 2^8) are exact, so a carry out of
// the mantissa field tells amax's above M's.
template <int FMT>
__device__ __forceinline__ uint32_t act8_scale(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int s = static_cast<int>((b + (FMT == GG_ACT8_INT8 ? 0x1FFFFu : 0x1FFFFFu)) >> 23) -
                  (FMT == GG_ACT8_INT8 ? 6 : 8);
    return b >= 0x7F000000u ? kActNaN : static_cast<uint32_t>(max(s, 10));
}
// 2^(127 - s), and 2^(s - 127) (NaN for s = 255).
__device__ __forceinline__ float act8_inverse(uint32_t s) { return __uint_as_float((254u - s) << 23); }
__device__ __forceinline__ float act8_factor(uint32_t s) {
    return __uint_as_float((s << 23) | (s == kActNaN ? 0x400000u : 0u));
}

// Four codes (the first in the low byte) of values times inv.
template <int FMT>
__device__ __forceinline__ uint32_t act8_code4(float a, float b, float c, float d, float inv) {
    if constexpr (FMT == GG_ACT8_INT8) {
        // adding 1.5 2^23 rounds half to even and leaves the integer in the low byte
        const float k = 12582912.0f;
        const uint32_t x = __float_as_uint(fmaf(a, inv, k)), y = __float_as_uint(fmaf(b, inv, k));
        const uint32_t z = __float_as_uint(fmaf(c, inv, k)), w = __float_as_uint(fmaf(d, inv, k));
        return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
    } else {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b * inv), "f"(a * inv));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d * inv), "f"(c * inv));
        return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
    }
}

// The four values that a word of codes stands for, f = act8_factor(s).
template <int FMT>
__device__ __forceinline__ void act8_value4(uint32_t w, float f, float (&v)[4]) {
    if constexpr (FMT == GG_ACT8_INT8) {
        // (conversions of single bytes: bytes put under 2^23's exponent by permutations, one
        // an element, took the kept activation's backward 474 us in place of 362)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i))) * f;
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t h;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w >> (16 * i))));
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h));
            v[2 * i] = p.x * f;
            v[2 * i + 1] = p.y * f;
        }
    }
}

// Whether [a, a + an) and [b, b + bn) share a byte (never where one is absent).
inline bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && an > 0 && bn > 0 && x < y + static_cast<uint64_t>(bn) && y < x + static_cast<uint64_t>(an);
}
// A tensor of a call; `row`: the bytes of a row where row t is read or written for token t
// alone, 0 for all others.
struct Span {
    const void* at;
    int64_t bytes;
    int64_t row = 0;
};
// Whether an output shares a byte with an input or with another output.  An output of rows may
// be an input of rows as long (each is read before it is written, by the CTA that writes it).
template <int N, int M>
inline bool outputs_overlap(const Span (&out)[N], const Span (&in)[M]) {
    for (int i = 0; i < N; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].at, out[i].bytes, out[j].at, out[j].bytes)) return true;
        for (int j = 0; j < M; ++j) {
            if (out[i].row && out[i].at == in[j].at && out[i].row == in[j].row) continue;
            if (overlap(out[i].at, out[i].bytes, in[j].at, in[j].bytes)) return true;
        }
    }
    return false;
}

// x / d for x < 2^31 and a launch constant d: a multiplication and a shift.
struct FastDiv {
    uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
    uint32_t s = 0;
    while ((uint64_t(1) << s) < d) ++s;
    return FastDiv{d, static_cast<uint32_t>(((uint64_t(1) << (32 + s)) + d - 1) / d - (uint64_t(1) << 32)), s};
}
__device__ __forceinline__ uint32_t operator/(uint32_t x, const FastDiv& q) {
    return (__umulhi(x, q.mul) + x) >> q.shift;
}

}  // namespace gg
