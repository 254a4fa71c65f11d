// Product of a few token vectors with a matrix of 4-bit codes: what its kernels share.
//
//   y[n][m] = sum over groups g of s[m][g] * sum over k in g of (c[m][k] - z[m][g]) x[n][k]
//
// The codes are unpacked to 16-bit floats in registers and multiplied on the matrix cores, tokens as
// the rows of A, 16 matrix rows as the columns of B, so that a lane holds results of one matrix row
// and its scale and zero point are one value each.  A code becomes the number 16 + c by placing its
// four bits at the top of the fraction of 16.0: one mask-and-or for two codes and a shift for most.
// float16: 16 + z is then taken off with one packed subtraction, exactly; bfloat16 has no packed
// arithmetic, so sums of (16 + c) x are kept per group and (16 + z) sum of x is taken off in fp32 once
// per group (the sums of x are one more product, with ones).  These numbers and ones are held 2^-12 times
// as large, and sums are multiplied by 2^12 when they are written: 128 products of up to 31 then stay below
// the largest x, whatever x is.
// Products of a code and x are exact, sums are fp32 and the scale is applied to a group's sum in fp32; y is
// rounded once to 16 bits.  What fp32 rounds is at most (K + 2 groups + 8) 2^-24 of the sum of the terms'
// magnitudes: |(c - z) x s| in float16, (32 + c + z) |x s| in bfloat16, where the difference is taken
// after summing.
#pragma once

#include "lscd_serve.h"
#include "lscd_serve_device.h"

namespace lscd {
namespace {

// What sums are multiplied by when they are written.
template <typename T>
constexpr float kUnit = T::bf ? 4096.f : 1.f;

// The four words (8 values 16 + c) of one word of codes.
template <typename T>
struct Unpack {
    const uint32_t mask, base;  // bfloat16: (16 + c) 2^-12 = 0x3B80 | c << 3; float16: 16 + c = 0x4C00 | c << 6
    __device__ __forceinline__ Unpack()
        : mask(scalar_constant(T::bf ? 0x00780078u : 0x03C003C0u)), base(vector_constant(T::bf ? 0x3B803B80u : 0x4C004C00u)) {}
    __device__ __forceinline__ u32x4v operator()(uint32_t w) const {
        if (T::bf)
            return u32x4v{(w >> 3 & mask) | base, (w >> 7 & mask) | base, (w << 1 & mask) | base,
                          (__builtin_amdgcn_alignbit(w, w, 11) & mask) | base};
        return u32x4v{(w & mask) | base, (w >> 4 & mask) | base, (w << 4 & mask) | base,
                      (__builtin_amdgcn_alignbit(w, w, 8) & mask) | base};
    }
};
// 16 + c - (16 + z) for two codes, in float16; `less` = -(16 + z) twice.
__device__ __forceinline__ uint32_t take_off(uint32_t w, uint32_t less) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, w) + __builtin_bit_cast(half2v, less));
}
// -(16 + z) twice: 0xCC00 | z << 6 in float16.
__device__ __forceinline__ uint32_t less_of(uint32_t z) { return (0xCC00u | z << 6) * 0x00010001u; }

// 8 values of x, whatever the alignment.
__device__ __forceinline__ u32x4v load_x(const uint16_t* x) {
    struct __attribute__((packed, aligned(2))) Loose {
        uint32_t w[4];
    };
    const Loose v = *(const Loose*)x;
    return u32x4v{v.w[0], v.w[1], v.w[2], v.w[3]};
}
// The same where many rows begin at odd multiples of 2 bytes: a 16-byte load costs a lane several times as
// much there as at a multiple of 4 (12288x4097 x 16 tokens: 31.7 us with such loads, 17.6 us so).  The
// aligned words that hold the values are loaded instead, and shifted when they are used.
struct OddX {
    u32x4v w;
    uint32_t next;
    __device__ __forceinline__ void load(const uint16_t* x) {
        const uint32_t half = (uint32_t)(uintptr_t)x & 2u;
        const uint32_t* p = (const uint32_t*)((uintptr_t)x - half);
        w = load_x((const uint16_t*)p);
        next = p[half ? 4 : 3];  // (never a word that holds none of the 8 values)
    }
    __device__ __forceinline__ u32x4v values(const uint16_t* x) const {
        const uint32_t by = ((uint32_t)(uintptr_t)x & 2u) * 8;
        return u32x4v{__builtin_amdgcn_alignbit(w[1], w[0], by), __builtin_amdgcn_alignbit(w[2], w[1], by),
                      __builtin_amdgcn_alignbit(w[3], w[2], by), __builtin_amdgcn_alignbit(next, w[3], by)};
    }
};
struct EvenX {
    u32x4v w;
    __device__ __forceinline__ void load(const uint16_t* x) { w = load_x(x); }
    __device__ __forceinline__ u32x4v values(const uint16_t*) const { return w; }
};
// Columns k to k + 7 of a row of fewer than 8: zeros behind its end.
__device__ __forceinline__ u32x4v load_x_end(const uint16_t* x, int k, int K) {
    u32x4v r = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < K) r[i / 2] |= (uint32_t)x[k + i] << (16 * (i & 1));
    return r;
}
// The same from the row's last 8 values `v`, loaded at column K - 8 where k > K - 8: s = k - (K - 8)
// values further on, zeros behind them.
__device__ __forceinline__ u32x4v shift_end(u32x4v v, int s) {
    if (s >= 8) v = u32x4v{0u, 0u, 0u, 0u};
    if (s > 0) {
        if (s & 4) v = u32x4v{v[2], v[3], 0u, 0u};
        if (s & 2) v = u32x4v{v[1], v[2], v[3], 0u};
        if (s & 1) v = u32x4v{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
    }
    return v;
}

// Scales and zero points of a lane's row for one unit (kinds of quant_kind).
template <typename T, int KIND>
struct Aux {
    static constexpr int kPer = KIND < 2 ? 1 : KIND;  // groups of a unit
    static constexpr int kBytes = KIND == 0 ? 2 : 4 * KIND;
    uint32_t w[kPer];
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, int voff, int soff) {
        if constexpr (KIND == 0) {
            w[0] = __builtin_amdgcn_raw_buffer_load_b16(rs, voff, soff, 0);
        } else if constexpr (KIND == 1) {
            w[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, voff, soff, 0);
        } else if constexpr (KIND == 2) {
            const u32x2v x = __builtin_amdgcn_raw_buffer_load_b64(rs, voff, soff, 0);
            w[0] = x[0];
            w[1] = x[1];
        } else {
            const u32x4v x = __builtin_amdgcn_raw_buffer_load_b128(rs, voff, soff, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = x[i];
        }
    }
    __device__ __forceinline__ float scale(int p) const { return T::low(w[p] & 0xFFFFu); }
    __device__ __forceinline__ uint32_t zero(int p) const { return KIND == 0 ? 8u : w[p] >> 16; }
};

}  // namespace
}  // namespace lscd
