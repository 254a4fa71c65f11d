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
// per group (the sums of x are one more product, with ones).  Products of a code and x are exact,
// sums are fp32, the scale is applied to a group's sum in fp32: the only rounding is y's.
#pragma once

#include "lscd_serve.h"
#include "lscd_serve_device.h"

namespace lscd {
namespace {

// The four words (8 values 16 + c) of one word of codes.
template <typename T>
__device__ __forceinline__ u32x4v unpack_codes(uint32_t w) {
    u32x4v r;
    if (T::bf) {  // 16 + c = 0x4180 | c << 3
        const uint32_t mask = 0x00780078u, base = 0x41804180u;
        r[0] = ((w >> 3) & mask) | base;
        r[1] = ((w >> 7) & mask) | base;
        r[2] = ((w << 1) & mask) | base;
        r[3] = (__builtin_amdgcn_alignbit(w, w, 11) & mask) | base;
    } else {  // 16 + c = 0x4C00 | c << 6
        const uint32_t mask = 0x03C003C0u, base = 0x4C004C00u;
        r[0] = (w & mask) | base;
        r[1] = ((w >> 4) & mask) | base;
        r[2] = ((w << 4) & mask) | base;
        r[3] = (__builtin_amdgcn_alignbit(w, w, 8) & mask) | base;
    }
    return r;
}
// 16 + c - (16 + z) for two codes, in float16; `less` = -(16 + z) twice.
__device__ __forceinline__ uint32_t take_off(uint32_t w, uint32_t less) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, w) + __builtin_bit_cast(half2v, less));
}

// 8 values of x from column k on, zeros from column K on.
__device__ __forceinline__ u32x4v load_x(const uint16_t* x, int k, int K) {
    struct __attribute__((packed, aligned(2))) Loose {
        uint32_t w[4];
    };
    u32x4v r = {0u, 0u, 0u, 0u};
    if (k + 8 <= K) {
        const Loose v = *(const Loose*)(x + k);  // rows need not be aligned
        r = u32x4v{v.w[0], v.w[1], v.w[2], v.w[3]};
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + i < K) r[i / 2] |= (uint32_t)x[k + i] << (16 * (i & 1));
    }
    return r;
}

}  // namespace
}  // namespace lscd
