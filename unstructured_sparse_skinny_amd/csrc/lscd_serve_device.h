// Device-side building blocks of the serving operators: the two 16-bit types, matrix
// instructions on them, e4m3 and e2m1 conversion, wavefront helpers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lscd {
namespace {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef short s16x4v __attribute__((ext_vector_type(4)));
typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef float f32x16v __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));

constexpr int kRawBuffer = 0x00020000;  // raw buffer descriptor, word 3 (gfx9)
constexpr int kNoRow = 0x40000000;      // an offset outside every descriptor used here: reads give zero

// (by value: a bit cast of a vector's element in place takes the vector's first element)
__device__ __forceinline__ float as_float(uint32_t x) { return __builtin_bit_cast(float, x); }

// The two 16-bit types.  A pair of values travels as one 32-bit word.
struct F16 {
    static constexpr bool bf = false;
    static constexpr float kWeightBits = 7.f;  // softmax weights are held 2^7 times as large
    static constexpr uint32_t kTopScale = 0x43800000u;  // bits of 2^8, whose codes (up to 448) may pass the largest value
    static constexpr uint32_t kTopScale4 = 127u + 14u;  // the same of e2m1 codes (up to 6), as the exponent + 127
    static constexpr uint32_t kInfinity = 0x7C00u;
    __device__ static __forceinline__ float low(uint32_t w) { return (float)__builtin_bit_cast(half2v, w)[0]; }
    __device__ static __forceinline__ float high(uint32_t w) { return (float)__builtin_bit_cast(half2v, w)[1]; }
    __device__ static __forceinline__ uint32_t pack(float a, float b) {  // nearest, ties to even
        half2v h = {(_Float16)a, (_Float16)b};
        return __builtin_bit_cast(uint32_t, h);
    }
    // two e4m3 codes of one half of w, times the power of two `scale`
    template <bool HI>
    __device__ static __forceinline__ uint32_t from_e4m3(uint32_t w, float scale) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, HI));
    }
    // the two e2m1 codes of byte B of w, times the power of two `scale` (its exponent alone counts: sign and
    // fraction may be anything); NaN where the exponent is that of infinity
    template <int B>
    __device__ static __forceinline__ uint32_t from_e2m1(uint32_t w, float scale) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, B));
    }
    __device__ static __forceinline__ f32x4v mfma16(u32x4v a, u32x4v b, f32x4v c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8v, a), __builtin_bit_cast(half8v, b), c, 0,
                                                      0, 0);
    }
    __device__ static __forceinline__ f32x16v mfma32(u32x4v a, u32x4v b, f32x16v c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8v, a), __builtin_bit_cast(half8v, b), c, 0,
                                                      0, 0);
    }
    // sum of the pair's values, and s
    __device__ static __forceinline__ float add_pair(uint32_t w, float s) {
        const half2v one = {(_Float16)1.f, (_Float16)1.f};
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(half2v, w), one, s, false);
    }
    // whether either value of the pair is an infinity or NaN
    __device__ static __forceinline__ bool odd(uint32_t w) {
        return (w & 0x7C00u) == 0x7C00u || (w & 0x7C000000u) == 0x7C000000u;
    }
    // the pair with such values replaced by zero
    __device__ static __forceinline__ uint32_t finite(uint32_t w) {
        return w & (((w & 0x7C00u) == 0x7C00u ? 0u : 0xFFFFu) | ((w & 0x7C000000u) == 0x7C000000u ? 0u : 0xFFFF0000u));
    }
};
struct BF16 {
    static constexpr bool bf = true;
    static constexpr float kWeightBits = 0.f;
    static constexpr uint32_t kTopScale = 0x7B800000u;  // 2^120
    static constexpr uint32_t kTopScale4 = 127u + 126u;
    static constexpr uint32_t kInfinity = 0x7F80u;
    __device__ static __forceinline__ float low(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
    __device__ static __forceinline__ float high(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }
    __device__ static __forceinline__ uint32_t pack(float a, float b) {
        bf2v h = {(__bf16)a, (__bf16)b};
        return __builtin_bit_cast(uint32_t, h);
    }
    template <bool HI>
    __device__ static __forceinline__ uint32_t from_e4m3(uint32_t w, float scale) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, HI));
    }
    template <int B>
    __device__ static __forceinline__ uint32_t from_e2m1(uint32_t w, float scale) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, B));
    }
    __device__ static __forceinline__ f32x4v mfma16(u32x4v a, u32x4v b, f32x4v c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8v, a), __builtin_bit_cast(bf8v, b), c, 0, 0,
                                                       0);
    }
    __device__ static __forceinline__ f32x16v mfma32(u32x4v a, u32x4v b, f32x16v c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8v, a), __builtin_bit_cast(bf8v, b), c, 0, 0,
                                                       0);
    }
    __device__ static __forceinline__ float add_pair(uint32_t w, float s) {
        const bf2v one = {(__bf16)1.f, (__bf16)1.f};
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf2v, w), one, s, false);
    }
    __device__ static __forceinline__ bool odd(uint32_t w) {
        return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
    }
    // the pair with such values replaced by zero
    __device__ static __forceinline__ uint32_t finite(uint32_t w) {
        return w & (((w & 0x7F80u) == 0x7F80u ? 0u : 0xFFFFu) | ((w & 0x7F800000u) == 0x7F800000u ? 0u : 0xFFFF0000u));
    }
};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }  // v_exp_f32

// The pair with infinities replaced by the largest value of their sign.
template <typename T>
__device__ __forceinline__ uint32_t saturate(uint32_t w) {
    return w - ((w & 0x7FFFu) == T::kInfinity ? 1u : 0u) - ((w & 0x7FFF0000u) == T::kInfinity << 16 ? 0x10000u : 0u);
}

// a * b rounded, also where a sum follows.
__device__ __forceinline__ float product(float a, float b) {
#pragma clang fp contract(off)
    return a * b;
}

// x, in a way that the compiler does not see through.
__device__ __forceinline__ int opaque(int x) {
    asm("" : "+v"(x));
    return x;
}

// Constants in registers that the compiler does not see through: x & mask | base is one v_and_or_b32
// with them, two instructions with literals.
__device__ __forceinline__ uint32_t scalar_constant(uint32_t x) {
    asm("" : "+s"(x));
    return x;
}
__device__ __forceinline__ uint32_t vector_constant(uint32_t x) {
    asm("" : "+v"(x));
    return x;
}

// A value that is the same in all lanes, as a scalar.
__device__ __forceinline__ int64_t uniform(int64_t x) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x), hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// A barrier for data in LDS: waits for this wavefront's LDS accesses, not (as __syncthreads does) for
// its loads from memory, which may stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Largest of three; NaN if one is (v_maximum3_f32, which asks for no quieting of its operands).
__device__ __forceinline__ float max3(float a, float b, float c) {
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}

// The values of the lanes l and l ^ 32 (l and l ^ 16): the swap exchanges halves (odd and even
// quarters) of two registers.
__device__ __forceinline__ void both_halves(float x, float* a, float* b) {
    const uint32_t w = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    *a = as_float(r[0]);
    *b = as_float(r[1]);
}
__device__ __forceinline__ void both_quarters(float x, float* a, float* b) {
    const uint32_t w = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    *a = as_float(r[0]);
    *b = as_float(r[1]);
}
// max and sum over the two lanes l, l ^ 32 and over the four lanes l, l ^ 16, l ^ 32, l ^ 48
__device__ __forceinline__ float max_halves(float x) {
    float a, b;
    both_halves(x, &a, &b);
    return fmaxf(a, b);
}
__device__ __forceinline__ float sum_halves(float x) {
    float a, b;
    both_halves(x, &a, &b);
    return a + b;
}
// x summed over the lanes l, l ^ 32 in the lower half, y in the upper; over l, l ^ 16 in the even quarters, the odd ones
__device__ __forceinline__ float add_halves(float x, float y) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y), false, false);
    return as_float(r[0]) + as_float(r[1]);
}
__device__ __forceinline__ float add_quarters(float x, float y) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y), false, false);
    return as_float(r[0]) + as_float(r[1]);
}
__device__ __forceinline__ float max_quarters(float x) {
    float a, b;
    both_quarters(x, &a, &b);
    return max_halves(fmaxf(a, b));
}
__device__ __forceinline__ float sum_quarters(float x) {
    float a, b;
    both_quarters(x, &a, &b);
    return sum_halves(a + b);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, bytes, kRawBuffer);
}

}  // namespace
}  // namespace lscd
