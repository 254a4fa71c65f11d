// Paged cache of keys and values: tokens written into slots (quantised to e4m3 or kept in 16
// bits) and read back.
//
// Quantisation of one token's head vector x: e = least integer >= -126 with max |x| <= 448 * 2^e
// over the finite values (e = 0 where all are zero), code = e4m3(x * 2^-e), nearest with ties to
// even; the product is exact, so the code is the only rounding.  e4m3 is a floating format: a
// power of two as the scale costs none of its 4 significant bits, and code * 2^e is exact in the
// 16-bit types' normal range, so reading back rounds nothing there and the attention can use the codes
// as they are.  (A value within 2^-5 of the type's largest may become a code that stands for the next
// power of two: read back as an infinity, counted by the attention as the largest value.)
//
// Both directions move about 3 bytes a value once and compute next to nothing: bound by HBM, and
// by latency for the few tokens of a decoding step.  A vector of up to 128 channels is one group
// of 16 lanes (8 values, one 16-byte access of the 16-bit side and one 8-byte access of the codes
// each); the 16 groups of a workgroup take 16 consecutive tokens of one head, so their codes and
// their scales, which lie token after token inside a page, fill whole lines.
//
// Measured: 4095 tokens of 56 heads of 128 channels (178 MB both ways) written in 36.2 us and read back in
// 36.2 us, 4.9 TB/s (a plain copy reaches 5.2); 64 tokens of 96 heads written in 5.7 us, a call's latency.

#include "lscd_serve.h"
#include "lscd_serve_device.h"

namespace lscd {
namespace {

constexpr int kMoveThreads = 256;

// Lanes that hold one vector of `dim` channels, 8 each: the next power of two of dim / 8.
__host__ __device__ inline int group_lanes(int dim) { return dim <= 64 ? 8 : (dim <= 128 ? 16 : 32); }

// e of the scale 2^e for a vector whose largest finite magnitude is `most` (0: all zero):
// 448 = 1.75 * 2^8, so with most = m * 2^x (1 <= m < 2), e = x - 8 where m <= 1.75, else x - 7.
__device__ __forceinline__ int scale_exponent(float most) {
    const uint32_t b = __builtin_bit_cast(uint32_t, most);
    if (b == 0) return 0;
    const int x = (int)(b >> 23) - 127, e = (b & 0x7FFFFFu) <= 0x600000u ? x - 8 : x - 7;
    return e < -126 ? -126 : e;
}
__device__ __forceinline__ float power_of_two(int e) { return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23); }

// One vector of 8 values per lane to its codes.  An infinity or NaN is stored as NaN and left out of
// the scale.
template <typename T, int LANES>
__device__ __forceinline__ u32x2v quantise(u32x4v x, float* scale) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = T::low(x[i]);
        f[2 * i + 1] = T::high(x[i]);
    }
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = fabsf(f[i]);
        most = a < __builtin_inff() ? fmaxf(most, a) : most;
    }
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) most = fmaxf(most, __shfl_xor(most, d, 64));
    const int e = scale_exponent(most);
    *scale = power_of_two(e);
    const float inv = power_of_two(-e);
    u32x2v codes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int w = 0;
        w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h] * inv, f[4 * h + 1] * inv, w, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h + 2] * inv, f[4 * h + 3] * inv, w, true);
        uint32_t u = (uint32_t)w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (!(fabsf(f[4 * h + i]) < __builtin_inff())) u |= 0x7Fu << (8 * i);
        codes[h] = u;
    }
    return codes;
}

// blockIdx.x: 256 / LANES tokens, blockIdx.y: HEADS heads, blockIdx.z: keys or values.  Nothing orders the
// stores of one token against another's: no two may have one slot.
template <typename T, bool E4M3, int LANES, int HEADS>
__global__ __launch_bounds__(kMoveThreads) void cache_write_kernel(CacheMoveArgs a) {
    constexpr int kGroups = kMoveThreads / LANES;
    const int lane = threadIdx.x % LANES;
    const int64_t t = (int64_t)blockIdx.x * kGroups + threadIdx.x / LANES;
    const int z = blockIdx.z, d = lane * 8, h0 = blockIdx.y * HEADS;
    const int64_t slots = a.c.num_pages * a.c.page_size;
    const int64_t slot = t < a.T ? a.slots[t] : -1;
    const bool to = slot >= 0 && slot < slots;
    const bool on = to && d < a.c.head_dim;
    const uint16_t* in = (const uint16_t*)a.in[z] + (to ? t * a.stride[z] : 0) + d;
    u32x4v x[HEADS];
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
        x[i] = u32x4v{0u, 0u, 0u, 0u};
        if (on && h0 + i < a.c.heads) x[i] = *(const u32x4v*)(in + (int64_t)(h0 + i) * a.c.head_dim);
    }
    const int64_t page = to ? slot / a.c.page_size : 0, row = to ? slot % a.c.page_size : 0;
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
        const int64_t vec = (page * a.c.heads + h0 + i) * a.c.page_size + row;
        const bool here = on && h0 + i < a.c.heads;
        if (E4M3) {
            float scale;
            const u32x2v codes = quantise<T, LANES>(x[i], &scale);
            if (here) {
                *(u32x2v*)((uint8_t*)(z ? a.c.v : a.c.k) + vec * a.c.head_dim + d) = codes;
                if (lane == 0) (z ? a.c.v_scale : a.c.k_scale)[vec] = scale;
            }
        } else if (here) {
            *(u32x4v*)((uint16_t*)(z ? a.c.v : a.c.k) + vec * a.c.head_dim + d) = x[i];
        }
    }
}

template <typename T, bool E4M3, int LANES, int HEADS>
__global__ __launch_bounds__(kMoveThreads) void cache_read_kernel(CacheMoveArgs a) {
    constexpr int kGroups = kMoveThreads / LANES;
    const int lane = threadIdx.x % LANES;
    const int64_t t = (int64_t)blockIdx.x * kGroups + threadIdx.x / LANES;
    const int z = blockIdx.z, d = lane * 8, h0 = blockIdx.y * HEADS;
    if (t >= a.T || d >= a.c.head_dim) return;
    const int64_t slots = a.c.num_pages * a.c.page_size;
    const int64_t slot = a.slots[t];
    const bool from = slot >= 0 && slot < slots;
    const int64_t page = from ? slot / a.c.page_size : 0, row = from ? slot % a.c.page_size : 0;
    uint16_t* out = (uint16_t*)a.out[z] + t * a.stride[z] + d;
    u32x4v x[HEADS];
    u32x2v codes[HEADS];
    float scale[HEADS];
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
        const int64_t vec = (page * a.c.heads + h0 + i) * a.c.page_size + row;
        const bool here = from && h0 + i < a.c.heads;
        x[i] = u32x4v{0u, 0u, 0u, 0u};
        codes[i] = u32x2v{0u, 0u};
        scale[i] = 0.f;
        if (E4M3) {
            if (here) {
                codes[i] = *(const u32x2v*)((const uint8_t*)(z ? a.c.v : a.c.k) + vec * a.c.head_dim + d);
                scale[i] = (z ? a.c.v_scale : a.c.k_scale)[vec];
            }
        } else if (here) {
            x[i] = *(const u32x4v*)((const uint16_t*)(z ? a.c.v : a.c.k) + vec * a.c.head_dim + d);
        }
    }
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
        if (h0 + i >= a.c.heads) break;
        if (E4M3 && from) {
            x[i][0] = T::template from_e4m3<false>(codes[i][0], scale[i]);
            x[i][1] = T::template from_e4m3<true>(codes[i][0], scale[i]);
            x[i][2] = T::template from_e4m3<false>(codes[i][1], scale[i]);
            x[i][3] = T::template from_e4m3<true>(codes[i][1], scale[i]);
        }
        *(u32x4v*)(out + (int64_t)(h0 + i) * a.c.head_dim) = x[i];
    }
}

template <bool WRITE, typename T, bool E4M3, int LANES>
hipError_t move_lanes(CacheMoveArgs a, hipStream_t s) {
    constexpr int kGroups = kMoveThreads / LANES;
    // (a dimension of a grid has fewer than 2^32 threads; more are cut off without an error)
    constexpr int64_t kMost = ((int64_t)1 << 31) / kMoveThreads * kGroups;
    for (int64_t left = a.T; left > 0; left -= kMost) {
        a.T = left < kMost ? left : kMost;
        // four heads per thread keep four accesses in flight
        const dim3 grid((unsigned)((a.T + kGroups - 1) / kGroups), (unsigned)((a.c.heads + 3) / 4), 2);
        if (WRITE)
            cache_write_kernel<T, E4M3, LANES, 4><<<grid, kMoveThreads, 0, s>>>(a);
        else
            cache_read_kernel<T, E4M3, LANES, 4><<<grid, kMoveThreads, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        a.slots += kMost;
        for (int z = 0; z < 2; ++z)
            if (WRITE)
                a.in[z] = (const uint16_t*)a.in[z] + kMost * a.stride[z];
            else
                a.out[z] = (uint16_t*)a.out[z] + kMost * a.stride[z];
    }
    return hipSuccess;
}

template <bool WRITE, typename T>
hipError_t move_type(const CacheMoveArgs& a, hipStream_t s) {
    const bool e = a.c.type == LSCD_E4M3;
    switch (group_lanes(a.c.head_dim)) {
        case 8: return e ? move_lanes<WRITE, T, true, 8>(a, s) : move_lanes<WRITE, T, false, 8>(a, s);
        case 16: return e ? move_lanes<WRITE, T, true, 16>(a, s) : move_lanes<WRITE, T, false, 16>(a, s);
        default: return e ? move_lanes<WRITE, T, true, 32>(a, s) : move_lanes<WRITE, T, false, 32>(a, s);
    }
}

}  // namespace

hipError_t launch_cache_write(const CacheMoveArgs& a, int type, hipStream_t s) {
    return type == LSCD_F16 ? move_type<true, F16>(a, s) : move_type<true, BF16>(a, s);
}
hipError_t launch_cache_read(const CacheMoveArgs& a, int type, hipStream_t s) {
    return type == LSCD_F16 ? move_type<false, F16>(a, s) : move_type<false, BF16>(a, s);
}

}  // namespace lscd
