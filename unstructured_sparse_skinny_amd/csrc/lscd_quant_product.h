// The product kernels of matrices of 4-bit codes (see lscd_quant.h for the arithmetic); compiled once
// per 16-bit type.
#pragma once

#include "lscd_quant.h"

namespace lscd {
namespace {

constexpr int kQuantThreads = 64 * kQuantWaves;

template <typename T>
__device__ __forceinline__ u32x4v ones_of() {
    static_assert(T::bf, "float16 needs no sums of x");
    const uint32_t w = 0x39803980u;  // 2^-12
    return u32x4v{w, w, w, w};
}

// Instructions that may cross the scheduling barriers below: arithmetic and matrix products.
constexpr int kFreeOrder = 0xE;

// A workgroup's row tiles as one buffer: unit u of its tile r begins (r * units + u) KB into it.
// (Offsets of lanes that are off lie outside it: no traffic, zeros.)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_buffer(const void* p, int64_t tile, int tiles, int64_t bytes) {
    const int64_t at = uniform((int64_t)(uintptr_t)p + tile * bytes);
    return buffer_of((const void*)(uintptr_t)at, __builtin_amdgcn_readfirstlane((int)(tiles * bytes)));
}

// Up to 16 tokens.  One workgroup: RT row tiles and one of a.splits ranges of units, which its eight
// wavefronts split further: each streams its own units of all RT tiles (one contiguous KB of codes
// per tile and unit) with x straight from the caches, kAhead units in flight, and needs no barrier
// until the sums are joined through LDS.  x costs 4 KB per unit of a wavefront for 16 tokens (less for
// fewer: lanes past N repeat a token, the same lines), against RT KB of codes.  Bound by the reading of
// the codes where the matrix is large (12288x49152 in groups of 128, one token: 54.5 us, 5.8 TB/s;
// 28672x7168 x 16 tokens: 23.0 us, 4.6 TB/s), by x from the caches for 16 tokens and few rows, and by a
// launch's latency where it is small (1024x1024 x 1: 5 us).
template <typename T, int KIND, int RT, typename X>
__global__ __launch_bounds__(kQuantThreads, 2) void quant_few_kernel(QuantArgs a) {
    using A = Aux<T, KIND>;
    constexpr int kAhead = quant_ahead(RT, KIND);
    const Unpack<T> unpack;
    __shared__ float sh[kQuantWaves][16][RT * 16 + 1];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4;
    const int rt0 = blockIdx.x * RT, parts = kQuantWaves * a.splits, part = blockIdx.y * kQuantWaves + wave;
    const int u0 = (int)((int64_t)a.units * part / parts), u1 = (int)((int64_t)a.units * (part + 1) / parts);
    const int have = min(RT, a.tiles - rt0);
    const auto cb = tile_buffer(a.codes, rt0, have, (int64_t)a.units * 1024);
    const auto ab = tile_buffer(a.aux, rt0, have, (int64_t)a.units * kQuantRows * A::kBytes);
    const int token = (lane & 15) < a.N ? lane & 15 : a.spare;
    const uint16_t* xp = a.x + token * a.ldx;
    const int whole = a.K / kQuantUnit;  // the last unit of a row may not be full
    const int last = a.K - 8;            // a row's last 8 values stand in for what reaches past its end

    f32x4v acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = f32x4v{0.f, 0.f, 0.f, 0.f};
    u32x4v c[kAhead][RT];
    X loaded[kAhead][4];
    A aux[kAhead][RT];
    auto load = [&](int i, int u) {
        const bool on = u < u1;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const bool here = on && r < have;  // (the scalar offset is not part of the bounds check)
            const int unit = here ? r * a.units + u : 0;
            c[i][r] = __builtin_amdgcn_raw_buffer_load_b128(cb, here ? lane * 16 : kNoRow, unit * 1024, 2);
            aux[i][r].load(ab, here ? (lane & 15) * A::kBytes : kNoRow, unit * (kQuantRows * A::kBytes));
        }
    };
    auto load_tokens = [&](int i, int u) {
        const int k = min(u, u1 - 1) * kQuantUnit + 8 * g;
#pragma unroll
        for (int s = 0; s < 4; ++s) loaded[i][s].load(xp + min(k + 32 * s, last));
    };
    auto tokens = [&](int i, int u, u32x4v* x) {
        const int k = u * kQuantUnit + 8 * g;
#pragma unroll
        for (int s = 0; s < 4; ++s) x[s] = loaded[i][s].values(xp + min(k + 32 * s, last));
        if (u == whole)
#pragma unroll
            for (int s = 0; s < 4; ++s) x[s] = shift_end(x[s], k + 32 * s - last);
    };
    auto multiply = [&](int i, const u32x4v* x) {
        const f32x4v none = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int p = 0; p < A::kPer; ++p) {
            constexpr int kSteps = 4 / A::kPer;
            f32x4v sx = none;
            if constexpr (T::bf)
#pragma unroll
                for (int s = kSteps * p; s < kSteps * (p + 1); ++s) sx = T::mfma16(x[s], ones_of<T>(), sx);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const uint32_t z = aux[i][r].zero(p), less = less_of(z);
                f32x4v d = none;
#pragma unroll
                for (int s = kSteps * p; s < kSteps * (p + 1); ++s) {
                    u32x4v w = unpack(c[i][r][s]);
                    if (!T::bf)
#pragma unroll
                        for (int j = 0; j < 4; ++j) w[j] = take_off(w[j], less);
                    d = T::mfma16(x[s], w, d);
                }
                const float scale = aux[i][r].scale(p), off = 16.f + (float)z;
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[r][e] += scale * (T::bf ? d[e] - off * sx[e] : d[e]);
            }
        }
    };
    auto compute = [&](int i, int u) {
        u32x4v x[4];
        tokens(i, u, x);
        multiply(i, x);
    };
    if (a.K < 8) {  // (one unit of one wavefront)
        if (u0 < u1) {
            load(0, 0);
            u32x4v x[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) x[s] = load_x_end(xp, 32 * s + 8 * g, a.K);
            multiply(0, x);
        }
    } else if (u0 < u1) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            load(i, u0 + i);
            load_tokens(i, u0 + i);
            __builtin_amdgcn_sched_barrier(0);
        }
        // (no loads under a branch: the waits count them; none for a next turn that is not there: they
        // would cost a range of a few units as much of x again)
        int u = u0;
        for (; u + kAhead < u1; u += kAhead) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                compute(i, u + i);
                load(i, u + i + kAhead);
                load_tokens(i, u + i + kAhead);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (u + i < u1) compute(i, u + i);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) sh[wave][4 * g + e][16 * r + (lane & 15)] = acc[r][e];
    __syncthreads();
    for (int i = threadIdx.x; i < a.N * RT * 16; i += kQuantThreads) {
        const int n = i / (RT * 16), m = i % (RT * 16);
        const int64_t row = (int64_t)rt0 * 16 + m;
        if (row >= a.M) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kQuantWaves; ++w) v += sh[w][n][m];
        if (a.splits == 1)
            a.y[n * a.ldy + row] = (uint16_t)T::pack(v * kUnit<T>, 0.f);
        else
            a.part[((int64_t)blockIdx.y * a.N + n) * a.M + row] = v;
    }
}

// 17 to 64 tokens (NT tiles of 16).  One workgroup: four wavefronts by rows, RT row tiles each, times
// two by units; the four share their units' x in LDS (double-buffered, one barrier per unit), so that
// x comes from the L2 once per 4 RT KB of codes.  Rows of x are 256 bytes in LDS, 16-byte chunks
// XOR-swizzled by the token.  12288x49152 in groups of 128: 80 us for 32 tokens, 107 us for 64 (722
// TFLOP/s; 100 us without its loads).  Unpacking a word takes the vector unit as long as its four products
// take the matrix cores, and two wavefronts per SIMD overlap the two in part.  (Two workgroups of four
// wavefronts each in place of the two halves of one, which leaves them free to drift apart, were no
// faster there, 110 us, and cost the smaller matrices a longer join: 28672x7168 x 64 52.7 us against 42.2.)
template <typename T, int KIND, int NT, int RT>
__global__ __launch_bounds__(kQuantThreads, 2) void quant_many_kernel(QuantArgs a) {
    using A = Aux<T, KIND>;
    constexpr int kRowWaves = 4, kTokens = 16 * NT, kTile = kTokens * 256, kPer = kTokens * 16 / 256;
    constexpr int kJoin = kRowWaves * 64 * RT * NT * 4 * 4;  // bytes of one half's sums
    constexpr int kLds = 4 * kTile > kJoin ? 4 * kTile : kJoin;
    const Unpack<T> unpack;
    __shared__ __attribute__((aligned(16))) unsigned char sh[kLds];
    const int tid = threadIdx.x & 255, lane = threadIdx.x & 63, g = lane >> 4;
    const int half = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);      // which units
    const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) & 3);  // which rows
    const int rt0 = (blockIdx.x * kRowWaves + wave) * RT;
    const int parts = 2 * a.splits, part = blockIdx.y * 2 + half;
    const int u0 = (int)((int64_t)a.units * part / parts), u1 = (int)((int64_t)a.units * (part + 1) / parts);
    const int rounds = (a.units + parts - 1) / parts;  // the same for all: barriers
    const int have = max(0, min(RT, a.tiles - rt0));
    const int first = min(rt0, a.tiles - 1);
    const auto cb = tile_buffer(a.codes, first, have, (int64_t)a.units * 1024);
    const auto ab = tile_buffer(a.aux, first, have, (int64_t)a.units * kQuantRows * A::kBytes);
    const int ch = tid & 15;
    const uint16_t* xp[kPer];
    int at[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int n = i * 16 + (tid >> 4);
        xp[i] = a.x + min(n, a.N - 1) * a.ldx;
        at[i] = n * 256 + ((ch ^ (n & 15)) << 4);
    }
    u32x4v c[2][RT], xs[kPer];
    A aux[2][RT];
    auto load = [&](int i, int u) {
        const bool on = u < u1;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const bool here = on && r < have;  // (the scalar offset is not part of the bounds check)
            const int unit = here ? r * a.units + u : 0;
            c[i][r] = __builtin_amdgcn_raw_buffer_load_b128(cb, here ? lane * 16 : kNoRow, unit * 1024, 2);
            aux[i][r].load(ab, here ? (lane & 15) * A::kBytes : kNoRow, unit * (kQuantRows * A::kBytes));
        }
    };
    // (K is at least 8 here: a row's last 8 values stand in for chunks that reach past its end)
    auto clamp = [&](int u) { return min(max(u0, min(u, u1 - 1)), a.units - 1); };
    auto load_tokens = [&](int u) {
        const int k = min(clamp(u) * kQuantUnit + 8 * ch, a.K - 8);
#pragma unroll
        for (int i = 0; i < kPer; ++i) xs[i] = load_x(xp[i] + k);
    };
    auto store_tokens = [&](int i, int u) {
        u = clamp(u);
        if ((u + 1) * kQuantUnit > a.K)
#pragma unroll
            for (int j = 0; j < kPer; ++j) xs[j] = shift_end(xs[j], u * kQuantUnit + 8 * ch - (a.K - 8));
#pragma unroll
        for (int j = 0; j < kPer; ++j) *(u32x4v*)(sh + (2 * i + half) * kTile + at[j]) = xs[j];
    };
    f32x4v acc[RT][NT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[r][n] = f32x4v{0.f, 0.f, 0.f, 0.f};

    load_tokens(u0);
    load(0, u0);
    __builtin_amdgcn_sched_barrier(0);
    store_tokens(0, u0);
    load_tokens(u0 + 1);
    load(1, u0 + 1);
    lds_barrier();
    auto unit = [&](int i, int k) {
        const unsigned char* xb = sh + (2 * i + half) * kTile;
        const f32x4v none = {0.f, 0.f, 0.f, 0.f};
        constexpr int kSteps = 4 / A::kPer;  // steps of one group
        // x of one step of 32 columns, read a step ahead: the reads of a workgroup take about half as long
        // as its products, so they have to go on beside them
        u32x4v x[2][NT];
        auto read = [&](int s) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
                x[s & 1][n] = *(const u32x4v*)(xb + (16 * n + (lane & 15)) * 256 + (((4 * s + g) ^ (lane & 15)) << 4));
        };
        f32x4v d[RT][NT], sx[NT];
        if (u0 + k < u1) {
        read(0);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int p = s / kSteps;
            if (s < 3) read(s + 1);
            __builtin_amdgcn_sched_barrier(kFreeOrder);
            const bool first = s % kSteps == 0;
            if constexpr (T::bf)
#pragma unroll
                for (int n = 0; n < NT; ++n) sx[n] = T::mfma16(x[s & 1][n], ones_of<T>(), first ? none : sx[n]);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                u32x4v w = unpack(c[i][r][s]);
                if (!T::bf) {
                    const uint32_t less = less_of(aux[i][r].zero(p));
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = take_off(w[j], less);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) d[r][n] = T::mfma16(x[s & 1][n], w, first ? none : d[r][n]);
            }
            if (s % kSteps == kSteps - 1)
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const float scale = aux[i][r].scale(p), off = 16.f + (float)aux[i][r].zero(p);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[r][n][e] += scale * (T::bf ? d[r][n][e] - off * sx[n][e] : d[r][n][e]);
                }
        }
        }
        // the next unit's x into the other buffer (its last reads were before the last barrier)
        store_tokens(i ^ 1, u0 + k + 1);
        load_tokens(u0 + k + 2);
        load(i, u0 + k + 2);
        lds_barrier();
    };
    // An even number of units (nothing is computed past the end), so that every wait can count on the
    // other buffer's loads behind its own.
    for (int k = 0; k < rounds; k += 2) {
        unit(0, k);
        unit(1, k + 1);
    }
    // join the two halves; wavefront `wave` of half 0 then holds the sums of its rows
    float* js = (float*)sh + (wave * 64 + lane) * (RT * NT * 4);
    if (half == 1)
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n) *(f32x4v*)(js + (r * NT + n) * 4) = acc[r][n];
    __syncthreads();
    if (half == 1) return;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int64_t row = (int64_t)(rt0 + r) * 16 + (lane & 15);
        if (row >= a.M) continue;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const f32x4v v = acc[r][n] + *(const f32x4v*)(js + (r * NT + n) * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 16 * n + 4 * g + e;
                if (t >= a.N) continue;
                if (a.splits == 1)
                    a.y[t * a.ldy + row] = (uint16_t)T::pack(v[e] * kUnit<T>, 0.f);
                else
                    a.part[((int64_t)blockIdx.y * a.N + t) * a.M + row] = v[e];
            }
        }
    }
}

// Second pass of a split product: the partial sums in ascending order.
template <typename T>
__global__ __launch_bounds__(256) void quant_join_kernel(QuantArgs a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, total = (int64_t)a.N * a.M;
    if (i >= total) return;
    float v = 0.f;
    for (int s = 0; s < a.splits; ++s) v += a.part[s * total + i];
    a.y[i / a.M * a.ldy + i % a.M] = (uint16_t)T::pack(v * kUnit<T>, 0.f);
}

template <typename T, int KIND, int NT>
void run_many(const QuantArgs& a, int rt, hipStream_t s) {
    const dim3 grid((unsigned)((a.tiles + 4 * rt - 1) / (4 * rt)), (unsigned)a.splits);
    if (rt == 1) quant_many_kernel<T, KIND, NT, 1><<<grid, kQuantThreads, 0, s>>>(a);
    else if (rt == 2) quant_many_kernel<T, KIND, NT, 2><<<grid, kQuantThreads, 0, s>>>(a);
    else if (rt == 3) quant_many_kernel<T, KIND, NT, 3><<<grid, kQuantThreads, 0, s>>>(a);
    else if constexpr (NT < 4) quant_many_kernel<T, KIND, NT, 4><<<grid, kQuantThreads, 0, s>>>(a);
}
template <typename T, int KIND, typename X>
void run_few(const QuantArgs& a, int rt, hipStream_t s) {
    const dim3 grid((unsigned)((a.tiles + rt - 1) / rt), (unsigned)a.splits);
    if (rt == 1) quant_few_kernel<T, KIND, 1, X><<<grid, kQuantThreads, 0, s>>>(a);
    else if (rt == 2) quant_few_kernel<T, KIND, 2, X><<<grid, kQuantThreads, 0, s>>>(a);
    else if (rt == 3) quant_few_kernel<T, KIND, 3, X><<<grid, kQuantThreads, 0, s>>>(a);
    else if (rt == 4 || KIND == 4) quant_few_kernel<T, KIND, 4, X><<<grid, kQuantThreads, 0, s>>>(a);
    else if constexpr (KIND < 4) {
        if (rt == 6) quant_few_kernel<T, KIND, 6, X><<<grid, kQuantThreads, 0, s>>>(a);
        else quant_few_kernel<T, KIND, 7, X><<<grid, kQuantThreads, 0, s>>>(a);
    }
}
template <typename T, int KIND>
void run_kind(QuantArgs a, const QuantPlan& p, hipStream_t s) {
    // Lanes whose rows begin at odd multiples of 2 bytes, lanes without a token repeating a row that does not.
    // 5003x4099 (plain loads against OddX): 11.1 against 12.4 us with 2 such lanes, 13.8 against 12.6
    // with 3; 12288x4097: 13.6 against 12.7 with 2, 16.4 against 13.0 with 3, 31.7 against 17.6 with 8.
    const bool first = (uintptr_t)a.x % 4, change = a.N > 1 && a.ldx % 2;
    a.spare = first && change;
    const int lanes = change ? (a.N + first) / 2 : 16 * first;
    const bool odd = lanes > 2;
    if (!p.shared && odd) run_few<T, KIND, OddX>(a, p.rt, s);
    else if (!p.shared) run_few<T, KIND, EvenX>(a, p.rt, s);
    else if (a.N <= 32) run_many<T, KIND, 2>(a, p.rt, s);
    else run_many<T, KIND, 4>(a, p.rt, s);
}
template <typename T>
hipError_t run_product(const QuantArgs& a, int kind, const QuantPlan& p, hipStream_t s) {
    if (kind == 0) run_kind<T, 0>(a, p, s);
    else if (kind == 1) run_kind<T, 1>(a, p, s);
    else if (kind == 2) run_kind<T, 2>(a, p, s);
    else run_kind<T, 4>(a, p, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    quant_join_kernel<T><<<(unsigned)(((int64_t)a.N * a.M + 255) / 256), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace
}  // namespace lscd
