// Product of a few token vectors with a matrix of 4-bit codes and group scales (see lscd_quant.h for
// the arithmetic): encoding into the device layout, decoding, and the product.

#include "lscd_quant.h"

namespace lscd {
namespace {

// ---------------------------------------------------------------- layout
// One workgroup per row tile and 4 units: 256 threads = 4 units x 64 lanes, 4 words each.
__global__ __launch_bounds__(256) void quant_encode_kernel(QuantEncodeArgs a) {
    const int blocks4 = (a.units + 3) / 4;
    const int rt = blockIdx.x / blocks4, u4 = blockIdx.x % blocks4;
    const int lane = threadIdx.x & 63, u = u4 * 4 + (threadIdx.x >> 6);
    const int64_t row = (int64_t)rt * kQuantRows + (lane & 15);
    auto zero_of = [&](int64_t r, int64_t g) { return r < a.M && g < a.groups && a.zeros ? a.zeros[r * a.groups + g] & 15u : 8u; };
    if (u < a.units) {
        u32x4v out;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            uint32_t w = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t k = (int64_t)u * kQuantUnit + 32 * s + 8 * (lane >> 4) + j;
                uint32_t c = zero_of(row, k / a.group);
                if (row < a.M && k < a.K) c = (a.q[row * a.row_bytes + k / 2] >> (4 * (k & 1))) & 15u;
#pragma unroll
                for (int b = 0; b < 4; ++b) w |= ((c >> b) & 1u) << quant_bit(j, b);
            }
            out[s] = w;
        }
        *(u32x4v*)(a.codes + (((int64_t)rt * a.units + u) * 64 + lane) * 4) = out;
    }
    if (threadIdx.x < kQuantRows) {
        const int64_t r = (int64_t)rt * kQuantRows + threadIdx.x;
        const int n = 4 * a.per_unit;
        const int64_t rec = ((int64_t)rt * blocks4 + u4) * kQuantRows + threadIdx.x;
        uint32_t z[2] = {0, 0};
        for (int i = 0; i < n; ++i) {
            const int64_t k = ((int64_t)u4 * 4 + i / a.per_unit) * kQuantUnit + (i % a.per_unit) * (kQuantUnit / a.per_unit);
            const int64_t g = k / a.group;
            a.scales_out[rec * n + i] = r < a.M && g < a.groups ? a.scales[r * a.groups + g] : (uint16_t)0;
            z[i / 8] |= zero_of(r, g) << (4 * (i % 8));
        }
        if (a.zeros_out) {
            const int words = a.per_unit == 4 ? 2 : 1;
            for (int i = 0; i < words; ++i) a.zeros_out[rec * words + i] = z[i];
        }
    }
}

// Scales and zero points of one lane's row for 4 units.
template <int PER>
struct Aux {
    static constexpr int kWords = 2 * PER;  // words of 4 * PER scales
    uint32_t s[kWords], z[PER == 4 ? 2 : 1];
    __device__ __forceinline__ void load(const QuantArgs& a, int64_t rec) {
        const uint32_t* p = (const uint32_t*)a.scales + rec * kWords;
#pragma unroll
        for (int i = 0; i < kWords; ++i) s[i] = p[i];
        constexpr int n = PER == 4 ? 2 : 1;
#pragma unroll
        for (int i = 0; i < n; ++i) z[i] = a.zeros ? a.zeros[rec * n + i] : 0x88888888u;
    }
    // group i (0 .. 4 PER - 1); i is a constant after unrolling
    template <typename T>
    __device__ __forceinline__ float scale(int i) const {
        return i & 1 ? T::high(s[i / 2]) : T::low(s[i / 2]);
    }
    __device__ __forceinline__ uint32_t zero(int i) const { return (z[i / 8] >> (4 * (i % 8))) & 15u; }
};

template <typename T, int PER>
__global__ __launch_bounds__(256) void quant_decode_kernel(QuantArgs a, uint16_t* w) {
    const int rt = blockIdx.x / ((a.units + 3) / 4), u4 = blockIdx.x % ((a.units + 3) / 4);
    const int lane = threadIdx.x & 63, u = u4 * 4 + (threadIdx.x >> 6);
    const int64_t row = (int64_t)rt * kQuantRows + (lane & 15);
    if (u >= a.units || row >= a.M) return;
    Aux<PER> x;
    x.load(a, ((int64_t)rt * ((a.units + 3) / 4) + u4) * kQuantRows + (lane & 15));
    const uint32_t* c = a.codes + (((int64_t)rt * a.units + u) * 64 + lane) * 4;
    for (int s = 0; s < 4; ++s) {
        const u32x4v v = unpack_codes<T>(c[s]);
        for (int j = 0; j < 8; ++j) {
            const int64_t k = (int64_t)u * kQuantUnit + 32 * s + 8 * (lane >> 4) + j;
            if (k >= a.K) continue;
            float f = 0.f;
#pragma unroll
            for (int i = 0; i < 4 * PER; ++i)  // constant indices only
                if (i == (u & 3) * PER + s * PER / 4) {
                    const uint32_t p = v[j / 2];
                    f = ((j & 1 ? T::high(p) : T::low(p)) - (16.f + (float)x.zero(i))) * x.template scale<T>(i);
                }
            w[row * a.K + k] = (uint16_t)T::pack(f, 0.f);
        }
    }
}

// ---------------------------------------------------------------- product
// One workgroup: RT row tiles, one of a.splits ranges of units, which its eight wavefronts split
// further; their sums are joined through LDS.  NT: tiles of 16 tokens.
template <typename T, int PER, int NT, int RT>
__global__ __launch_bounds__(64 * kQuantWaves) void quant_kernel(QuantArgs a) {
    __shared__ float sh[kQuantWaves][NT * 16][RT * 16 + 1];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4;
    const int blocks4 = (a.units + 3) / 4;
    const int rt0 = blockIdx.x * RT, parts = kQuantWaves * a.splits, part = blockIdx.y * kQuantWaves + wave;
    const int u0 = (int)((int64_t)a.units * part / parts), u1 = (int)((int64_t)a.units * (part + 1) / parts);
    f32x4v acc[RT][NT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[r][n] = f32x4v{0.f, 0.f, 0.f, 0.f};
    const f32x4v none = {0.f, 0.f, 0.f, 0.f};
    const u32x4v ones = T::bf ? u32x4v{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}
                              : u32x4v{0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
    for (int b = u0 / 4; b * 4 < u1; ++b) {
        Aux<PER> aux[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
            aux[r].load(a, ((int64_t)min(rt0 + r, a.tiles - 1) * blocks4 + b) * kQuantRows + (lane & 15));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int u = 4 * b + i;
            if (u < u0 || u >= u1) continue;
            u32x4v c[RT], x[NT][4];
#pragma unroll
            for (int r = 0; r < RT; ++r)
                c[r] = *(const u32x4v*)(a.codes + (((int64_t)min(rt0 + r, a.tiles - 1) * a.units + u) * 64 + lane) * 4);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int token = 16 * n + (lane & 15);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    x[n][s] = u32x4v{0u, 0u, 0u, 0u};
                    if (token < a.N) x[n][s] = load_x(a.x + token * a.ldx, u * kQuantUnit + 32 * s + 8 * g, a.K);
                }
            }
#pragma unroll
            for (int p = 0; p < PER; ++p) {
                f32x4v sx[NT];
                if (T::bf) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        sx[n] = none;
#pragma unroll
                        for (int s = 4 / PER * p; s < 4 / PER * (p + 1); ++s) sx[n] = T::mfma16(x[n][s], ones, sx[n]);
                    }
                }
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const uint32_t z = aux[r].zero(i * PER + p);
                    const float scale = aux[r].template scale<T>(i * PER + p);
                    // -(16 + z): 0xCC00 | z << 6 in float16
                    const uint32_t less = (0xCC00u | z << 6) * 0x00010001u;
                    f32x4v d[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) d[n] = none;
#pragma unroll
                    for (int s = 4 / PER * p; s < 4 / PER * (p + 1); ++s) {
                        u32x4v w = unpack_codes<T>(c[r][s]);
                        if (!T::bf)
#pragma unroll
                            for (int j = 0; j < 4; ++j) w[j] = take_off(w[j], less);
#pragma unroll
                        for (int n = 0; n < NT; ++n) d[n] = T::mfma16(x[n][s], w, d[n]);
                    }
                    const float off = 16.f + (float)z;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[r][n][e] += scale * (T::bf ? d[n][e] - off * sx[n][e] : d[n][e]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sh[wave][16 * n + 4 * g + e][16 * r + (lane & 15)] = acc[r][n][e];
    __syncthreads();
    for (int i = threadIdx.x; i < a.N * RT * 16; i += 64 * kQuantWaves) {
        const int n = i / (RT * 16), m = i % (RT * 16);
        const int64_t row = (int64_t)rt0 * 16 + m;
        if (row >= a.M) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kQuantWaves; ++w) v += sh[w][n][m];
        if (a.splits == 1)
            a.y[n * a.ldy + row] = (uint16_t)T::pack(v, 0.f);
        else
            a.part[((int64_t)blockIdx.y * a.N + n) * a.M + row] = v;
    }
}

// Second pass of a split product: the partial sums in ascending order.
template <typename T>
__global__ __launch_bounds__(256) void quant_join_kernel(QuantArgs a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, total = (int64_t)a.N * a.M;
    if (i >= total) return;
    float v = 0.f;
    for (int s = 0; s < a.splits; ++s) v += a.part[s * total + i];
    a.y[i / a.M * a.ldy + i % a.M] = (uint16_t)T::pack(v, 0.f);
}

template <typename T, int PER, int NT, int RT>
hipError_t run(const QuantArgs& a, hipStream_t s) {
    quant_kernel<T, PER, NT, RT><<<dim3((a.tiles + RT - 1) / RT, a.splits), 64 * kQuantWaves, 0, s>>>(a);
    if (a.splits > 1) {
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        quant_join_kernel<T><<<(unsigned)(((int64_t)a.N * a.M + 255) / 256), 256, 0, s>>>(a);
    }
    return hipGetLastError();
}
template <typename T, int PER>
hipError_t run_tokens(const QuantArgs& a, hipStream_t s) {
    if (a.N <= 16) return run<T, PER, 1, 2>(a, s);
    if (a.N <= 32) return run<T, PER, 2, 2>(a, s);
    return run<T, PER, 4, 2>(a, s);
}
template <typename T>
hipError_t run_groups(const QuantArgs& a, int per_unit, hipStream_t s) {
    if (per_unit == 1) return run_tokens<T, 1>(a, s);
    if (per_unit == 2) return run_tokens<T, 2>(a, s);
    return run_tokens<T, 4>(a, s);
}

}  // namespace

hipError_t launch_quant_encode(const QuantEncodeArgs& a, hipStream_t s) {
    quant_encode_kernel<<<(unsigned)(a.tiles * (int64_t)((a.units + 3) / 4)), 256, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_quant_decode(const QuantArgs& a, int type, int per_unit, uint16_t* w, hipStream_t s) {
    const unsigned grid = (unsigned)(a.tiles * (int64_t)((a.units + 3) / 4));
    if (type == LSCD_F16) {
        if (per_unit == 1) quant_decode_kernel<F16, 1><<<grid, 256, 0, s>>>(a, w);
        else if (per_unit == 2) quant_decode_kernel<F16, 2><<<grid, 256, 0, s>>>(a, w);
        else quant_decode_kernel<F16, 4><<<grid, 256, 0, s>>>(a, w);
    } else {
        if (per_unit == 1) quant_decode_kernel<BF16, 1><<<grid, 256, 0, s>>>(a, w);
        else if (per_unit == 2) quant_decode_kernel<BF16, 2><<<grid, 256, 0, s>>>(a, w);
        else quant_decode_kernel<BF16, 4><<<grid, 256, 0, s>>>(a, w);
    }
    return hipGetLastError();
}

hipError_t launch_quant(const QuantArgs& a, int type, int per_unit, hipStream_t s) {
    return type == LSCD_F16 ? run_groups<F16>(a, per_unit, s) : run_groups<BF16>(a, per_unit, s);
}

}  // namespace lscd
