// Matrices of 4-bit codes: encoding into the device layout, decoding, and how a product is split.

#include <algorithm>
#include <cmath>

#include "lscd_quant.h"

namespace lscd {
namespace {

// One workgroup per row tile and 4 units: 256 threads = 4 units x 64 lanes, 4 words each.
__global__ __launch_bounds__(256) void quant_encode_kernel(QuantEncodeArgs a) {
    const int blocks4 = (a.units + 3) / 4;
    const int rt = blockIdx.x / blocks4, u = blockIdx.x % blocks4 * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)rt * kQuantRows + (lane & 15);
    auto zero_of = [&](int64_t r, int64_t g) { return r < a.M && g < a.groups && a.zeros ? a.zeros[r * a.groups + g] & 15u : 8u; };
    if (u >= a.units) return;
    u32x4v out;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        uint32_t w = 0;
        const int64_t k0 = (int64_t)u * kQuantUnit + 32 * s + 8 * (lane >> 4);
        const uint32_t z = zero_of(row, k0 / a.group);  // (groups are multiples of 32: one for the word)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t k = k0 + j;
            uint32_t c = z;
            if (row < a.M && k < a.K) c = (a.q[row * a.row_bytes + k / 2] >> (4 * (k & 1))) & 15u;
#pragma unroll
            for (int b = 0; b < 4; ++b) w |= ((c >> b) & 1u) << quant_bit(j, b);
        }
        out[s] = w;
    }
    const int64_t unit = (int64_t)rt * a.units + u;
    *(u32x4v*)(a.codes + (unit * 64 + lane) * 4) = out;
    if (lane < kQuantRows) {
        for (int p = 0; p < a.per_unit; ++p) {
            const int64_t k = (int64_t)u * kQuantUnit + p * (kQuantUnit / a.per_unit), g = k / a.group;
            const uint32_t s = row < a.M && g < a.groups ? a.scales[row * a.groups + g] : 0u;
            const int64_t at = (unit * kQuantRows + lane) * a.per_unit + p;
            if (a.short_aux)
                ((uint16_t*)a.aux)[at] = (uint16_t)s;
            else
                ((uint32_t*)a.aux)[at] = s | zero_of(row, g) << 16;
        }
    }
}

template <typename T, int KIND>
__global__ __launch_bounds__(256) void quant_decode_kernel(QuantArgs a, uint16_t* w) {
    using A = Aux<T, KIND>;
    const int blocks4 = (a.units + 3) / 4;
    const int rt = blockIdx.x / blocks4, u = blockIdx.x % blocks4 * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)rt * kQuantRows + (lane & 15);
    if (u >= a.units || row >= a.M) return;
    const int64_t unit = (int64_t)rt * a.units + u;
    const uint8_t* rec = (const uint8_t*)a.aux + (unit * kQuantRows + (lane & 15)) * A::kBytes;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        uint32_t x;
        if (KIND == 0)
            x = *(const uint16_t*)rec | 8u << 16;
        else
            x = ((const uint32_t*)rec)[s * A::kPer / 4];
        const u32x4v v = Unpack<T>()(a.codes[(unit * 64 + lane) * 4 + s]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t k = (int64_t)u * kQuantUnit + 32 * s + 8 * (lane >> 4) + j;
            const uint32_t p = v[j / 2];
            const float c = (j & 1 ? T::high(p) : T::low(p)) * kUnit<T> - (16.f + (float)(x >> 16));
            if (k < a.K) w[row * a.K + k] = (uint16_t)T::pack(c * T::low(x & 0xFFFFu), 0.f);
        }
    }
}

template <typename T>
hipError_t decode_kind(const QuantArgs& a, int kind, uint16_t* w, hipStream_t s) {
    const unsigned grid = (unsigned)(a.tiles * (int64_t)((a.units + 3) / 4));
    if (kind == 0) quant_decode_kernel<T, 0><<<grid, 256, 0, s>>>(a, w);
    else if (kind == 1) quant_decode_kernel<T, 1><<<grid, 256, 0, s>>>(a, w);
    else if (kind == 2) quant_decode_kernel<T, 2><<<grid, 256, 0, s>>>(a, w);
    else quant_decode_kernel<T, 4><<<grid, 256, 0, s>>>(a, w);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_encode(const QuantEncodeArgs& a, hipStream_t s) {
    quant_encode_kernel<<<(unsigned)(a.tiles * (int64_t)((a.units + 3) / 4)), 256, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_quant_decode(const QuantArgs& a, int type, int kind, uint16_t* w, hipStream_t s) {
    return type == LSCD_F16 ? decode_kind<F16>(a, kind, w, s) : decode_kind<BF16>(a, kind, w, s);
}

// Row tiles per wavefront and splits along K: the least time by a model of this GPU, in microseconds.
// Up to 16 tokens: a CU moves about 20 KB of codes a microsecond; x costs up to half of what its 256 bytes
// a token and unit of a wavefront would from HBM, and is loaded for all units of a wavefront's turn.  A
// workgroup takes 1 us to start and join where others run, 3 us and a memory latency for each turn of its
// loads alone.  More than 16 tokens: a workgroup's round (two units of 4 RT row tiles) measured 0.35 + 0.58
// RT (64 tokens) and 0.3 + 0.45 RT (32).  A split adds a launch and its partial sums.  It picks 7 row tiles
// for 28672 x 7168 (1792 tiles, 7 on every CU: 23.0 us at 16 tokens, 38.2 with one), 1 for 4096 x 4096 (6.6
// us).  More row tiles than 4 with records of four words do not fit the registers (27648 x 9216 x 16 in groups
// of 32: 722 us with 7, 41.7 with 4); nor do 4 row tiles of 64 tokens.
// (Of the numbers between, 5 is not built: 20480 rows, 5 tiles on every CU, take 6, by the model a seventh slower.)
QuantPlan plan_quant(int tiles, int units, int N, int kind, int cus) {
    QuantPlan best = {N > 16, 1, 1};
    double cost = 0;
    static const int few[] = {1, 2, 3, 4, 6, 7}, many[] = {1, 2, 3, 4};
    const int* rts = best.shared ? many : few;
    const int n = N > 32 ? 3 : (best.shared || kind == 4 ? 4 : 6);
    const int wr = best.shared ? 4 : 1, wk = kQuantWaves / wr;
    for (int i = 0; i < n; ++i) {
        const int rt = rts[i];
        const int64_t groups = (tiles + (int64_t)rt * wr - 1) / (rt * wr);
        for (int s = 1; s <= 16 && (s == 1 || s * wk <= units); ++s) {
            const double rounds = (double)((groups * s + cus - 1) / cus), per_wave = (double)((units + s * wk - 1) / (s * wk));
            double t;
            if (best.shared) {
                t = 3.0 + rounds * per_wave * (N > 32 ? 0.35 + 0.58 * rt : 0.3 + 0.45 * rt);
            } else {
                const int ahead = quant_ahead(rt, kind);
                const double turns = std::ceil(per_wave / ahead);  // (x is loaded for all of a turn's units)
                t = std::max(rounds * (1.0 + wk * (per_wave * rt + turns * ahead * N / 8.0) * 0.05), 3.0 + per_wave / ahead);
            }
            if (s > 1) t += 4.0 + (double)s * N * tiles * 16 * 8 / 5e6;
            if ((i == 0 && s == 1) || t < cost) {
                cost = t;
                best.rt = rt;
                best.splits = s;
            }
        }
    }
    return best;
}

}  // namespace lscd
