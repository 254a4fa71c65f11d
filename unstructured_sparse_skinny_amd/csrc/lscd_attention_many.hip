// Attention over a paged cache for many query rows (a chunk of a prompt): 256 rows (tokens x heads
// that share a key head) per item, bound by the matrix cores and the exponentials between the two
// products.
//
// A workgroup is eight wavefronts of 32 rows each; they share tiles of keys and values in LDS (64
// positions for heads of 65 to 128 channels, 128 for less, 32 for more: what the registers hold),
// double-buffered with one barrier per tile: the next tile's loads are issued before the current
// one is computed and written to the other buffer after it (codes of an 8-bit cache become 16-bit
// values on the way; scales are powers of two, so that this rounds nothing inside the type's range).  Keys are read back row by
// row (128-bit reads), values as V^T by the transposing LDS read (ds_read_b64_tr_b16): 16 lanes read
// a 4 x 16 block and get its columns, which is the A operand in the token order that P has.
// 16-byte chunks are XOR-swizzled by the row so that the lanes of one read spread over the banks.
//
// Measured: 2048 new tokens of 32 heads over 16384 positions (515 GFLOP) 521 to 590 us from one card to
// the next, 870 to 990 TFLOP/s; a matrix product in bfloat16 reaches 1232.  The matrix cores are busy 43 %
// of the cycles and the vector unit 40 %, and two wavefronts per SIMD overlap little of the two.  Heads of
// 256 channels: 1024 tokens of 16 heads over 8192 positions in 473 us, 270 TFLOP/s, against 98 us and 660 for
// 128 channels: 54 to 62 registers do not fit and go through memory in the loop.

#include <type_traits>

#include "lscd_attention.h"

namespace lscd {
namespace {

constexpr int kManyWaves = kManyRows / 32;
constexpr int kManyThreads = 64 * kManyWaves;

typedef __attribute__((address_space(3))) s16x4v lds_s16x4;

// Instructions that may cross the scheduling barriers below: vector and scalar arithmetic.
constexpr int kSchedFree = 0x6;

// Tokens of a tile: as many as the registers hold, so that a tile's products cover the next one's loads.
constexpr int many_tokens(int dp) { return dp <= 64 ? 2 * kManyTokens : (dp <= 128 ? kManyTokens : kManyTokens / 2); }

template <typename T, bool E4M3, int DP>
struct Many {
    static constexpr int kSteps = DP / 16;    // MFMA steps over the channels of q . k
    static constexpr int kBlocks = DP / 32;   // 32-channel blocks of the output
    static constexpr int kRow = DP * 2;       // bytes of an LDS row
    static constexpr int kTokens = many_tokens(DP);
    static constexpr int kTile = kTokens * kRow;
    // 16-byte loads: lanes per row (a power of two that covers DP), rows per pass, passes
    static constexpr int kPer = DP <= 64 ? (E4M3 ? 4 : 8) : DP <= 128 ? (E4M3 ? 8 : 16) : (E4M3 ? 16 : 32);
    static constexpr int kPassRows = kManyThreads / kPer;
    static constexpr int kPasses = kTokens / kPassRows;
    static_assert(kTokens % kPassRows == 0, "every thread has a row in every pass");
    static_assert(64 / kPer <= 16, "a wavefront's rows of one pass lie in one page");

    __device__ static __forceinline__ int key_at(int row, int chunk) {
        constexpr int mask = DP == 96 ? 3 : (DP == 64 ? 7 : 15);
        return row * kRow + ((chunk ^ (row & mask)) << 4);
    }
    __device__ static __forceinline__ int val_swizzle(int row) {
        return DP == 96 ? 0 : (DP == 64 ? ((row >> 1) & 1) << 2 : (row & 3) << 2);
    }
    __device__ static __forceinline__ int val_at(int row, int chunk) { return row * kRow + ((chunk ^ val_swizzle(row)) << 4); }

    u32x4v k[kPasses], v[kPasses];
    float ks[kPasses], vs[kPasses];
    int entry[kPasses];  // table entries of the next tile to load

    __device__ __forceinline__ static int row_of(int pass, int tid) { return pass * kPassRows + tid / kPer; }

    __device__ __forceinline__ void look_up(const AttnArgs& a, int seq, int t0, int wave) {
#pragma unroll
        for (int i = 0; i < kPasses; ++i) entry[i] = entry_of(a, seq, t0 + i * kPassRows + wave * (64 / kPer));
    }
    // Loads the tile whose entries look_up() found; rows from `high` on are zero.
    __device__ __forceinline__ void load(const AttnArgs& a, const HeadBase& hb, int t0, int low, int high, int tid) {
        const int D = a.c.head_dim, width = E4M3 ? 1 : 2, d = (tid % kPer) * (E4M3 ? 16 : 8);
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int t = t0 + row_of(i, tid), row = t & (a.c.page_size - 1);
            const uint32_t p = page_of(a, entry[i]);
            const bool on = t < high && t >= low;
            const int at = on && d < D ? (row * D + d) * width : kNoRow;
            k[i] = __builtin_amdgcn_raw_buffer_load_b128(hb.keys(p), at, 0, 0);
            v[i] = __builtin_amdgcn_raw_buffer_load_b128(hb.values(p), at, 0, 0);
            if (E4M3) {
                ks[i] = as_float(__builtin_amdgcn_raw_buffer_load_b32(hb.key_scales(p), on ? row * 4 : kNoRow, 0, 0));
                vs[i] = as_float(__builtin_amdgcn_raw_buffer_load_b32(hb.value_scales(p), on ? row * 4 : kNoRow, 0, 0));
            }
        }
    }
    // Writes the loaded tile as 16-bit values.  `edge`: some row may not see some position; such a row's
    // weight is 0, but 0 * infinity is NaN, so infinities and NaN among the values become zeros (the kernel
    // adds them where they are seen, when the item is done).  Returns whether this lane had any.
    __device__ __forceinline__ bool store(unsigned char* kb, unsigned char* vb, int tid, bool edge) {
        const int c = tid % kPer;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int row = row_of(i, tid);
            if (DP == 96 && c >= DP / (E4M3 ? 16 : 8)) continue;
            const bool top = E4M3 && __any(max(__builtin_bit_cast(uint32_t, ks[i]), __builtin_bit_cast(uint32_t, vs[i])) >= T::kTopScale);
#pragma unroll
            for (int h = 0; h < (E4M3 ? 2 : 1); ++h) {
                u32x4v x = k[i], y = v[i];
                if (E4M3) {
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        x[2 * w] = T::template from_e4m3<false>(k[i][2 * h + w], ks[i]);
                        x[2 * w + 1] = T::template from_e4m3<true>(k[i][2 * h + w], ks[i]);
                        y[2 * w] = T::template from_e4m3<false>(v[i][2 * h + w], vs[i]);
                        y[2 * w + 1] = T::template from_e4m3<true>(v[i][2 * h + w], vs[i]);
                    }
                    if (top) {
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            x[w] = saturate<T>(x[w]);
                            y[w] = saturate<T>(y[w]);
                        }
                    }
                }
                if (edge) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t f = T::finite(y[w]);
                        odd |= f != y[w];
                        y[w] = f;
                    }
                }
                const int chunk = E4M3 ? 2 * c + h : c;
                *(u32x4v*)(kb + key_at(row, chunk)) = x;
                *(u32x4v*)(vb + val_at(row, chunk)) = y;
            }
        }
        return odd;
    }
};

template <typename T, bool E4M3, int DP>
__global__ __launch_bounds__(kManyThreads, 2) void attention_many_kernel(AttnArgs a) {
    using F = Many<T, E4M3, DP>;
    __shared__ __attribute__((aligned(16))) unsigned char sh[2][2][F::kTile];
    __shared__ float sh_m[kManyThreads];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int half = lane >> 5;
    const int G = gridDim.x;
    // consecutive ranges on one XCD (workgroups go to the 8 XCDs in turn): they share keys in its L2
    const int me = (G & 7) == 0 ? (blockIdx.x & 7) * (G >> 3) + (blockIdx.x >> 3) : blockIdx.x;
    if (tid == 0) a.record[me] = int4{0, 0, 0, 0};
    Work p;
    if (!find_work<kManyRows, F::kTokens, false>(a, lane, me, G, &p)) return;
    const Cut cut = p.cut;
    int u = p.u;
    const int end = p.end;
    Seq& q = p.q;
    const int D = a.c.head_dim;

    // LDS offsets of this lane: key chunks by step, value columns by block
    const int key_row = lane & 31;
    const int vtok = 4 * half + ((lane & 15) >> 2);
    const int vchunk = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1), vhalf = (lane & 1) * 8;

    while (u < end) {
        int low, high;
        tile_range<kManyRows>(a, q, p.tile, &low, &high);
        const int units = max(1, (high + F::kTokens - 1) / F::kTokens - low / F::kTokens);
        const int item = u - p.unit;  // the slot of the item's first unit
        if (p.unit < 0) {
            u = item;
            p.unit = 0;
            if (u >= end) break;
        }
        const int last = min(units, p.unit + (end - u));
        const int t_base = low / F::kTokens * F::kTokens;

        const int row0 = p.tile * kManyRows + 32 * wave, row = row0 + (lane & 31);
        const bool live = row < q.rows;
        const int token = row / a.share;
        const int qh = p.head * a.share + row % a.share;
        const uint16_t* qp = (const uint16_t*)a.q + (int64_t)(q.first + (live ? token : 0)) * a.q_stride + (int64_t)qh * D;
        u32x4v qr[F::kSteps];
#pragma unroll
        for (int s = 0; s < F::kSteps; ++s) {
            const int d = 16 * s + 8 * half;
            qr[s] = u32x4v{0u, 0u, 0u, 0u};
            if (live && d < D) qr[s] = *(const u32x4v*)(qp + d);
            if (a.scale_log2 < 0.f) qr[s] ^= 0x80008000u;  // so that the scale below is positive
        }
        const float scale = fmaxf(fabsf(a.scale_log2), 1e-37f);  // (hidden scores of -infinity stay that with a scale of 0)
        const int pos = q.len - q.n + token;
        const int see_high = live ? (a.causal ? min(pos + 1, q.len) : q.len) : 0;
        const int see_low = a.window ? pos - a.window + 1 : 0;
        // this wavefront's rows: what some row sees, and what every row sees
        const int tok0 = row0 / a.share, tok1 = (min(q.rows, row0 + 32) - 1) / a.share;
        const int some_high = row0 < q.rows ? (a.causal ? min(q.len - q.n + tok1 + 1, q.len) : q.len) : 0;
        const int some_low = a.window ? q.len - q.n + tok0 - a.window + 1 : 0;
        const int all_high = a.causal ? min(q.len - q.n + tok0 + 1, q.len) : q.len;
        const int all_low = a.window ? q.len - q.n + tok1 - a.window + 1 : 0;

        // the same for all rows of the item
        const int end0 = p.tile * kManyRows / a.share, end1 = (min(q.rows, (p.tile + 1) * kManyRows) - 1) / a.share;
        const int tile_all_high = a.causal ? min(q.len - q.n + end0 + 1, q.len) : q.len;
        const int tile_all_low = a.window ? q.len - q.n + end1 - a.window + 1 : 0;

        float m = kNoScore, l = 0.f;
        f32x16v o[F::kBlocks];
#pragma unroll
        for (int b = 0; b < F::kBlocks; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[b][i] = 0.f;

        F f;
        const HeadBase hb(a, p.head, E4M3 ? 1 : 2);
        int t0 = t_base + p.unit * F::kTokens;
        f.look_up(a, p.seq, t0, wave);
        f.load(a, hb, t0, low, high, tid);
        f.look_up(a, p.seq, t0 + F::kTokens, wave);
        // One fma per weight takes the maximum, which is rounded, from a product that is not: no matter until
        // the rounding comes near 1, for scores of 2^23.  An item in which this wavefront has had scores of
        // kLarge rounds the product too: scores become exponents in place, and the maximum waits in LDS (one
        // register more through the products costs the 256-channel kernels a tenth of their time).
        bool large = false;
        float slope = scale;
        int any_odd = 0;     // an edge tile had infinities or NaN among its values
        auto is_edge = [&](int t) { return t < tile_all_low || t + F::kTokens > tile_all_high; };
        auto put = [&](int buf, int t) {
            const bool edge = is_edge(t);
            const bool odd = f.store(sh[buf][0], sh[buf][1], tid, edge);
            if (edge) any_odd |= __syncthreads_or(odd);
        };
        __syncthreads();  // the previous item's reads of the buffers are done
        put(0, t0);
        __syncthreads();
        for (int k = p.unit; k < last; ++k, t0 += F::kTokens) {
            const int buf = (k - p.unit) & 1;
            if (k + 1 < last) {
                f.load(a, hb, t0 + F::kTokens, low, high, tid);
                f.look_up(a, p.seq, t0 + 2 * F::kTokens, wave);
            }
            if (t0 < some_high && t0 + F::kTokens > some_low) {
                const unsigned char* kb = sh[buf][0];
                unsigned char* vb = sh[buf][1];
                constexpr int kHalves = F::kTokens / 32;
                f32x16v s[kHalves];
// reads run kAhead steps before the products that use them; the barriers keep that order
                constexpr int kAhead = 4, kKeySteps = kHalves * F::kSteps;
                auto key = [&](int i) {
                    return *(const u32x4v*)(kb + F::key_at(key_row, 2 * (i % F::kSteps) + half) + i / F::kSteps * 32 * F::kRow);
                };
                u32x4v kr[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) kr[i] = key(i);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < kKeySteps; ++i) {
                    const int h = i / F::kSteps;
                    if (i % F::kSteps == 0)
#pragma unroll
                        for (int e = 0; e < 16; ++e) s[h][e] = 0.f;
                    s[h] = T::mfma32(kr[i % kAhead], qr[i % F::kSteps], s[h]);
                    if (i + kAhead < kKeySteps) kr[i % kAhead] = key(i + kAhead);
                    __builtin_amdgcn_sched_barrier(kSchedFree);
                }
                const bool masked = t0 < all_low || t0 + F::kTokens > all_high;
                if (masked) {
#pragma unroll
                    for (int h = 0; h < kHalves; ++h)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int t = t0 + 32 * h + 8 * (i / 4) + 4 * half + i % 4;
                            if (t >= see_high || t < see_low) s[h][i] = -__builtin_inff();
                        }
                }
                float most = s[0][0];
#pragma unroll
                for (int i = 1; i < 16 * kHalves - 1; i += 2) most = max3(most, s[i / 16][i % 16], s[(i + 1) / 16][(i + 1) % 16]);
                most = max3(most, s[kHalves - 1][15], s[kHalves - 1][15]);
                if (large) m = sh_m[tid];
                if (large || __any(most * scale > m + (kLazy + T::kWeightBits))) {
                    const float to = fmaxf(m, max_halves(most) * scale - T::kWeightBits);
                    const float by = exp2_fast(m - to);
                    m = to;
                    l *= by;
#pragma unroll
                    for (int b = 0; b < F::kBlocks; ++b)
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[b][i] *= by;
                    large = large || __any(fabsf(m) >= kLarge && m != kNoScore);
                    if (large) {
#pragma unroll
                        for (int h = 0; h < kHalves; ++h)
#pragma unroll
                            for (int i = 0; i < 16; ++i) s[h][i] = product(s[h][i], scale) - m;
                        sh_m[tid] = m;
                        m = 0.f;
                        slope = 1.f;
                    }
                }
                // weights of the 16 tokens of step ks, as the B operand
                auto weights = [&](int ks) {
                    u32x4v w;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = exp2_fast(__builtin_fmaf(s[ks / 2][8 * (ks % 2) + 2 * i], slope, -m));
                        const float y = exp2_fast(__builtin_fmaf(s[ks / 2][8 * (ks % 2) + 2 * i + 1], slope, -m));
                        w[i] = T::pack(x, y);
                        l = T::add_pair(w[i], l);
                    }
                    return w;
                };
                auto value = [&](int b, int ks) {  // A operand of channels 32 b .., tokens 16 ks ..
                    const int at = vtok * F::kRow + (((4 * b + vchunk) ^ F::val_swizzle(vtok)) << 4) + vhalf + 16 * ks * F::kRow;
                    const auto x = __builtin_bit_cast(u32x2v, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(vb + at)));
                    const auto y = __builtin_bit_cast(u32x2v, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(vb + at + 8 * F::kRow)));
                    return u32x4v{x[0], x[1], y[0], y[1]};
                };
                constexpr int kValSteps = F::kBlocks * F::kTokens / 16;
                u32x4v vr[kAhead], pb[2];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) vr[i] = value(i % F::kBlocks, i / F::kBlocks);
                __builtin_amdgcn_sched_barrier(kSchedFree);
                pb[0] = weights(0);
#pragma unroll
                for (int i = 0; i < kValSteps; ++i) {
                    const int ks = i / F::kBlocks, b = i % F::kBlocks;
                    if (b == 0 && ks + 1 < F::kTokens / 16) pb[(ks + 1) & 1] = weights(ks + 1);  // between the products
                    o[b] = T::mfma32(vr[i % kAhead], pb[ks & 1], o[b]);
                    if (i + kAhead < kValSteps) vr[i % kAhead] = value((i + kAhead) % F::kBlocks, (i + kAhead) / F::kBlocks);
                    __builtin_amdgcn_sched_barrier(kSchedFree);
                }
            }
            if (k + 1 < last) put(buf ^ 1, t0 + F::kTokens);
            __syncthreads();
        }
        if (large) m = sh_m[tid];
        l = sum_halves(l);
        // What follows runs once per item: addresses are worked out here, not kept in registers through
        // the loop above (the compiler would move them out of all loops).
        const int lane_e = opaque(lane), half_e = lane_e >> 5;
        if (any_odd) {
            // The infinities and NaN of edge tiles, which store() left out, for the rows that see them (a
            // weight that is not zero leaves them as they are).  Rare: straight from the cache.
#pragma unroll 1
            for (int t = t_base + p.unit * F::kTokens; t < t_base + last * F::kTokens; ++t) {
                if (!is_edge(t / F::kTokens * F::kTokens)) continue;
                const uint32_t pg = page_of(a, entry_of(a, p.seq, t));
                const int at = t & (a.c.page_size - 1);
                const bool seen = t < see_high && t >= see_low;
                float vscale = 1.f;
                if (E4M3)
                    vscale = as_float(__builtin_amdgcn_raw_buffer_load_b32(hb.value_scales(pg), seen ? at * 4 : kNoRow, 0, 0));
#pragma unroll
                for (int b = 0; b < F::kBlocks; ++b)
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const int d = 32 * b + 8 * (i / 4) + 4 * half_e;
                        const int off = seen && d < D ? (at * D + d) * (E4M3 ? 1 : 2) : kNoRow;
                        u32x2v x;
                        if (E4M3) {
                            const uint32_t c = __builtin_amdgcn_raw_buffer_load_b32(hb.values(pg), off, 0, 0);
                            x = u32x2v{saturate<T>(T::template from_e4m3<false>(c, vscale)), saturate<T>(T::template from_e4m3<true>(c, vscale))};
                        } else {
                            x = __builtin_amdgcn_raw_buffer_load_b64(hb.values(pg), off, 0, 0);
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t xw = x[j], w = seen ? xw ^ T::finite(xw) : 0u;
                            o[b][i + 2 * j] += T::low(w);
                            o[b][i + 2 * j + 1] += T::high(w);
                        }
                    }
            }
        }

        const bool whole = p.unit == 0 && last == units;
        constexpr int64_t kFloats = (int64_t)kManyRows * (DP + 2);
        if (!whole) {
            // A part: a pair (maximum, sum) per row, then each lane's values as it holds them.  The
            // workgroup that has the item's first unit says what there is to join.
            const int owner = cut.owner(item), behind = cut.owner(item + units - 1);
            float* mine = a.part + (int64_t)(2 * me + (p.unit == 0 ? 1 : 0)) * kFloats;
            if (tid == 0 && owner == me) a.record[me] = int4{behind - owner, p.seq, p.head, p.tile};
            if (row0 < q.rows) {
                if (half_e == 0) *(float2*)(mine + 2 * (32 * wave + lane_e)) = float2{m, l};
#pragma unroll
                for (int b = 0; b < F::kBlocks; ++b)
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        *(f32x4v*)(mine + 2 * kManyRows + (((wave * F::kBlocks + b) * 4 + i / 4) * 64 + lane_e) * 4) =
                            f32x4v{o[b][i], o[b][i + 1], o[b][i + 2], o[b][i + 3]};
            }
        } else if (live) {
            const float inv = l != 0.f ? 1.f / l : 0.f;
            uint16_t* op = (uint16_t*)a.o + (int64_t)(q.first + opaque(token)) * a.o_stride + (int64_t)opaque(qh) * D;
#pragma unroll
            for (int b = 0; b < F::kBlocks; ++b)
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const int d = 32 * b + 8 * (i / 4) + 4 * half_e;
                    u32x2v x = {T::pack(o[b][i] * inv, o[b][i + 1] * inv), T::pack(o[b][i + 2] * inv, o[b][i + 3] * inv)};
                    if (l == 0.f) x = u32x2v{0u, 0u};
                    if (d < D) *(u32x2v*)(op + d) = x;
                }
        }

        u += last - p.unit;
        if (u >= end) break;
        p.unit = -kStart;
        next_item<kManyRows, false>(a, &p.seq, &p.head, &p.tile, &q);
    }
}

// Joins the parts of the items that were cut (records of G workgroups).  The work, cut items times
// wavefronts' rows times blocks of 32 channels, is spread over the grid: one vector of four values per
// thread and part.  Parts are 256 rows: joined by an item's last workgroup inside the kernel above, they
// came one after the other (64 new tokens of 32 heads over 8192 positions: 268 us that way).
constexpr int kJoinGrid = 2048, kJoinMasks = 32;
template <typename T, int DP>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a, int G) {
    constexpr int kBlocks = DP / 32, kSlabs = kManyWaves * kBlocks;
    constexpr int64_t kFloats = (int64_t)kManyRows * (DP + 2);
    __shared__ uint64_t sh_mask[kJoinMasks];
    const int lane = threadIdx.x & 63, i = threadIdx.x >> 6;
    for (int g = i; g * 64 < G; g += 4) {
        const uint64_t mask = __ballot(g * 64 + lane < G && a.record[min(g * 64 + lane, G - 1)].x != 0);
        if (lane == 0) sh_mask[g] = mask;
    }
    __syncthreads();
    int items = 0;
    for (int g = 0; g * 64 < G; ++g) items += __popcll(sh_mask[g]);
    for (int work = blockIdx.x; work < items * kSlabs; work += gridDim.x) {
        const int slab = work % kSlabs, wave = slab / kBlocks, b = slab % kBlocks;
        int n = work / kSlabs, g = 0;  // the n-th record that is set
        for (; n >= __popcll(sh_mask[g]); ++g) n -= __popcll(sh_mask[g]);
        uint64_t mask = sh_mask[g];
        for (; n > 0; --n) mask &= mask - 1;
        const int owner = __builtin_amdgcn_readfirstlane(g * 64 + __builtin_ctzll(mask));
        const int4 rec = a.record[owner];
        const Seq q = read_seq(a, __builtin_amdgcn_readfirstlane(rec.y));
        const int in_tile = 32 * wave + (lane & 31), row = rec.w * kManyRows + in_tile, behind = owner + rec.x;
        if (row >= q.rows) continue;
        float m = kNoScore, l = 0.f;
        f32x4v o = {0.f, 0.f, 0.f, 0.f};
        constexpr int kBatch = 8;  // parts in flight
        for (int w0 = owner; w0 <= behind; w0 += kBatch) {
            float2 ml[kBatch];
            f32x4v x[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (j >= 2 && w0 + j > behind) continue;
                const int w = min(w0 + j, behind);
                const float* part = a.part + (int64_t)(2 * w + (w == owner ? 1 : 0)) * kFloats;
                ml[j] = *(const float2*)(part + 2 * in_tile);
                x[j] = *(const f32x4v*)(part + 2 * kManyRows + ((slab * 4 + i) * 64 + lane) * 4);
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (w0 + j > behind) continue;
                const float to = fmaxf(m, ml[j].x), b0 = exp2_fast(m - to), b1 = exp2_fast(ml[j].x - to);
                m = to;
                l = l * b0 + ml[j].y * b1;
#pragma unroll
                for (int r = 0; r < 4; ++r) o[r] = o[r] * b0 + x[j][r] * b1;
            }
        }
        const int d = 32 * b + 8 * i + 4 * (lane >> 5);
        if (d >= a.c.head_dim) continue;
        const float inv = l != 0.f ? 1.f / l : 0.f;
        u32x2v out = {T::pack(o[0] * inv, o[1] * inv), T::pack(o[2] * inv, o[3] * inv)};
        if (l == 0.f) out = u32x2v{0u, 0u};
        *(u32x2v*)((uint16_t*)a.o + (int64_t)(q.first + row / a.share) * a.o_stride +
                   (int64_t)(rec.z * a.share + row % a.share) * a.c.head_dim + d) = out;
    }
}

template <typename T, bool E4M3, int DP>
hipError_t many_run(const AttnArgs& a, int grid, hipStream_t s) {
    attention_many_kernel<T, E4M3, DP><<<grid, kManyThreads, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    attention_join_kernel<T, DP><<<kJoinGrid, 256, 0, s>>>(a, grid);
    return hipGetLastError();
}

template <typename T, bool E4M3>
hipError_t many_dim(const AttnArgs& a, int grid, hipStream_t s) {
    const int D = a.c.head_dim;
    if (D <= 64) return many_run<T, E4M3, 64>(a, grid, s);
    if (D <= 96) return many_run<T, E4M3, 96>(a, grid, s);
    if (D <= 128) return many_run<T, E4M3, 128>(a, grid, s);
    return many_run<T, E4M3, 256>(a, grid, s);
}

}  // namespace

int attention_many_grid(int cus) { return cus < 64 * kJoinMasks ? cus : 64 * kJoinMasks; }
int attention_many_tokens(int dim) { return many_tokens(dim <= 64 ? 64 : dim <= 128 ? 128 : 256); }
int64_t attention_many_floats(int dim) {
    return (int64_t)kManyRows * ((dim <= 64 ? 64 : dim <= 96 ? 96 : dim <= 128 ? 128 : 256) + 2);
}

hipError_t launch_attention_many(const AttnArgs& a, int type, int grid, hipStream_t s) {
    const bool e = a.c.type == LSCD_E4M3;
    if (type == LSCD_F16) return e ? many_dim<F16, true>(a, grid, s) : many_dim<F16, false>(a, grid, s);
    return e ? many_dim<BF16, true>(a, grid, s) : many_dim<BF16, false>(a, grid, s);
}

}  // namespace lscd
