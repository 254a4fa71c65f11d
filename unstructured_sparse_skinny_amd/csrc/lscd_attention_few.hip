// Attention over a paged cache for few query rows (decoding): up to 16 rows (tokens x heads that
// share a key head) per item, memory-bound: every key and value is read once, straight into
// registers.
//
// A workgroup is four wavefronts; each takes 32 of a unit's 128 positions with a running maximum
// and sums of its own, joined through LDS where an item ends.  Per 32 positions a wavefront needs
// no LDS at all: the key rows are the A operand as they lie in memory (16 bytes of 64 channels per
// lane), and the values become the A operand V^T by an in-register transposition: lane l loads the
// same 8 channels of 8 tokens, and one v_perm_b32 per pair of values puts two tokens into one word
// (half an instruction per value; an LDS transposition would cost a write and a read).  The loads
// of the next unit's keys are issued when the scores are done with this one's, the next values
// when the second product is, so that 8 to 16 KB per wavefront are always in flight; the next item's
// first loads are issued before the present one's end.
//
// Measured: 64 sequences of one token over up to 2048 positions of 96 heads (e4m3, 1.72 GB) 313 us, 5.5
// TB/s, which is what a plain read reaches here; one token over 1000 positions of 8 heads 9.5 us, a chain
// of dependent latencies (tables, keys, values, partial results, their join) rather than its 4 MB.

#include <type_traits>

#include "lscd_attention.h"

namespace lscd {
namespace {

constexpr int kFewWaves = 4;

// DP: channels padded to 64, 128 or 256.
template <typename T, bool E4M3, int DP>
struct Few {
    static constexpr int kSteps = DP / 32;  // MFMA steps over the channels of q . k
    static constexpr int VW = DP / 16;      // channels per lane of a value row
    static constexpr int kKeyRegs = E4M3 ? DP / 16 : DP / 8;        // words of one 16-token key tile per lane
    static constexpr int kValWords = E4M3 ? VW / 4 : VW / 2;        // words of one value row per lane
    uint32_t kr[2][kKeyRegs];
    uint32_t vr[8][kValWords];
    uint32_t ks[2], vs[8];  // scales as loaded (e4m3)

    // 32 positions from t0 on, in the pages of the table entries e; positions from `high` on are zero
    // (lanes without a position read outside the descriptor, which costs no traffic).
    __device__ __forceinline__ void load_keys(const AttnArgs& a, const HeadBase& hb, const int (&e)[2], int t0, int high,
                                              int lane) {
        const int D = a.c.head_dim;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int t = t0 + 16 * h, row = (t & (a.c.page_size - 1)) + (lane & 15);
            const uint32_t p = page_of(a, e[h]);
            const bool on = t + (lane & 15) < high;
            const auto rs = hb.keys(p);
            if (E4M3) {
#pragma unroll
                for (int u = 0; u < DP / 64; ++u) {
                    const int d = 64 * u + 16 * (lane >> 4);
                    const u32x4v x = __builtin_amdgcn_raw_buffer_load_b128(rs, on && d < D ? row * D + d : kNoRow, 0, 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i) kr[h][4 * u + i] = x[i];
                }
                ks[h] = __builtin_amdgcn_raw_buffer_load_b32(hb.key_scales(p), on ? row * 4 : kNoRow, 0, 0);
            } else {
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    const int d = 32 * s + 8 * (lane >> 4);
                    const u32x4v x = __builtin_amdgcn_raw_buffer_load_b128(rs, on && d < D ? (row * D + d) * 2 : kNoRow, 0, 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i) kr[h][4 * s + i] = x[i];
                }
            }
        }
    }

    // Value rows of lane group g: positions 4g .. 4g+3 of each of the two 16-position halves.
    // Positions outside [low, high) are zero (their scales are left out by value_scale).
    __device__ __forceinline__ void load_values(const AttnArgs& a, const HeadBase& hb, const int (&e)[2], int t0, int low,
                                                int high, int lane) {
        constexpr int W = E4M3 ? 1 : 2;
        const int D = a.c.head_dim, g = lane >> 4, d = VW * (lane & 15);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int t = t0 + 16 * h, r0 = (t & (a.c.page_size - 1)) + 4 * g;
            const uint32_t p = page_of(a, e[h]);
            const auto rs = hb.values(p);
            if (E4M3) {
                const u32x4v sc = __builtin_amdgcn_raw_buffer_load_b128(hb.value_scales(p), r0 * 4, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j) vs[4 * h + j] = sc[j];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int pos = t + 4 * g + j;
                const bool on = pos < high && pos >= low;
                constexpr int kPer = kValWords < 4 ? kValWords : 4;  // words of one load
#pragma unroll
                for (int w = 0; w < kValWords; w += kPer) {
                    const int at = d + w * 4 / W;
                    const int off = on && at < D ? ((r0 + j) * D + at) * W : kNoRow;
                    if constexpr (kPer == 1) {
                        vr[4 * h + j][w] = __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0);
                    } else if constexpr (kPer == 2) {
                        const u32x2v x = __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0);
                        vr[4 * h + j][w] = x[0];
                        vr[4 * h + j][w + 1] = x[1];
                    } else {
                        const u32x4v x = __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0);
#pragma unroll
                        for (int i = 0; i < 4; ++i) vr[4 * h + j][w + i] = x[i];
                    }
                }
            }
        }
    }
    // A position that was not loaded has zeros for codes, but any scale: 1 instead.
    __device__ __forceinline__ void mask_scales(int t0, int low, int high, int lane) {
        if (!E4M3) return;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int pos = t0 + 16 * (j / 4) + 4 * (lane >> 4) + j % 4;
            if (pos >= high || pos < low) vs[j] = 0x3F800000u;
        }
    }

    // Whether some key's or value's code times its scale may pass the type's largest value.  (Scales are
    // positive: they compare as whole numbers.)
    __device__ __forceinline__ bool top_keys() const { return E4M3 && __any(max(ks[0], ks[1]) >= T::kTopScale); }
    __device__ __forceinline__ bool top_values() const {
        if (!E4M3) return false;
        uint32_t most = vs[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) most = max(most, vs[j]);
        return __any(most >= T::kTopScale);
    }
    // Word of codes `w` in 16 bits.  TOP: saturated.  (The scale is opaque there, so that the conversions of
    // the two forms are not taken for the same and moved out of their branches.)
    template <bool HI, bool TOP>
    __device__ static __forceinline__ uint32_t from_code(uint32_t w, uint32_t scale) {
        if (TOP) return saturate<T>(T::template from_e4m3<HI>(w, as_float(opaque(scale))));
        return T::template from_e4m3<HI>(w, as_float(scale));
    }
    // The A operand of key half h, step s, in 16 bits.
    template <bool TOP>
    __device__ __forceinline__ u32x4v key_operand(int h, int s) const {
        u32x4v x;
        if (E4M3) {  // two words of codes per step: channels 16 g + 8 (s % 2) of the 64 of step s / 2
            const uint32_t lo = kr[h][4 * (s / 2) + 2 * (s % 2)], hi = kr[h][4 * (s / 2) + 2 * (s % 2) + 1];
            x[0] = from_code<false, TOP>(lo, ks[h]);
            x[1] = from_code<true, TOP>(lo, ks[h]);
            x[2] = from_code<false, TOP>(hi, ks[h]);
            x[3] = from_code<true, TOP>(hi, ks[h]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = kr[h][4 * s + i];
        }
        return x;
    }
    // The channel that step s, lane group g begins with (the q operand uses the same order).
    __device__ static __forceinline__ int step_channel(int s, int g) {
        return E4M3 ? 64 * (s / 2) + 16 * g + 8 * (s % 2) : 32 * s + 8 * g;
    }
    // Word of channels 2w, 2w+1 of value row j in 16 bits.
    __device__ __forceinline__ uint32_t value_word(int j, int w) const {
        if (E4M3) return w % 2 ? T::template from_e4m3<true>(vr[j][w / 2], as_float(vs[j])) : T::template from_e4m3<false>(vr[j][w / 2], as_float(vs[j]));
        return vr[j][w];
    }
    // The A operands of channels 2w and 2w + 1 of every lane: tokens in pairs.
    __device__ __forceinline__ void value_operands(int w, u32x4v& v0, u32x4v& v1) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = value_word(2 * i, w), y = value_word(2 * i + 1, w);
            v0[i] = __builtin_amdgcn_perm(y, x, 0x05040100u);
            v1[i] = __builtin_amdgcn_perm(y, x, 0x07060302u);
        }
    }
    __device__ __forceinline__ bool any_odd() const {
        bool odd = false;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int w = 0; w < VW / 2; ++w) odd |= T::odd(value_word(j, w));
        return odd;
    }
};

// One item, a row tile: its rows, and the positions that they see.
struct FewItem {
    Seq q;
    int seq, head, tile;
    int low, high, units;  // positions [low, high) are seen by some row; units from low / kFewTokens on
    __device__ __forceinline__ void measure(const AttnArgs& a) {
        tile_range<kFewRows>(a, q, tile, &low, &high);
        units = max(1, (high + kFewTokens - 1) / kFewTokens - low / kFewTokens);
    }
    __device__ __forceinline__ int first_position(int unit) const { return (low / kFewTokens + unit) * kFewTokens; }
};

template <typename T, bool E4M3, int DP>
__global__ __launch_bounds__(64 * kFewWaves) void attention_few_kernel(AttnArgs a) {
    using F = Few<T, E4M3, DP>;
    constexpr int VW = F::VW;
    __shared__ float sh_o[kFewWaves][kFewRows][DP];
    __shared__ float sh_m[kFewWaves][kFewRows], sh_l[kFewWaves][kFewRows];
    __shared__ uint32_t sh_last;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int me = blockIdx.x;
    Work wk;
    if (!find_work<kFewRows, kFewTokens, true>(a, lane, me, gridDim.x, &wk)) return;
    const Cut cut = wk.cut;
    const int end = wk.end, D = a.c.head_dim;

    FewItem it = {wk.q, wk.seq, wk.head, wk.tile};
    it.measure(a);
    int item = wk.u - wk.unit;                 // the slot of the item's first unit
    int first = max(wk.unit, 0), k = first;    // the first unit of it in this range; the present one
    if (item + first >= end) return;

    // What the lane's query row is and sees.
    bool live;
    int see_high, see_low, all_high, all_low;
    u32x4v qr[F::kSteps];
    auto load_queries = [&]() {
        const int row = it.tile * kFewRows + (lane & 15);
        live = row < it.q.rows;
        const int token = row / a.share, qh = it.head * a.share + row % a.share;
        const uint16_t* qp = (const uint16_t*)a.q + (int64_t)(it.q.first + (live ? token : 0)) * a.q_stride + (int64_t)qh * D;
#pragma unroll
        for (int s = 0; s < F::kSteps; ++s) {
            const int d = F::step_channel(s, lane >> 4);
            qr[s] = u32x4v{0u, 0u, 0u, 0u};
            if (live && d < D) qr[s] = *(const u32x4v*)(qp + d);
        }
        const int pos = it.q.len - it.q.n + token;
        see_high = live ? (a.causal ? min(pos + 1, it.q.len) : it.q.len) : 0;
        see_low = a.window ? pos - a.window + 1 : 0;
        // every row sees positions [all_low, all_high): no masks there
        const int tok0 = it.tile * kFewRows / a.share, tok1 = (min(it.q.rows, (it.tile + 1) * kFewRows) - 1) / a.share;
        all_high = a.causal ? min(it.q.len - it.q.n + tok0 + 1, it.q.len) : it.q.len;
        all_low = a.window ? it.q.len - it.q.n + tok1 - a.window + 1 : 0;
    };

    float m = kNoScore, l = 0.f;
    f32x4v o[VW];
    auto clear = [&]() {
        m = kNoScore;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < VW; ++i) o[i] = f32x4v{0.f, 0.f, 0.f, 0.f};
    };

    // The end of an item, or of the part of it in this range: joins the four wavefronts and writes the
    // rows, or a partial result.
    auto finish = [&]() {
        // (worked out here, not kept in registers through the loop)
        const int tid = opaque(threadIdx.x), le = tid & 63;
        l = sum_quarters(l);

        // Join the four wavefronts.
        lds_barrier();
        if (le < 16) {
            sh_m[wave][le] = m;
            sh_l[wave][le] = l;
        }
        if (live) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int i = 0; i < VW; i += 4) {
                    f32x4v x = {o[i][r], o[i + 1][r], o[i + 2][r], o[i + 3][r]};
                    *(f32x4v*)&sh_o[wave][le & 15][VW * (4 * (le >> 4) + r) + i] = x;
                }
        }
        lds_barrier();
        const int rows = min(kFewRows, it.q.rows - it.tile * kFewRows);
        const bool whole = first == 0 && k + 1 == it.units;
        const int owner = whole ? me : cut.owner(item), behind = whole ? me : cut.owner(item + it.units - 1);
        constexpr int kFloats = kFewRows * (DP + 2);  // a pair (maximum, sum) per row, then the rows
        float* mine = a.part + (int64_t)(2 * me + (first == 0 ? 1 : 0)) * kFloats;
        auto write = [&](int r, int d, float L, float x, float y) {  // channels d, d + 1 of row r
            const int rw = it.tile * kFewRows + r;
            const float inv = L != 0.f ? 1.f / L : 0.f;
            uint16_t* op = (uint16_t*)a.o + (int64_t)(it.q.first + rw / a.share) * a.o_stride +
                           (int64_t)(it.head * a.share + rw % a.share) * D + d;
            if (d < D) *(uint32_t*)op = L != 0.f ? T::pack(x * inv, y * inv) : 0u;
        };
        for (int i = tid; i < rows * (DP / 2); i += 64 * kFewWaves) {
            const int r = i / (DP / 2), d = 2 * (i % (DP / 2));
            float M = sh_m[0][r];
#pragma unroll
            for (int w = 1; w < kFewWaves; ++w) M = fmaxf(M, sh_m[w][r]);
            float L = 0.f, x = 0.f, y = 0.f;
#pragma unroll
            for (int w = 0; w < kFewWaves; ++w) {
                const float by = exp2_fast(sh_m[w][r] - M);
                L += by * sh_l[w][r];
                x += by * sh_o[w][r][d];
                y += by * sh_o[w][r][d + 1];
            }
            if (whole) {
                write(r, d, L, x, y);
            } else {
                put2(mine + 2 * kFewRows + r * DP + d, x, y);
                if (d == 0) put2(mine + 2 * r, M, L);
            }
        }
        if (!whole && arrive_last(a.count + owner, (uint32_t)(behind - owner + 1), &sh_last)) {
            // The parts in ascending order, 32 at a time: their maxima and sums through LDS, then each
            // thread's channels, eight loads in flight (a long sequence has a part per workgroup).
            constexpr int kParts = 32, kMine = kFewRows * (DP / 2) / (64 * kFewWaves);
            float* pair = &sh_o[0][0][0];
            float M[kMine], L[kMine], x[kMine], y[kMine];
#pragma unroll
            for (int j = 0; j < kMine; ++j) {
                M[j] = kNoScore;
                L[j] = x[j] = y[j] = 0.f;
            }
            auto part_of = [&](int w) { return a.part + (int64_t)(2 * w + (w == owner ? 1 : 0)) * kFloats; };
            for (int w0 = owner; w0 <= behind; w0 += kParts) {
                const int n = min(kParts, behind - w0 + 1);
                lds_barrier();
                for (int i = tid; i < n * rows; i += 64 * kFewWaves)
                    get2(part_of(w0 + i / rows) + 2 * (i % rows), pair + 2 * i, pair + 2 * i + 1);
                lds_barrier();
#pragma unroll
                for (int j = 0; j < kMine; ++j) {
                    const int i = tid + j * 64 * kFewWaves;
                    if (i >= rows * (DP / 2)) continue;
                    const int r = i / (DP / 2), d = 2 * (i % (DP / 2));
                    float to = M[j];
                    for (int w = 0; w < n; ++w) to = fmaxf(to, pair[2 * (w * rows + r)]);
                    const float b = exp2_fast(M[j] - to);
                    M[j] = to;
                    L[j] *= b;
                    x[j] *= b;
                    y[j] *= b;
                    for (int w1 = 0; w1 < n; w1 += 8) {
                        float x1[8], y1[8];
#pragma unroll
                        for (int w = 0; w < 8; ++w)
                            get2(part_of(w0 + min(w1 + w, n - 1)) + 2 * kFewRows + r * DP + d, &x1[w], &y1[w]);
#pragma unroll
                        for (int w = 0; w < 8; ++w) {
                            if (w1 + w >= n) break;
                            const float b1 = exp2_fast(pair[2 * ((w1 + w) * rows + r)] - to);
                            L[j] += pair[2 * ((w1 + w) * rows + r) + 1] * b1;
                            x[j] += x1[w] * b1;
                            y[j] += y1[w] * b1;
                        }
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kMine; ++j) {
                const int i = tid + j * 64 * kFewWaves;
                if (i < rows * (DP / 2)) write(i / (DP / 2), 2 * (i % (DP / 2)), L[j], x[j], y[j]);
            }
        }
    };

    F f;
    {
        const HeadBase hb(a, it.head, E4M3 ? 1 : 2);
        const int t0 = it.first_position(k) + 32 * wave;
        const int e[2] = {entry_of(a, it.seq, t0), entry_of(a, it.seq, t0 + 16)};
        load_queries();
        // keys before values, here as in the loop: the wait for the older loads then leaves the younger
        // ones in flight
        __builtin_amdgcn_sched_barrier(0);
        f.load_keys(a, hb, e, t0, it.high, lane);
        __builtin_amdgcn_sched_barrier(0);
        f.load_values(a, hb, e, t0, it.low, it.high, lane);
        __builtin_amdgcn_sched_barrier(0);
    }
    clear();
    for (;;) {
        const int t0 = it.first_position(k) + 32 * wave, low = it.low, high = it.high;
        // The unit after this one, maybe the next item's first: its loads are issued while this one is
        // computed, so that an item's end does not drain them.  (Past the range's end nothing is
        // loaded, with the same instructions: no branch between loads, whose number the waits count.)
        FewItem nx = it;
        int nk = k + 1, nitem = item;
        bool more = item + nk < end;
        const bool ends = nk == it.units || !more;
        if (ends && nk == it.units) {
            nitem = item + it.units + kStart;
            more = nitem < end;
            nk = 0;
            if (more) {
                next_item<kFewRows, true>(a, &nx.seq, &nx.head, &nx.tile, &nx.q);
                nx.measure(a);
            }
        }
        const HeadBase hb(a, nx.head, E4M3 ? 1 : 2);
        const int nt = nx.first_position(nk) + 32 * wave, next_high = more ? nx.high : 0;
        const int e[2] = {entry_of(a, nx.seq, nt), entry_of(a, nx.seq, nt + 16)};
        f32x4v s[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            s[h] = f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int st = 0; st < F::kSteps; ++st) s[h] = T::mfma16(f.template key_operand<false>(h, st), qr[st], s[h]);
        }
        if (f.top_keys()) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                s[h] = f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int st = 0; st < F::kSteps; ++st) s[h] = T::mfma16(f.template key_operand<true>(h, st), qr[st], s[h]);
            }
        }
        f.load_keys(a, hb, e, nt, next_high, lane);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = product(s[i / 4][i % 4], a.scale_log2);
        const bool masked = t0 < all_low || t0 + 32 > all_high;
        if (masked) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int t = t0 + 16 * (i / 4) + 4 * (lane >> 4) + i % 4;
                if (t >= see_high || t < see_low) x[i] = -__builtin_inff();
            }
        }
        float most = x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) most = fmaxf(most, x[i]);
        if (__any(most - m > kLazy + T::kWeightBits)) {
            const float to = fmaxf(m, max_quarters(most) - T::kWeightBits);
            const float by = exp2_fast(m - to);
            m = to;
            l *= by;
#pragma unroll
            for (int i = 0; i < VW; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) o[i][r] *= by;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = exp2_fast(x[i] - m);
        u32x4v pb;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            pb[i] = T::pack(x[2 * i], x[2 * i + 1]);
            l = T::add_pair(pb[i], l);  // (as they are multiplied: a mean of equal values is that value)
        }
        bool odd = false;  // an infinity or NaN that some row may not see, or a code past the largest value
        if (masked || f.top_values()) {
            f.mask_scales(t0, low, high, lane);
            odd = __any(f.any_odd());
        }
        if (!odd) {
#pragma unroll
            for (int w = 0; w < VW / 2; ++w) {
                u32x4v v0, v1;
                f.value_operands(w, v0, v1);
                o[2 * w] = T::mfma16(v0, pb, o[2 * w]);
                o[2 * w + 1] = T::mfma16(v1, pb, o[2 * w + 1]);
            }
        } else {
            // 0 * infinity would be NaN in rows that do not see the token: what is finite as
            // ever, the rest one token at a time and added only where it is seen (infinities that codes
            // became, which have none of their own, as the largest value)
#pragma unroll
            for (int w = 0; w < VW / 2; ++w) {
                u32x4v v0, v1, f0, f1;
                f.value_operands(w, v0, v1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f0[i] = T::finite(v0[i]);
                    f1[i] = T::finite(v1[i]);
                    v0[i] ^= f0[i];
                    v1[i] ^= f1[i];
                    if (E4M3) {
                        v0[i] = saturate<T>(v0[i]);
                        v1[i] = saturate<T>(v1[i]);
                    }
                }
                o[2 * w] = T::mfma16(f0, pb, o[2 * w]);
                o[2 * w + 1] = T::mfma16(f1, pb, o[2 * w + 1]);
#pragma unroll 1
                for (int j = 0; j < 32; ++j) {
                    const int t = t0 + 16 * ((j & 7) / 4) + 4 * (j >> 3) + (j & 3);
                    const bool mine = (lane >> 4) == (j >> 3);
                    u32x4v b0, b1;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t keep = mine && (j & 7) / 2 == i ? ((j & 1) ? 0xFFFF0000u : 0x0000FFFFu) : 0u;
                        b0[i] = v0[i] & keep;
                        b1[i] = v1[i] & keep;
                    }
                    const f32x4v z = {0.f, 0.f, 0.f, 0.f};
                    const f32x4v y0 = T::mfma16(b0, pb, z), y1 = T::mfma16(b1, pb, z);
                    if (t < see_high && t >= see_low) {
                        o[2 * w] += y0;
                        o[2 * w + 1] += y1;
                    }
                }
            }
        }
        f.load_values(a, hb, e, nt, nx.low, next_high, lane);
        if (ends) {
            finish();
            if (!more) break;
            clear();
            it = nx;
            first = 0;
            load_queries();
        }
        item = nitem;
        k = nk;
    }
}

template <typename T, bool E4M3>
hipError_t few_dim(const AttnArgs& a, int grid, hipStream_t s) {
    const int D = a.c.head_dim;
    if (D <= 64)
        attention_few_kernel<T, E4M3, 64><<<grid, 64 * kFewWaves, 0, s>>>(a);
    else if (D <= 128)
        attention_few_kernel<T, E4M3, 128><<<grid, 64 * kFewWaves, 0, s>>>(a);
    else
        attention_few_kernel<T, E4M3, 256><<<grid, 64 * kFewWaves, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

int attention_few_grid(int cus) { return 2 * cus; }
int64_t attention_few_floats(int dim) { return kFewRows * ((dim <= 64 ? 64 : dim <= 128 ? 128 : 256) + 2); }

hipError_t launch_attention_few(const AttnArgs& a, int type, int grid, hipStream_t s) {
    const bool e = a.c.type == LSCD_E4M3;
    if (type == LSCD_F16) return e ? few_dim<F16, true>(a, grid, s) : few_dim<F16, false>(a, grid, s);
    return e ? few_dim<BF16, true>(a, grid, s) : few_dim<BF16, false>(a, grid, s);
}

}  // namespace lscd
