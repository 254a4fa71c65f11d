// Attention of new tokens over a paged cache: what its two kernels share.
//
// For query row r (token i of a sequence's n new ones, one of the heads that share a key head):
//   o_r = sum_j exp(s_rj - m_r) v_j / sum_j exp(s_rj - m_r),  s_rj = scale * q_r . k_j,
// over the positions j that the row sees: j <= length - n + i (causal) or j < length, and
// j > that - window.  One pass over the keys and values with a running maximum m and running sums;
// scores are kept in units of log2, so that exp is one v_exp_f32.  A row that sees nothing is zero.
//
// Both kernels compute S^T = K Q^T and O^T = V^T P^T on the matrix cores.  In that orientation a
// lane holds scores of one query row only, so maximum, sum and rescaling are (nearly) lane-local,
// and the scores of a lane are, after rounding to 16 bits, already the B operand of the second
// product: its k index may run over the tokens in any order as long as V^T uses the same one.
// The maximum is moved only when some score exceeds it by 8 (a factor 256, far inside 16-bit
// range for P and fp32 for the sums): most tiles then skip the exchange and the rescaling.
// Sums, maxima and the output accumulate in fp32.  P is rounded once to the model's 16-bit type for the
// second product: a step of 2^-11 or 2^-8 of each weight, that of the values it multiplies (a second
// product with what the rounding leaves out would give every infinity among the values a weight of zero or
// less).  float16 has few exponents, so its weights are held 2^7 times as large (m is that much less), at
// most 2^15: they keep their step down to 2^-21 of the largest and are rounded in steps of 2^-31 of it below.
// Both kernels sum the weights as they multiply them.  Where the logarithm of a row's sum is asked for (lse),
// they sum the weights before that rounding too: ln of the sum as rounded would be off by up to 2^-9 in bfloat16.
//
// Work is split over all sequences, key heads, row tiles and cached positions at once: the units
// (one row tile x one stretch of positions) are numbered in that order and cut into equal ranges,
// one per workgroup, wherever the cuts fall.  An item (row tile) cut by a range's end leaves partial
// results (maximum, sum, unnormalised output), which are added in ascending order, so that results do
// not depend on who arrives when: by the last workgroup to arrive where they are few rows, by a second
// kernel where they are many.  Ragged batches, one long sequence and many short ones all balance.
// Lengths are read on the device: no host copy, no plan.
//
// Sequences of up to 16 query rows (one MFMA tile) are bound by the reading of their keys and values and
// go to the kernel for few rows, longer ones to the other; a call whose batch may hold both launches both.
// (Two tiles of 16 in the kernel for few rows, 32 rows a sequence: 64 sequences of 8 key heads over 2048
// positions 189 us against 111, one sequence over 8192 positions 33 against 23.)
#pragma once

#include "lscd_serve.h"
#include "lscd_serve_device.h"

namespace lscd {
namespace {

constexpr float kNoScore = -3.4028234663852886e38f;  // maximum before any score: finite, so that differences stay
                                                     // defined, and below every finite score
constexpr float kLazy = 8.f;        // how far a score may exceed the maximum before it is moved
constexpr float kLarge = 1048576.f;
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;

// Natural logarithm of a row's sum of exponentials: sum * 2^m, -infinity where there are none.
__device__ __forceinline__ float log_of_sum(float m, float sum) {
    return sum != 0.f ? (m + __builtin_amdgcn_logf(sum)) * kLn2 : -__builtin_inff();
}

// The rows and positions of one sequence.
struct Seq {
    int first;      // its first row in q
    int n, len;     // new tokens; cached positions, new ones among them
    int rows;       // n * share
};

// Starts, lengths and tables do not change while a kernel runs: read as constants, so that uniform
// reads are scalar loads, which do not queue behind the loads of keys and values.
typedef __attribute__((address_space(4))) const int32_t const_i32;

// Reads are clamped to what the arguments allow, whatever the arrays hold.
__device__ __forceinline__ Seq read_seq(const AttnArgs& a, int s) {
    Seq q;
    const const_i32* start = (const const_i32*)(uintptr_t)a.start;
    const const_i32* length = (const const_i32*)(uintptr_t)a.length;
    const int64_t b0 = min(max((int64_t)start[s], (int64_t)0), a.T);
    const int64_t b1 = min(max((int64_t)start[s + 1], b0), a.T);
    q.first = (int)b0;
    q.n = (int)(b1 - b0);
    q.len = min(max((int64_t)length[s], (int64_t)0), (int64_t)a.table_pages << a.page_log2);
    q.rows = q.n * a.share;
    return q;
}

// Positions [low, high) that some row of tile `t` (ROWS rows) sees.
template <int ROWS>
__device__ __forceinline__ void tile_range(const AttnArgs& a, const Seq& q, int t, int* low, int* high) {
    const int i0 = t * ROWS / a.share, i1 = (min(q.rows, (t + 1) * ROWS) - 1) / a.share;
    const int p0 = q.len - q.n + i0, p1 = q.len - q.n + i1;
    *high = a.causal ? min(max(p1 + 1, 0), q.len) : q.len;
    *low = a.window ? min(max(p0 - a.window + 1, 0), *high) : 0;
}
template <int ROWS, int TOKENS>
__device__ __forceinline__ int tile_units(const AttnArgs& a, const Seq& q, int t) {
    int low, high;
    tile_range<ROWS>(a, q, t, &low, &high);
    return max(1, (high + TOKENS - 1) / TOKENS - low / TOKENS);
}
// The units are laid out on a line, sequence after sequence, key head after key head, row tile after
// row tile; kStart slots before an item's units stand for what its start and end cost.  Slots of one
// key head of the sequence; 0 if it belongs to the other kernel.
constexpr int kStart = 1;
template <int ROWS, int TOKENS, bool FEW>
__device__ __forceinline__ int head_slots(const AttnArgs& a, const Seq& q) {
    if (q.rows == 0 || (q.rows <= a.few_limit) != FEW) return 0;
    int u = 0;
    for (int t = 0; t * ROWS < q.rows; ++t) u += tile_units<ROWS, TOKENS>(a, q, t) + kStart;
    return u;
}

// The cut of U slots into G ranges whose sizes differ by at most one.
struct Cut {
    int base, extra;
    Cut() = default;
    __device__ __forceinline__ Cut(int U, int G) : base(U / G), extra(U % G) {}
    __device__ __forceinline__ int begin(int w) const { return w * base + (w < extra ? w : extra); }
    __device__ __forceinline__ int owner(int u) const {
        const int big = extra * (base + 1);
        return u < big ? u / (base + 1) : extra + (u - big) / base;
    }
};

// A workgroup's range of slots, and the item it begins in: sequence, key head, row tile, unit (or
// -1, -2 .. in the slots before its units).
struct Work {
    Cut cut;
    int u, end;
    int seq, head, tile, unit;
    Seq q;
};
// The caller sees to it that sequences which share no token have fewer slots than this.  Starts that do not
// ascend may make them more: sums saturate, and all workgroups leave.
constexpr int kMostSlots = 0x7FFFFFFF;
// Works it out (every wavefront for itself, 64 sequences at a time).  False: there is nothing to do.
template <int ROWS, int TOKENS, bool FEW>
__device__ __forceinline__ bool find_work(const AttnArgs& a, int lane, int me, int G, Work* w) {
    auto slots_of = [&](int s, Seq* q) {
        if (s >= a.sequences) return 0;
        *q = read_seq(a, s);
        return head_slots<ROWS, TOKENS, FEW>(a, *q);
    };
    auto scan = [&](int x) {  // inclusive sums over the lanes
        for (int d = 1; d < 64; d <<= 1) {
            const int up = __shfl_up(x, d, 64);
            if (lane >= d) x = __builtin_elementwise_add_sat(x, up);
        }
        return x;
    };
    Seq q = {};
    int per = slots_of(lane, &q), sum = scan(per * a.c.heads);
    int U = __builtin_amdgcn_readlane(sum, 63);
    for (int s0 = 64; s0 < a.sequences; s0 += 64) {
        Seq other = {};
        U = __builtin_elementwise_add_sat(U, __builtin_amdgcn_readlane(scan(slots_of(s0 + lane, &other) * a.c.heads), 63));
    }
    if (U == kMostSlots) return false;
    w->cut = Cut(U, G);
    w->u = w->cut.begin(me);
    w->end = w->cut.begin(me + 1);
    if (w->u >= w->end) return false;
    int before = 0, s0 = 0;
    for (;;) {
        const uint64_t past = __ballot(before + sum > w->u);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int ph = __builtin_amdgcn_readlane(per, l);
            const int rest = w->u - (before + __builtin_amdgcn_readlane(sum, l) - ph * a.c.heads);
            w->seq = s0 + l;
            w->head = rest / ph;
            w->unit = rest % ph;
            w->q.first = __builtin_amdgcn_readlane(q.first, l);
            w->q.n = __builtin_amdgcn_readlane(q.n, l);
            w->q.len = __builtin_amdgcn_readlane(q.len, l);
            w->q.rows = __builtin_amdgcn_readlane(q.rows, l);
            break;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
        s0 += 64;
        q = Seq{};
        per = slots_of(s0 + lane, &q);
        sum = scan(per * a.c.heads);
    }
    for (w->tile = 0; (w->tile + 1) * ROWS < w->q.rows; ++w->tile) {
        const int n = tile_units<ROWS, TOKENS>(a, w->q, w->tile) + kStart;
        if (w->unit < n) break;
        w->unit -= n;
    }
    w->unit -= kStart;
    return true;
}

// The next item that belongs to this kernel; there has to be one.
template <int ROWS, bool FEW>
__device__ __forceinline__ void next_item(const AttnArgs& a, int* seq, int* head, int* tile, Seq* q) {
    if ((++*tile) * ROWS < q->rows) return;
    *tile = 0;
    if (++*head < a.c.heads) return;
    *head = 0;
    do {
        ++*seq;
        *q = read_seq(a, *seq);
    } while (q->rows == 0 || (q->rows <= a.few_limit) != FEW);
}

// The table's entry for position t (the last one behind the table), and the page it names (an entry
// outside the pool is read as page 0).
__device__ __forceinline__ int entry_of(const AttnArgs& a, int seq, int t) {
    const int i = min(t >> a.page_log2, a.table_pages - 1);
    return ((const const_i32*)(uintptr_t)a.table)[seq * a.table_stride + i];
}
__device__ __forceinline__ uint32_t page_of(const AttnArgs& a, int entry) {
    return (uint32_t)entry < (uint32_t)a.c.num_pages ? (uint32_t)entry : 0u;
}

// One key head's part of the cache: its block of page 0, and the bytes from a page's to the next's.
struct HeadBase {
    const uint8_t *k, *v;
    const uint8_t *ks, *vs;
    uint64_t page, page_scales;
    int block, block_scales;  // bytes of one page's block
    // BITS: of one value; SCALES: bytes of one token's scales
    template <int BITS, int SCALES>
    __device__ __forceinline__ void set(const lscd_cache_t& c, int head) {
        block = c.page_size * c.head_dim / 8 * BITS;
        block_scales = c.page_size * SCALES;
        page = (uint64_t)c.heads * block;
        page_scales = (uint64_t)c.heads * block_scales;
        k = (const uint8_t*)c.k + (uint64_t)head * block;
        v = (const uint8_t*)c.v + (uint64_t)head * block;
        ks = (const uint8_t*)c.k_scale + (uint64_t)head * block_scales;
        vs = (const uint8_t*)c.v_scale + (uint64_t)head * block_scales;
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t keys(uint32_t p) const { return buffer_of(k + p * page, block); }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t values(uint32_t p) const { return buffer_of(v + p * page, block); }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t key_scales(uint32_t p) const {
        return buffer_of(ks + p * page_scales, block_scales);
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t value_scales(uint32_t p) const {
        return buffer_of(vs + p * page_scales, block_scales);
    }
};

// Key rows of 16 positions as an operand of the 16 x 16 x 32 matrix instructions, straight from memory: the
// lane's row is position lane % 16, its channels are those of step_channel().  FORM: how the cache holds its
// values.  DP: channels padded to 64, 128 or 256.  TILES: of 16 positions.
template <typename T, int FORM, int DP, int TILES = 2>
struct Keys {
    static constexpr int kTiles = TILES;
    static constexpr bool kScaled = FORM != kForm16;
    static constexpr int kBits = form_bits(FORM);
    static constexpr int kScaleBytes = FORM == kForm4 ? scale_row(DP) : 4;  // of one token's scales
    static constexpr int kSteps = DP / 32;  // MFMA steps over the channels of q . k
    static constexpr int kKeyRegs = DP * kBits / 128;                       // words of one 16-token key tile per lane
    static constexpr int kKeyScales = FORM == kForm4 && DP == 256 ? 2 : 1;    // scales of one key tile per lane
    // 1 as a scale is loaded
    static constexpr uint32_t kOne = FORM == kForm4 ? 127u : 0x3F800000u, kTop = FORM == kForm4 ? T::kTopScale4 : T::kTopScale;
    uint32_t kr[TILES][kKeyRegs];
    uint32_t ks[TILES][kKeyScales];  // scales as loaded: bits of a float (e4m3), exponent + 127 (e2m1)

    // A key row of 4-bit codes lies in the four lane groups as 16 channels each, of 64 (DP 64), or as 32 each, of
    // 128: the lane's channels of unit u of them have one scale.  Rows that end in the middle of 32 channels are
    // loaded to their end, 16 channels too early; the query has zeros there.
    __device__ static __forceinline__ int unit_channel(int u, int g) { return DP == 64 ? 16 * g : 128 * u + 32 * g; }
    __device__ static __forceinline__ int unit_start(int u, int g, int D) {
        return DP == 64 ? unit_channel(u, g) : min(unit_channel(u, g), D - 32);
    }

    // Tile h: 16 positions from row `row` of a page on, whose keys and scales the descriptors are of; lanes whose
    // position is not `on` have zeros (they read outside the descriptor, which costs no traffic).  Offsets are the
    // lane's, which do not change, and the tile's first row's, a scalar.
    __device__ __forceinline__ void load_tile(int h, __amdgpu_buffer_rsrc_t rs, __amdgpu_buffer_rsrc_t scales, int D, int row,
                                              bool on, int lane) {
        const int r = lane & 15, g = lane >> 4, at = row * D * kBits / 8;
        if (FORM == kForm8) {
#pragma unroll
            for (int u = 0; u < DP / 64; ++u) {
                const int d = 64 * u + 16 * g;
                const u32x4v x = __builtin_amdgcn_raw_buffer_load_b128(rs, on && d < D ? r * D + d : kNoRow, at, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) kr[h][4 * u + i] = x[i];
            }
            ks[h][0] = __builtin_amdgcn_raw_buffer_load_b32(scales, on ? r * 4 : kNoRow, row * 4, 0);
        } else if (FORM == kForm4) {
#pragma unroll
            for (int u = 0; u < kKeyScales; ++u) {
                const int d = unit_channel(u, g);
                const int off = on && d < D ? (r * D + unit_start(u, g, D)) / 2 : kNoRow;
                if constexpr (DP == 64) {
                    const u32x2v x = __builtin_amdgcn_raw_buffer_load_b64(rs, off, at, 0);
                    kr[h][0] = x[0];
                    kr[h][1] = x[1];
                } else {
                    const u32x4v x = __builtin_amdgcn_raw_buffer_load_b128(rs, off, at, 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i) kr[h][4 * u + i] = x[i];
                }
                ks[h][u] = __builtin_amdgcn_raw_buffer_load_b8(
                    scales, on && d < D ? r * kScaleBytes + d / kScaleGroup : kNoRow, row * kScaleBytes, 0);
            }
        } else {
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int d = 32 * s + 8 * g;
                const u32x4v x = __builtin_amdgcn_raw_buffer_load_b128(rs, on && d < D ? (r * D + d) * 2 : kNoRow, at, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) kr[h][4 * s + i] = x[i];
            }
        }
    }
    // 16 TILES positions from t0 on, in the pages of the table entries e; positions from `high` on are zero.
    // (Not by load_tile: with its scalar offsets the attention over e4m3 heads of 64 channels took 231 us in place of
    // 216, one sequence over 32768 positions 28.7 in place of 26.0.)
    __device__ __forceinline__ void load_keys(const AttnArgs& a, const HeadBase& hb, const int (&e)[TILES], int t0, int high,
                                              int lane) {
        static_assert(FORM != kForm4, "4-bit codes are loaded tile by tile");
        const int D = a.c.head_dim;
#pragma unroll
        for (int h = 0; h < TILES; ++h) {
            const int t = t0 + 16 * h, row = (t & (a.c.page_size - 1)) + (lane & 15);
            const uint32_t p = page_of(a, e[h]);
            const bool on = t + (lane & 15) < high;
            const auto rs = hb.keys(p);
            if (FORM == kForm8) {
#pragma unroll
                for (int u = 0; u < DP / 64; ++u) {
                    const int d = 64 * u + 16 * (lane >> 4);
                    const u32x4v x = __builtin_amdgcn_raw_buffer_load_b128(rs, on && d < D ? row * D + d : kNoRow, 0, 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i) kr[h][4 * u + i] = x[i];
                }
                ks[h][0] = __builtin_amdgcn_raw_buffer_load_b32(hb.key_scales(p), on ? row * 4 : kNoRow, 0, 0);
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

    // Whether some key's code times its scale may pass the type's largest value.  (Scales are positive: they
    // compare as whole numbers.)
    __device__ __forceinline__ bool top_keys() const {
        if (!kScaled) return false;
        uint32_t most = 0u;
#pragma unroll
        for (int h = 0; h < TILES; ++h)
#pragma unroll
            for (int u = 0; u < kKeyScales; ++u) most = max(most, ks[h][u]);
        return __any(most >= kTop);
    }
    // Word of codes `w` in 16 bits.  TOP: saturated.  (The scale is opaque there, so that the conversions of
    // the two forms are not taken for the same and moved out of their branches.)
    template <bool HI, bool TOP>
    __device__ static __forceinline__ uint32_t from_code(uint32_t w, uint32_t scale) {
        if (TOP) return saturate<T>(T::template from_e4m3<HI>(w, as_float(opaque(scale))));
        return T::template from_e4m3<HI>(w, as_float(scale));
    }
    template <int B, bool TOP>
    __device__ static __forceinline__ uint32_t from_code4(uint32_t w, uint32_t scale) {
        if (TOP) return saturate<T>(T::template from_e2m1<B>(w, as_float(opaque(scale << 23))));
        return T::template from_e2m1<B>(w, as_float(scale << 23));
    }
    // The A operand of key half h, step s, in 16 bits.
    template <bool TOP>
    __device__ __forceinline__ u32x4v key_operand(int h, int s) const {
        u32x4v x;
        if constexpr (FORM == kForm4) {  // one word of codes per step
            x[0] = from_code4<0, TOP>(kr[h][s], ks[h][s / 4]);
            x[1] = from_code4<1, TOP>(kr[h][s], ks[h][s / 4]);
            x[2] = from_code4<2, TOP>(kr[h][s], ks[h][s / 4]);
            x[3] = from_code4<3, TOP>(kr[h][s], ks[h][s / 4]);
        } else if constexpr (FORM == kForm8) {  // two words of codes per step: channels 16 g + 8 (s % 2) of the 64 of step s / 2
            const uint32_t lo = kr[h][4 * (s / 2) + 2 * (s % 2)], hi = kr[h][4 * (s / 2) + 2 * (s % 2) + 1];
            x[0] = from_code<false, TOP>(lo, ks[h][0]);
            x[1] = from_code<true, TOP>(lo, ks[h][0]);
            x[2] = from_code<false, TOP>(hi, ks[h][0]);
            x[3] = from_code<true, TOP>(hi, ks[h][0]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = kr[h][4 * s + i];
        }
        return x;
    }
    // The channel that step s, lane group g begins with (the q operand uses the same order); D and more where it
    // has none.
    __device__ static __forceinline__ int step_channel(int s, int g, int D) {
        if (FORM == kForm4) {
            const int d = unit_start(s / 4, g, D) + 8 * (s % 4);
            return d < unit_channel(s / 4, g) ? D : d;
        }
        return FORM == kForm8 ? 64 * (s / 2) + 16 * g + 8 * (s % 2) : 32 * s + 8 * g;
    }
};

// Partial results travel between workgroups, maybe on different XCDs, by relaxed agent-scope accesses:
// the stores go through to memory and the loads come from there, whatever the L2 caches hold.  (A
// release fence would write back and an acquire fence invalidate a whole L2 instead; under full load a
// fence per cut took longer than the rest: 584 us against 310 us for 64 ragged sequences of 96 heads.)
__device__ __forceinline__ void put2(float* p, float x, float y) {
    const uint64_t w = (uint64_t)__builtin_bit_cast(uint32_t, y) << 32 | __builtin_bit_cast(uint32_t, x);
    __hip_atomic_store((uint64_t*)p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void get2(const float* p, float* x, float* y) {
    const uint64_t w = __hip_atomic_load((uint64_t*)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *x = as_float((uint32_t)w);
    *y = as_float((uint32_t)(w >> 32));
}
// Counts this workgroup's arrival after its put2 stores have completed (the wait below: a store that
// goes through is counted off when it has reached memory).  Returns whether it is the last of
// `expected`, and clears the count for the next call.
__device__ __forceinline__ bool arrive_last(uint32_t* count, uint32_t expected, uint32_t* shared) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t before = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *shared = before + 1 == expected;
        if (before + 1 == expected) __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    return *shared != 0;
}

}  // namespace
}  // namespace lscd
