// The softmax weights that new tokens give to the cached positions, added up per position and key head:
//   weight[j] (+)= sum over the sequence's query rows r of the key head of exp(scale * q_r . k_j - lse_r),
// over the rows that see position j; lse_r is what the attention found for the row, so that one pass over the
// keys is enough and every position's sum is finished where its keys are: no partial results, no atomics, a
// fixed order of addition.  Positions of the new tokens themselves start from the sum, it is added to the others'.
//
// S = Q K^T on the matrix cores: a lane then holds scores of one position and of four rows, whose sum is taken in
// the lane and over its quarters.  Products are exact and sums fp32, as in the attention.
//
// Few rows: the units (stretches of positions of one sequence and key head) are numbered sequence after sequence,
// head after head, and cut into equal ranges by what they cost, one for each wavefront; a unit belongs to the range
// in which its first slot lies.  Twice as many wavefronts as run at once even out what they wait for (64 sequences
// of one token over up to 2048 positions of 96 heads, 4-bit codes: 114 us, 121 with half as many).
//
// Measured: those 497 MB in 114 us, 4.4 TB/s; 1500 tokens of 32 heads over 8000 positions of 8 (89 GFLOP and 348
// million exponentials) in 121 us, 740 TFLOP/s; 4096 over 16384 in 561 us, 858 TFLOP/s.  Over e4m3 122 us, over e2m1
// 123, in float16 125; heads of 64 channels 82, of 256 277, one workgroup a CU.  One token each over 16-bit caches 365 us
// (1.72 GB, 4.7 TB/s), over e4m3 207 (914 MB, 4.4 TB/s).

#include "lscd_attention.h"

namespace lscd {
namespace {

constexpr int kWeighWaves = 4;
// Key tiles of 16 positions in a unit of the kernel for few rows: the fewer bytes a row has, the more of them.
constexpr int weigh_tiles(int form, int dp) { return form == kForm4 && dp <= 128 ? 4 : 2; }
static_assert(kWeighTokens == 32, "no unit is smaller");

// What the rows of a sequence see together: positions [low, high), in `units` stretches; a unit costs a slot for
// every tile of 16 rows.
template <int TOKENS>
struct Stretch {
    int low, high, units, cost;
    __device__ __forceinline__ void measure(const AttnArgs& a, const Seq& q) {
        // (the last token sees all with or without causality)
        high = q.rows > 0 && q.rows <= a.few_limit ? q.len : 0;
        low = a.window ? min(max(q.len - q.n - a.window + 1, 0), high) : 0;
        units = high > low ? (high + TOKENS - 1) / TOKENS - low / TOKENS : 0;
        cost = (q.rows + kFewRows - 1) / kFewRows;
    }
};

// Where a range begins: the first unit whose first slot is in it.
template <int TOKENS>
struct WeighWork {
    int u, end;  // that slot; the range's end
    int seq, head, unit;
    Seq q;
    Stretch<TOKENS> st;
};
template <int TOKENS>
__device__ __forceinline__ bool find_weigh(const AttnArgs& a, int lane, int me, int G, WeighWork<TOKENS>* w) {
    auto slots_of = [&](int s, Seq* q) {
        if (s >= a.sequences) return 0;
        *q = read_seq(a, s);
        Stretch<TOKENS> st;
        st.measure(a, *q);
        return st.units * st.cost;
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
    const Cut cut(U, G);
    w->u = cut.begin(me);
    w->end = cut.begin(me + 1);
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
            w->unit = rest % ph;  // (in slots, so far)
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
    w->st.measure(a, w->q);
    const int in = w->unit, unit = (in + w->st.cost - 1) / w->st.cost;
    w->u += unit * w->st.cost - in;
    w->unit = unit;
    return true;
}

// To the unit that w names, which may be another head's or sequence's first; false past the range's end.
template <int TOKENS>
__device__ __forceinline__ bool settle(const AttnArgs& a, WeighWork<TOKENS>* w) {
    if (w->u >= w->end) return false;
    if (w->unit < w->st.units) return true;
    w->unit = 0;
    if (++w->head < a.c.heads) return true;
    w->head = 0;
    do {
        ++w->seq;
        w->q = read_seq(a, w->seq);
        w->st.measure(a, w->q);
    } while (w->st.units == 0);
    return true;
}

__device__ __forceinline__ int share_of(const AttnArgs& a, int row) {  // row / a.share
    return (int)((uint64_t)(uint32_t)row * a.share_magic >> a.share_shift);
}

// Where the pages of a sequence hold one key head: lane l has the addresses of its keys, scales and weights in the
// page of table entry base + l, worked out for 64 pages at a time and read from there as scalars.
struct Window {
    int seq, head, base;
    uint32_t k_lo, k_hi, s_lo, s_hi, w_lo, w_hi;  // weights: null for a page outside the pool

    template <int BITS, int SCALES>
    __device__ __forceinline__ void fill(const AttnArgs& a, int sq, int hd, int page, int lane) {
        seq = sq;
        head = hd;
        base = page;
        const int32_t e = a.table[seq * a.table_stride + min(page + lane, a.table_pages - 1)];
        const int64_t row = ((int64_t)page_of(a, e) * a.c.heads + head) * a.c.page_size;  // the page's first
        const uint64_t k = (uint64_t)a.c.k + row * (a.c.head_dim * BITS / 8), s = (uint64_t)a.c.k_scale + row * SCALES;
        const uint64_t w = (uint32_t)e < (uint32_t)a.c.num_pages ? (uint64_t)(a.weight + row) : 0;
        k_lo = (uint32_t)k;
        k_hi = (uint32_t)(k >> 32);
        s_lo = (uint32_t)s;
        s_hi = (uint32_t)(s >> 32);
        w_lo = (uint32_t)w;
        w_hi = (uint32_t)(w >> 32);
    }
    __device__ static __forceinline__ uint64_t at(uint32_t lo, uint32_t hi, int page) {
        return (uint64_t)(uint32_t)__builtin_amdgcn_readlane(hi, page) << 32 | (uint32_t)__builtin_amdgcn_readlane(lo, page);
    }
};

// Few rows: bound by the reading of the keys.  A wavefront loads the next unit's keys into the registers of the
// present one's as soon as its products are issued, before the exponentials, and keeps its query rows while
// sequence and head stay the same.
template <typename T, int FORM, int DP>
__global__ __launch_bounds__(64 * kWeighWaves, (DP <= 64 || (FORM == kForm4 && DP <= 128) ? 4 : DP <= 128 ? 3 : 2)) void weigh_few_kernel(AttnArgs a) {
    constexpr int kTiles = weigh_tiles(FORM, DP), kTokens = 16 * kTiles;
    using F = Keys<T, FORM, DP, kTiles>;
    using Work = WeighWork<kTokens>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Work w;
    if (!find_weigh(a, lane, blockIdx.x * kWeighWaves + wave, gridDim.x * kWeighWaves, &w) || !settle(a, &w)) return;
    const int D = a.c.head_dim, g = lane >> 4;
    const int row_bytes = D * F::kBits / 8, key_block = a.c.page_size * row_bytes, scale_block = a.c.page_size * F::kScaleBytes;

    F f;
    Window win;
    win.seq = -1;
    // (past the range's end nothing is loaded, by the same instructions: the waits count them)
    auto load_keys = [&](const Work& w, bool more) {
        const int t0 = (w.st.low / kTokens + w.unit) * kTokens;
        if (w.seq != win.seq || w.head != win.head || ((t0 + kTokens - 1) >> a.page_log2) - win.base >= 64)
            win.fill<F::kBits, F::kScaleBytes>(a, w.seq, w.head, t0 >> a.page_log2, lane);
        const int high = more ? w.st.high : 0;
#pragma unroll
        for (int h = 0; h < kTiles; ++h) {
            const int t = t0 + 16 * h, i = (t >> a.page_log2) - win.base;
            f.load_tile(h, buffer_of((const void*)Window::at(win.k_lo, win.k_hi, i), key_block),
                        F::kScaled ? buffer_of((const void*)Window::at(win.s_lo, win.s_hi, i), scale_block) : buffer_of(nullptr, 0),
                        D, t & (a.c.page_size - 1), t + (lane & 15) < high, lane);
        }
    };
    // The place of the lane's position's weight (as many lanes as positions), null if it has none, and what is there.
    float* place = nullptr;
    float old = 0.f;
    auto load_weight = [&](const Work& w) {
        const int t = (w.st.low / kTokens + w.unit) * kTokens + (lane & (kTokens - 1)), i = (t >> a.page_log2) - win.base;
        const uint64_t at = (uint64_t)(uint32_t)__shfl((int)win.w_hi, i, 64) << 32 | (uint32_t)__shfl((int)win.w_lo, i, 64);
        const bool own = lane < kTokens && t >= w.st.low && t < w.st.high && at != 0;
        place = own ? (float*)at + (t & (a.c.page_size - 1)) : nullptr;
        old = *(own ? place : a.weight);
    };
    // The query rows of a tile; rows that are none repeat the last one, and weigh nothing.  One whose logarithm is
    // -infinity sees nothing: 2^(score - infinity) would be NaN where the score is.
    u32x4v qr[F::kSteps];
    float log[4];  // of the rows whose scores the lane has, in units of log2
    int see_high[4], see_low[4], all_high, all_low;
    auto queries = [&](const Work& w, int tile) {
        auto row = [&](int r, int* token, int* head) {
            const int x = min(tile * kFewRows + r, w.q.rows - 1);
            *token = share_of(a, x);
            *head = w.head * a.share + x - *token * a.share;
        };
        int token, head;
        row(lane & 15, &token, &head);
        const uint16_t* qp = (const uint16_t*)a.q + (int64_t)(w.q.first + token) * a.q_stride + (int64_t)head * D;
#pragma unroll
        for (int s = 0; s < F::kSteps; ++s) {
            const int d = F::step_channel(s, g, D);
            qr[s] = u32x4v{0u, 0u, 0u, 0u};
            if (d < D) qr[s] = *(const u32x4v*)(qp + d);
        }
        all_high = w.q.len;
        all_low = 0;
        bool out = false;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            row(4 * g + r, &token, &head);
            const float x = a.row_lse[(int64_t)(w.q.first + token) * a.q_heads + head];
            const bool none = x == -__builtin_inff();
            out |= none;
            log[r] = tile * kFewRows + 4 * g + r < w.q.rows ? x * kLog2e : __builtin_inff();
            const int pos = w.q.len - w.q.n + token;
            see_high[r] = none ? 0 : a.causal ? min(pos + 1, w.q.len) : w.q.len;
            see_low[r] = a.window ? pos - a.window + 1 : 0;
        }
        // what every row sees: the first one's end, the last one's begin
        if (a.causal) all_high = __builtin_amdgcn_readfirstlane(see_high[0]);
        if (a.window) all_low = __builtin_amdgcn_readlane(see_low[3], 48);
        if (__any(out)) all_high = 0;
    };

    // Scores of the tile of rows in qr with the keys in f, and what they weigh.
    f32x4v s[kTiles];
    auto products = [&]() {
#pragma unroll
        for (int h = 0; h < kTiles; ++h) s[h] = f32x4v{0.f, 0.f, 0.f, 0.f};
        if (!f.top_keys()) {
#pragma unroll
            for (int h = 0; h < kTiles; ++h)
#pragma unroll
                for (int st = 0; st < F::kSteps; ++st) s[h] = T::mfma16(qr[st], f.template key_operand<false>(h, st), s[h]);
        } else {
#pragma unroll
            for (int h = 0; h < kTiles; ++h)
#pragma unroll
                for (int st = 0; st < F::kSteps; ++st) s[h] = T::mfma16(qr[st], f.template key_operand<true>(h, st), s[h]);
        }
    };
    float sum[kTiles];
    auto weigh = [&](int t0) {
#pragma unroll
        for (int h = 0; h < kTiles; ++h)
#pragma unroll
            for (int r = 0; r < 4; ++r) s[h][r] = exp2_fast(__builtin_fmaf(s[h][r], a.scale_log2, -log[r]));
        if (t0 < all_low || t0 + kTokens > all_high) {
#pragma unroll
            for (int h = 0; h < kTiles; ++h) {
                const int t = t0 + 16 * h + (lane & 15);
#pragma unroll
                for (int r = 0; r < 4; ++r) s[h][r] = t < see_high[r] && t >= see_low[r] ? s[h][r] : 0.f;
            }
        }
#pragma unroll
        for (int h = 0; h < kTiles; ++h) sum[h] += (s[h][0] + s[h][1]) + (s[h][2] + s[h][3]);
    };

    load_keys(w, true);
    load_weight(w);
    int seq = -1, head = -1;
    for (;;) {
        Work nw = w;
        nw.u += w.st.cost;
        ++nw.unit;
        const bool more = settle(a, &nw);
        if (!more) nw = w;
        const int t0 = (w.st.low / kTokens + w.unit) * kTokens, last = w.st.cost - 1;
#pragma unroll
        for (int h = 0; h < kTiles; ++h) sum[h] = 0.f;
        for (int tile = 0; tile < last; ++tile) {
            queries(w, tile);
            products();
            weigh(t0);
        }
        if (last || w.seq != seq || w.head != head) queries(w, last);
        seq = last ? -1 : w.seq;
        head = w.head;
        products();
        load_keys(nw, more);
        weigh(t0);
        // the sums over the four quarters, that of tile h in quarter h (of two tiles: in h and h + 2)
        float y = add_quarters(sum[0], sum[1]);
        y = kTiles == 4 ? add_halves(y, add_quarters(sum[kTiles - 2], sum[kTiles - 1])) : sum_halves(y);
        if (place) *place = (t0 + (lane & (kTokens - 1)) < w.q.len - w.q.n ? old : 0.f) + y;
        if (!more) break;
        w = nw;
        load_weight(w);
    }
}

// Many rows: a workgroup has a block of positions, whose keys its four wavefronts all hold in registers (as 16-bit
// values) while they stream the query rows past them, 64 at a time and every wavefront its own; at the end the
// four sums of each position are added.  A wavefront brings its next rows into its part of LDS by loads that pass
// no registers, 32 rows as soon as those before them are read: no barrier inside the loop.  Per 32 rows and 128
// positions of 128 channels that is 8 KB of LDS read against 32 matrix instructions of 32 cycles, and 64
// exponentials of 16 cycles with two more instructions each beside them, which bound it.
// TILES: key tiles of 32 positions, what the registers hold (4, or 2 of 256 channels), or 1 where there would be
// fewer blocks than compute units.
template <typename T, int FORM, int DP, int TILES>
struct Block {
    static constexpr int kTiles = TILES;
    static constexpr int kTokens = 32 * kTiles;
    static constexpr int kSteps = DP / 16;                 // matrix instructions of a tile
    static constexpr int kChunks = DP <= 64 ? 8 : DP <= 128 ? 16 : 32;  // 16-byte chunks of a query row in LDS
    static constexpr int kRowMask = DP <= 64 ? 7 : 15;
    static constexpr int kRow = 16 * kChunks, kHalf = 32 * kRow;  // bytes of a query row and of 32
    static constexpr int kBits = form_bits(FORM);
    static constexpr int kScaleBytes = FORM == kForm4 ? scale_row(DP) : 4;

    // The chunk of channels that step s has in the lanes of half `half`: what one load of a key row brings.
    __device__ static __forceinline__ int chunk(int s, int half) {
        return FORM == kForm4 ? 8 * (s / 4) + 4 * half + s % 4 : FORM == kForm8 ? 4 * (s / 2) + 2 * half + s % 2 : 2 * s + half;
    }

    u32x4v key[kTiles][kSteps];

    // Positions t0 .. of the lane's columns; zeros outside [low, high) and behind a row's end.
    __device__ __forceinline__ void load(const AttnArgs& a, int seq, int head, int t0, int low, int high, int lane) {
        const int D = a.c.head_dim, half = lane >> 5, page = a.c.page_size;
        const int bytes = D * kBits / 8;
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            const int t = t0 + 32 * i + (lane & 31);
            const bool on = t >= low && t < high;
            const uint32_t p = on ? page_of(a, a.table[seq * a.table_stride + (t >> a.page_log2)]) : 0u;
            const int64_t row = ((int64_t)p * a.c.heads + head) * page + (t & (page - 1));
            const uint8_t* k = (const uint8_t*)a.c.k + row * bytes;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int d = 8 * chunk(s, half);
                u32x4v x = {0u, 0u, 0u, 0u};
                if (on && d < D) {
                    if constexpr (FORM == kForm4) {
                        const uint32_t w = *(const uint32_t*)(k + d / 2);
                        const uint32_t by = ((const uint8_t*)a.c.k_scale)[row * scale_row(D) + d / kScaleGroup];
                        const float scale = as_float(by << 23);
                        x = u32x4v{T::template from_e2m1<0>(w, scale), T::template from_e2m1<1>(w, scale),
                                   T::template from_e2m1<2>(w, scale), T::template from_e2m1<3>(w, scale)};
                    } else if constexpr (FORM == kForm8) {
                        const u32x2v w = *(const u32x2v*)(k + d);
                        const float scale = a.c.k_scale[row];
                        x = u32x4v{T::template from_e4m3<false>(w[0], scale), T::template from_e4m3<true>(w[0], scale),
                                   T::template from_e4m3<false>(w[1], scale), T::template from_e4m3<true>(w[1], scale)};
                    } else {
                        x = *(const u32x4v*)(k + 2 * d);
                    }
                    if constexpr (FORM != kForm16)
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[j] = saturate<T>(x[j]);
                }
                key[i][s] = x;
            }
        }
    }
};

// 16 bytes a lane from memory into LDS, lane after lane from `to` on (a byte offset, the same in all lanes).  In
// assembly: the compiler would wait for every such load before any later read of LDS.  What reads the bytes waits
// for vmcnt by itself.
typedef __attribute__((address_space(3))) const void lds_void;
__device__ __forceinline__ void load_to_lds(const void* from, uint32_t to) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "s"(to) : "memory", "m0");
}

// The units of the kernel for many rows: kTokens positions of one sequence and key head.
template <int TOKENS>
__device__ __forceinline__ int block_units(const AttnArgs& a, const Seq& q, int* low, int* high) {
    const bool mine = q.rows > a.few_limit;
    *high = mine ? q.len : 0;
    *low = a.window ? min(max(q.len - q.n - a.window + 1, 0), *high) : 0;
    return *high > *low ? (*high + TOKENS - 1) / TOKENS - *low / TOKENS : 0;
}

template <typename T, int FORM, int DP, int TILES>
__global__ __launch_bounds__(64 * kWeighWaves, 2) void weigh_many_kernel(AttnArgs a) {
    using F = Block<T, FORM, DP, TILES>;
    __shared__ __attribute__((aligned(16))) unsigned char rows[kWeighWaves][2][F::kHalf];
    __shared__ float logs[kWeighWaves][64];
    __shared__ int highs[kWeighWaves][64], lows[kWeighWaves][64];
    __shared__ const uint16_t* places[kWeighWaves][64];
    __shared__ float sums[kWeighWaves][F::kTokens];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), half = lane >> 5;
    const int D = a.c.head_dim;

    auto scan = [&](int x) {  // inclusive sums over the lanes
        for (int d = 1; d < 64; d <<= 1) {
            const int up = __shfl_up(x, d, 64);
            if (lane >= d) x = __builtin_elementwise_add_sat(x, up);
        }
        return x;
    };
    auto units_of = [&](int s, Seq* q) {
        if (s >= a.sequences) return 0;
        int low, high;
        *q = read_seq(a, s);
        return block_units<F::kTokens>(a, *q, &low, &high);
    };
    int U = 0;
    for (int s0 = 0; s0 < a.sequences; s0 += 64) {
        Seq x = {};
        U = __builtin_elementwise_add_sat(U, __builtin_amdgcn_readlane(scan(units_of(s0 + lane, &x) * a.c.heads), 63));
    }
    if (U == kMostSlots) return;
    // Consecutive units on one XCD (workgroups go to the 8 XCDs in turn): they share query rows in its L2.
    const int xcds = (gridDim.x & 7) == 0 ? 8 : 1, per_xcd = (U + xcds - 1) / xcds;
    const int begin = blockIdx.x % xcds * per_xcd, end = min(begin + per_xcd, U);
    for (int u = begin + blockIdx.x / xcds; u < end; u += gridDim.x / xcds) {
        // the sequence of unit u
        Seq q = {};
        int seq = 0, head = 0, unit = 0, before = 0;
        for (int s0 = 0;; s0 += 64) {
            Seq x = {};
            const int per = units_of(s0 + lane, &x), sum = scan(per * a.c.heads);
            const uint64_t past = __ballot(before + sum > u);
            if (past) {
                const int l = __builtin_ctzll(past);
                const int ph = __builtin_amdgcn_readlane(per, l);
                const int rest = u - (before + __builtin_amdgcn_readlane(sum, l) - ph * a.c.heads);
                seq = s0 + l;
                head = rest / ph;
                unit = rest % ph;
                q.first = __builtin_amdgcn_readlane(x.first, l);
                q.n = __builtin_amdgcn_readlane(x.n, l);
                q.len = __builtin_amdgcn_readlane(x.len, l);
                q.rows = __builtin_amdgcn_readlane(x.rows, l);
                break;
            }
            before += __builtin_amdgcn_readlane(sum, 63);
        }
        int low, high;
        block_units<F::kTokens>(a, q, &low, &high);
        const int t0 = (low / F::kTokens + unit) * F::kTokens;
        F f;
        f.load(a, seq, head, t0, low, high, lane);

        // the rows that may see some of it: tiles [r0, r1) of 64
        const int base = q.len - q.n;
        const int64_t first = a.causal ? (int64_t)max(0, t0 - base) * a.share : 0;
        const int64_t last = a.window ? min((int64_t)q.rows, max((int64_t)0, (int64_t)t0 + F::kTokens - 1 + a.window - base) * a.share) : q.rows;
        const int r0 = (int)(first / 64), r1 = (int)((last + 63) / 64);
        // What lane l says about row l of a tile: where it is, its logarithm, the positions that it sees.
        const uint16_t* place = nullptr;
        float row_log = 0.f;
        int row_high = 0, row_low = 0;
        auto describe = [&](int tile) {
            const int row = tile * 64 + lane, at = min(row, q.rows - 1), tk = share_of(a, at), hs = at - tk * a.share;
            const bool on = row < q.rows;
            place = (const uint16_t*)a.q + (int64_t)(q.first + tk) * a.q_stride + (int64_t)(head * a.share + hs) * D;
            const float x = a.row_lse[(int64_t)(q.first + tk) * a.q_heads + head * a.share + hs];
            row_log = x;  // (not looked at before the rows are: that would wait for it)
            row_high = on ? (a.causal ? min(base + tk + 1, q.len) : q.len) : 0;
            row_low = a.window ? base + tk - a.window + 1 : 0;
            places[wave][lane] = place;
        };
        // Brings the rows of half p that were described: their chunks swizzled by the row, so that the lanes of a read
        // spread over the banks; chunks behind a row's end (its last one again) meet zeros of the keys.
        auto bring = [&](int p) {
            const uint32_t to = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void*)rows[wave][p]);
            const int l = opaque(lane), r = l / F::kChunks;  // (worked out here, not kept in registers through the loop)
            const int at = (l % F::kChunks ^ r) << 4, most = 2 * D - 16;
            constexpr int kRows = 64 / F::kChunks;  // of one load
            constexpr int kBatch = F::kHalf / 1024 < 8 ? F::kHalf / 1024 : 8;  // addresses read at a time
#pragma unroll
            for (int i0 = 0; i0 < F::kHalf / 1024; i0 += kBatch) {
                const uint8_t* from[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) from[i] = (const uint8_t*)places[wave][32 * p + (i0 + i) * kRows + r];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    load_to_lds(from[i] + (uint32_t)min(at ^ (((i0 + i) * kRows & F::kRowMask) << 4), most), to + (i0 + i) * 1024);
            }
        };
        float sum[F::kTiles];
#pragma unroll
        for (int i = 0; i < F::kTiles; ++i) sum[i] = 0.f;
        // 32 rows, half p of a tile; next: what brings the rows that come where they were
        auto half_tile = [&](int p, bool masked, auto next) {
            const int l = opaque(lane);
            auto query = [&](int s) {
                const int r = l & 31;
                return *(const u32x4v*)(rows[wave][p] + r * F::kRow + ((F::chunk(s, l >> 5) ^ (r & F::kRowMask)) << 4));
            };
            // (all of a row in registers where they are enough, so that the next rows may come at once)
            constexpr bool kHeld = DP <= 128;
            u32x4v qr[kHeld ? F::kSteps : 1];
            if (kHeld)
#pragma unroll
                for (int s = 0; s < F::kSteps; ++s) qr[s] = query(s);
            f32x4v log[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) log[j] = *(const f32x4v*)&logs[wave][32 * p + 8 * j + 4 * half];
            auto ahead = [&]() {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                __builtin_amdgcn_sched_barrier(0);
                next();
            };
            if (kHeld) ahead();
            auto product = [&](int i, int st, f32x16v& s) {
                if (st == 0)
#pragma unroll
                    for (int j = 0; j < 16; ++j) s[j] = 0.f;
                s = T::mfma32(kHeld ? qr[kHeld ? st : 0] : query(st), f.key[i][st], s);
            };
            auto weigh = [&](int i, int j, const f32x16v& s) {
                sum[i] += exp2_fast(__builtin_fmaf(s[j], a.scale_log2, -log[j / 4][j % 4]));
            };
            if (!masked) {
                // a tile's products between the exponentials of the tile before it
                f32x16v s[2];
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int st = 0; st < F::kSteps; ++st) product(0, st, s[0]);
#pragma unroll
                for (int i = 0; i < F::kTiles; ++i) {
                    const bool then = i + 1 < F::kTiles;
                    if (then)
#pragma unroll
                        for (int st = 0; st < F::kSteps; ++st) product(i + 1, st, s[(i + 1) & 1]);
#pragma unroll
                    for (int j = 0; j < 16; ++j) weigh(i, j, s[i & 1]);
                    if (then) {
#pragma unroll
                        for (int st = 0; st < F::kSteps; ++st) {
                            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                            __builtin_amdgcn_sched_group_barrier(0x402, 48 / F::kSteps, 0);
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
#pragma unroll
                for (int i = 0; i < F::kTiles; ++i) {
                    f32x16v s;
#pragma unroll
                    for (int st = 0; st < F::kSteps; ++st) product(i, st, s);
                    const int t = t0 + 32 * i + (lane & 31);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int r = 32 * p + 8 * (j / 4) + 4 * half + j % 4;
                        const int to = highs[wave][r], from = lows[wave][r];
                        const float x = exp2_fast(__builtin_fmaf(s[j], a.scale_log2, -log[j / 4][j % 4]));
                        sum[i] += t < to && t >= from ? x : 0.f;
                    }
                }
            }
            if (!kHeld) ahead();
        };
        if (r0 + wave < r1) {
            describe(r0 + wave);
            bring(0);
            bring(1);
        }
        for (int tile = r0 + wave; tile < r1; tile += kWeighWaves) {
            // (here the first half's rows have come, too)
            if (row_log == -__builtin_inff()) row_high = 0;  // (it sees nothing: 2^(score - infinity) may be NaN)
            logs[wave][lane] = tile * 64 + lane < q.rows ? row_log * kLog2e : __builtin_inff();
            highs[wave][lane] = row_high;
            lows[wave][lane] = row_low;
            // some row does not see some position (or is none)
            const uint64_t masked = __ballot(row_high < t0 + F::kTokens || row_low > t0);
            const bool more = tile + kWeighWaves < r1;
            constexpr int kLoads = F::kHalf / 1024;
            asm volatile("s_waitcnt vmcnt(%0)" ::"i"(kLoads) : "memory");  // all but the second half's
            half_tile(0, (uint32_t)masked != 0, [&]() {
                if (!more) return;
                describe(tile + kWeighWaves);
                bring(0);
            });
            if (more)
                asm volatile("s_waitcnt vmcnt(%0)" ::"i"(kLoads) : "memory");  // all but the next first half's
            else
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            half_tile(1, masked >> 32 != 0, [&]() {
                if (more) bring(1);
            });
        }
#pragma unroll
        for (int i = 0; i < F::kTiles; ++i) {
            const float x = sum_halves(sum[i]);
            if (lane < 32) sums[wave][32 * i + lane] = x;
        }
        __syncthreads();
        if (tid < F::kTokens) {
            const int t = t0 + tid;
            float x = sums[0][tid];
#pragma unroll
            for (int w = 1; w < kWeighWaves; ++w) x += sums[w][tid];
            if (t >= low && t < high) {
                const int entry = a.table[seq * a.table_stride + (t >> a.page_log2)];
                if ((uint32_t)entry < (uint32_t)a.c.num_pages) {
                    float* w = a.weight + ((int64_t)entry * a.c.heads + head) * a.c.page_size + (t & (a.c.page_size - 1));
                    *w = (t < base ? *w : 0.f) + x;
                }
            }
        }
        __syncthreads();
    }
}

template <typename T, int FORM, int DP>
hipError_t weigh_run(const AttnArgs& a, int cus, int which, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (which & 1) {
        weigh_few_kernel<T, FORM, (DP == 96 ? 128 : DP)><<<8 * cus, 64 * kWeighWaves, 0, s>>>(a);
        e = hipGetLastError();
    }
    if (e == hipSuccess && (which & 2)) {
        constexpr int kTiles = DP <= 128 ? 4 : 2;
        const double blocks = (double)a.sequences * a.c.heads * ((double)a.table_pages * a.c.page_size / (32 * kTiles) + 1);
        // (blocks of 32 positions where those of 128 would leave CUs idle, as far as the table's width tells: 128 blocks
        // of 1500 tokens x 4 heads 77 against 48 us, 192 74 against 75, 256 73 against 95.  Sequences of few rows count as
        // if they were of many, so that one prompt among many decoding ones takes the large blocks)
        if (blocks < 0.75 * cus)
            weigh_many_kernel<T, FORM, DP, 1><<<2 * cus, 64 * kWeighWaves, 0, s>>>(a);
        else
            weigh_many_kernel<T, FORM, DP, kTiles><<<2 * cus, 64 * kWeighWaves, 0, s>>>(a);
        e = hipGetLastError();
    }
    return e;
}

template <typename T, int FORM>
hipError_t weigh_dim(const AttnArgs& a, int cus, int which, hipStream_t s) {
    const int D = a.c.head_dim;
    if (D <= 64) return weigh_run<T, FORM, 64>(a, cus, which, s);
    // (4-bit rows are read 64 channels at a time)
    if (D <= 96 && FORM != kForm4) return weigh_run<T, FORM, (FORM == kForm4 ? 128 : 96)>(a, cus, which, s);
    if (D <= 128) return weigh_run<T, FORM, 128>(a, cus, which, s);
    return weigh_run<T, FORM, 256>(a, cus, which, s);
}

template <typename T>
hipError_t weigh_type(const AttnArgs& a, int cus, int which, hipStream_t s) {
    switch (cache_form(a.c.type)) {
        case kForm8: return weigh_dim<T, kForm8>(a, cus, which, s);
        case kForm4: return weigh_dim<T, kForm4>(a, cus, which, s);
        default: return weigh_dim<T, kForm16>(a, cus, which, s);
    }
}

}  // namespace

// which: 1 the kernel for few rows, 2 the one for many, 3 both.
hipError_t launch_weigh(const AttnArgs& a, int type, int cus, int which, hipStream_t s) {
    return type == LSCD_F16 ? weigh_type<F16>(a, cus, which, s) : weigh_type<BF16>(a, cus, which, s);
}

}  // namespace lscd
