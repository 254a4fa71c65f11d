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
// Both kernels sum the weights as they multiply them.
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
    const float *ks, *vs;
    uint64_t page, page_scales;
    int block, block_scales;  // bytes of one page's block
    __device__ __forceinline__ HeadBase(const AttnArgs& a, int head, int width) {
        block = a.c.page_size * a.c.head_dim * width;
        block_scales = a.c.page_size * 4;
        page = (uint64_t)a.c.heads * block;
        page_scales = (uint64_t)a.c.heads * block_scales;
        k = (const uint8_t*)a.c.k + (uint64_t)head * block;
        v = (const uint8_t*)a.c.v + (uint64_t)head * block;
        ks = a.c.k_scale + (uint64_t)head * a.c.page_size;
        vs = a.c.v_scale + (uint64_t)head * a.c.page_size;
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t keys(uint32_t p) const { return buffer_of(k + p * page, block); }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t values(uint32_t p) const { return buffer_of(v + p * page, block); }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t key_scales(uint32_t p) const {
        return buffer_of((const uint8_t*)ks + p * page_scales, block_scales);
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t value_scales(uint32_t p) const {
        return buffer_of((const uint8_t*)vs + p * page_scales, block_scales);
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
