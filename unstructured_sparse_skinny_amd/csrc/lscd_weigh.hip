// The softmax weights that new tokens give to the cached positions, added up per position and key head:
//   weight[j] (+)= sum over the sequence's query rows r of the key head of exp(scale * q_r . k_j - lse_r),
// over the rows that see position j; lse_r is what the attention found for the row, so that one pass over the
// keys is enough and every position's sum is finished where its keys are: no partial results, no atomics, a
// fixed order of addition.  Positions of the new tokens themselves start from the sum, it is added to the others'.
//
// S = Q K^T on the matrix cores: a lane then holds scores of one position and of four rows, whose sum is taken in
// the lane and over its quarters.  Products are exact and sums fp32, as in the attention.
//
// The units (stretches of kWeighTokens positions of one sequence and key head) are numbered sequence after
// sequence, head after head, and cut into equal ranges by what they cost, one for each wavefront; a unit belongs
// to the range in which its first slot lies.

#include "lscd_attention.h"

namespace lscd {
namespace {

constexpr int kWeighWaves = 4;
static_assert(kWeighTokens == 32, "a unit is two key tiles of 16 positions");

// What the rows of a sequence see together: positions [low, high), in `units` stretches; a unit costs a slot for
// every tile of 16 rows.
struct Stretch {
    int low, high, units, cost;
    __device__ __forceinline__ void measure(const AttnArgs& a, const Seq& q) {
        high = q.rows > 0 ? q.len : 0;  // (the last token sees all with or without causality)
        low = a.window ? min(max(q.len - q.n - a.window + 1, 0), high) : 0;
        units = high > low ? (high + kWeighTokens - 1) / kWeighTokens - low / kWeighTokens : 0;
        cost = (q.rows + kFewRows - 1) / kFewRows;
    }
};

// Where a range begins: the first unit whose first slot is in it.
struct WeighWork {
    int u, end;  // that slot; the range's end
    int seq, head, unit;
    Seq q;
    Stretch st;
};
__device__ __forceinline__ bool find_weigh(const AttnArgs& a, int lane, int me, int G, WeighWork* w) {
    auto slots_of = [&](int s, Seq* q) {
        if (s >= a.sequences) return 0;
        *q = read_seq(a, s);
        Stretch st;
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

// The unit after this one; false past the range's end.
__device__ __forceinline__ bool next_unit(const AttnArgs& a, WeighWork* w) {
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

template <typename T, int FORM, int DP>
__global__ __launch_bounds__(64 * kWeighWaves) void weigh_few_kernel(AttnArgs a) {
    using F = Keys<T, FORM, DP>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    WeighWork w;
    if (!find_weigh(a, lane, blockIdx.x * kWeighWaves + wave, gridDim.x * kWeighWaves, &w)) return;
    const int D = a.c.head_dim, g = lane >> 4;
    while (next_unit(a, &w)) {
        const int t0 = (w.st.low / kWeighTokens + w.unit) * kWeighTokens;
        const int e[2] = {entry_of(a, w.seq, t0), entry_of(a, w.seq, t0 + 16)};
        HeadBase hb;
        hb.set<F::kBits, F::kScaleBytes>(a.c, w.head);
        F f;
        f.load_keys(a, hb, e, t0, w.st.high, lane);
        // the weights of the lane's position (lanes 0 .. 31)
        const int mine = t0 + (lane & 31), page = a.c.page_size;
        const int entry = lane & 16 ? e[1] : e[0];
        const int64_t at = ((int64_t)page_of(a, entry) * a.c.heads + w.head) * page + (mine & (page - 1));
        const bool own = lane < 32 && mine >= w.st.low && mine < w.st.high && (uint32_t)entry < (uint32_t)a.c.num_pages;
        const float old = own && mine < w.q.len - w.q.n ? a.weight[at] : 0.f;
        float sum[2] = {0.f, 0.f};
        for (int tile = 0; tile < w.st.cost; ++tile) {
            const int row = tile * kFewRows + (lane & 15);
            const bool live = row < w.q.rows;
            const int token = row / a.share;
            const uint16_t* qp = (const uint16_t*)a.q + (int64_t)(w.q.first + (live ? token : 0)) * a.q_stride +
                                 (int64_t)(w.head * a.share + row % a.share) * D;
            u32x4v qr[F::kSteps];
#pragma unroll
            for (int s = 0; s < F::kSteps; ++s) {
                const int d = F::step_channel(s, g, D);
                qr[s] = u32x4v{0u, 0u, 0u, 0u};
                if (live && d < D) qr[s] = *(const u32x4v*)(qp + d);
            }
            float lse[4];  // of the rows whose scores the lane has, in units of log2; rows that are none weigh nothing
            int see_high[4], see_low[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int rw = tile * kFewRows + 4 * g + r, tk = rw / a.share, pos = w.q.len - w.q.n + tk;
                const bool on = rw < w.q.rows;
                const float x = on ? a.row_lse[(int64_t)(w.q.first + tk) * a.q_heads + w.head * a.share + rw % a.share] : -__builtin_inff();
                lse[r] = x == -__builtin_inff() ? __builtin_inff() : x * kLog2e;
                see_high[r] = on ? (a.causal ? min(pos + 1, w.q.len) : w.q.len) : 0;
                see_low[r] = a.window ? pos - a.window + 1 : 0;
            }
            const bool top = f.top_keys();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f32x4v s = {0.f, 0.f, 0.f, 0.f};
                if (!top)
#pragma unroll
                    for (int st = 0; st < F::kSteps; ++st) s = T::mfma16(qr[st], f.template key_operand<false>(h, st), s);
                else
#pragma unroll
                    for (int st = 0; st < F::kSteps; ++st) s = T::mfma16(qr[st], f.template key_operand<true>(h, st), s);
                const int t = t0 + 16 * h + (lane & 15);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float p = exp2_fast(__builtin_fmaf(s[r], a.scale_log2, -lse[r]));
                    sum[h] += t < see_high[r] && t >= see_low[r] ? p : 0.f;
                }
            }
        }
        const float x = sum_quarters(sum[0]), y = sum_quarters(sum[1]);
        if (own) a.weight[at] = old + (lane & 16 ? y : x);
        w.u += w.st.cost;
        ++w.unit;
    }
}

template <typename T, int FORM>
hipError_t weigh_dim(const AttnArgs& a, int grid, hipStream_t s) {
    const int D = a.c.head_dim;
    if (D <= 64)
        weigh_few_kernel<T, FORM, 64><<<grid, 64 * kWeighWaves, 0, s>>>(a);
    else if (D <= 128)
        weigh_few_kernel<T, FORM, 128><<<grid, 64 * kWeighWaves, 0, s>>>(a);
    else
        weigh_few_kernel<T, FORM, 256><<<grid, 64 * kWeighWaves, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t weigh_type(const AttnArgs& a, int grid, hipStream_t s) {
    switch (cache_form(a.c.type)) {
        case kForm8: return weigh_dim<T, kForm8>(a, grid, s);
        case kForm4: return weigh_dim<T, kForm4>(a, grid, s);
        default: return weigh_dim<T, kForm16>(a, grid, s);
    }
}

}  // namespace

hipError_t launch_weigh(const AttnArgs& a, int type, int cus, hipStream_t s) {
    return type == LSCD_F16 ? weigh_type<F16>(a, 4 * cus, s) : weigh_type<BF16>(a, 4 * cus, s);
}

}  // namespace lscd
