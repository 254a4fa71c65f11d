// Eviction from a paged cache: of every sequence and key head, the last positions and those of the others with
// the largest weights are kept and moved, in their order, to the front of the sequence's pages (or of others).
//
// Which ones: one workgroup per sequence and head finds the k-th largest weight among n by its digits, 11, 11 and
// 10 bits from the top: a histogram in LDS says in which digit's bin the k-th lies, and the next digit is looked
// at among that bin's weights only.  Weights are compared as whole numbers in the order of their values.  With the
// threshold known, every wavefront counts what of its stretch is above it and equal to it, and then writes the
// positions in order: equal ones from the lowest position on until there are k.  Nothing depends on the order of
// the histogram's atomics.
//
// Moving: position i of the front takes the i-th position kept, which is i or more.  Into other pages the rows are
// independent.  In place, a workgroup takes a column of the rows (128 bytes of keys or values, or the scales and
// weights) from the front to the back: it reads some rows into registers before it writes them, and what it writes
// lies before everything that is still to be read.
//
// Measured: one sequence of 16384 positions of 8 heads (16 bits) cut to 4096 in 26 us, 18.5 of them to choose (eight
// workgroups on 256 CUs, whose passes wait for each other: 5 us to read the weights, 3 to 6 for a digit) and 7 to
// move; in place 40 (40 workgroups, a memory latency and a drain a round).  64 sequences of 100 to 4096 positions cut to
// 1024 (e4m3, 247 MB) in 71 us, 12 to choose and 57 to move; in place 52.  131072 positions, whose weights are read
// from memory five times (three digits, a count, the writing), cut to 32768: 270 us, in place 415.  4-bit codes: 23 us
// and 56, in place 30 and 31.

#include "lscd_serve.h"
#include "lscd_serve_device.h"

namespace lscd {
namespace {

constexpr int kBins = 2048;

// Order of the weights: larger values have larger keys, zeros are equal, NaN counts as the largest.
__device__ __forceinline__ uint32_t key_of(float w) {
    if (w != w) return 0xFFFFFFFFu;
    const uint32_t b = __builtin_bit_cast(uint32_t, w + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct Kept {
    int len, all, first;  // the sequence's positions; how many stay; the first of the last ones, which stay anyway
    __device__ __forceinline__ Kept(const EvictArgs& a, int s) {
        len = (int)min(max((int64_t)a.length[s], (int64_t)0), (int64_t)a.table_pages * a.c.page_size);
        all = min(len, a.keep);
        first = len - min(a.recent, all);
    }
};

// The page that a table names (page 0 for an entry outside the pool).
__device__ __forceinline__ int64_t page_at(const EvictArgs& a, const int32_t* table, int64_t stride, int s, int page) {
    const int32_t e = table[s * stride + page];
    return (uint32_t)e < (uint32_t)a.c.num_pages ? e : 0;
}

// PER: weights that a thread holds; longer sequences (of the first positions more than THREADS x PER) are read
// again for every digit.  A wavefront has one stretch of positions, 64 after 64.
template <int THREADS, int PER>
__global__ __launch_bounds__(THREADS) void evict_select_kernel(EvictArgs a) {
    constexpr int kSelectThreads = THREADS, kSelectWaves = THREADS / 64, kMine = kBins / THREADS;  // (bins of a thread)
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t sums[2 * kSelectWaves];
    __shared__ uint32_t found[2];  // a digit, and how many of its bin are wanted
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int s = blockIdx.x / a.c.heads, h = blockIdx.x % a.c.heads;
    const Kept kp(a, s);
    int32_t* out = a.kept + ((int64_t)s * a.c.heads + h) * a.keep;
    for (int i = kp.all + tid; i < a.keep; i += kSelectThreads) out[i] = -1;
    const int n = kp.first, k = kp.all - (kp.len - kp.first);  // k of the first n
    for (int i = tid; i < kp.len - n; i += kSelectThreads) out[k + i] = n + i;
    if (k == n) {
        for (int i = tid; i < n; i += kSelectThreads) out[i] = i;
        return;
    }
    if (k == 0) return;

    const int steps = (n + kSelectThreads - 1) / kSelectThreads;
    const int low = min(wave * steps * 64, n), high = min(low + steps * 64, n);
    auto entry = [&](int i) { return page_at(a, a.table, a.table_stride, s, min(low + i * 64 + lane, n - 1) >> a.page_log2); };
    auto weight = [&](int64_t page, int i) {
        return a.weight[(page * a.c.heads + h) * a.c.page_size + (min(low + i * 64 + lane, n - 1) & (a.c.page_size - 1))];
    };
    const bool held = steps <= PER;
    uint32_t keys[PER];
    // The keys of steps i0 .. i0 + kBatch - 1 into x: all loads in flight together.
    constexpr int kBatch = PER <= 16 ? PER : 12;
    static_assert(PER % kBatch == 0, "whole batches");
    auto load = [&](int i0, uint32_t* x) {
        int64_t page[kBatch];
        float w[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) page[i] = entry(i0 + i);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) w[i] = weight(page[i], i0 + i);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) x[i] = key_of(w[i]);
    };
    if (held) {
#pragma unroll
        for (int i0 = 0; i0 < PER; i0 += kBatch) {
            if (i0 >= steps) break;
            load(i0, keys + i0);
        }
    }
    // f(position, key, whether there is one) for every step of the wavefront's stretch
    auto each = [&](auto f) {
        if (held) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (i < steps) f(low + i * 64 + lane, keys[i], low + i * 64 + lane < high);
        } else {
            for (int i0 = 0; i0 < steps; i0 += kBatch) {
                uint32_t x[kBatch];
                load(i0, x);
#pragma unroll
                for (int i = 0; i < kBatch; ++i) f(low + (i0 + i) * 64 + lane, x[i], low + (i0 + i) * 64 + lane < high);
            }
        }
    };
    // the sum of what the wavefronts before this one have put into x
    auto before = [&](const uint32_t* x) {
        const uint32_t mine = x[lane % kSelectWaves];
        uint32_t sum = 0;
#pragma unroll
        for (int w = 0; w < kSelectWaves - 1; ++w) sum += w < wave ? __builtin_amdgcn_readlane(mine, w) : 0u;
        return sum;
    };

    uint32_t prefix = 0, mask = 0;  // the digits found, and their bits
    uint32_t want = (uint32_t)k;
    for (int digit = 0; digit < 3; ++digit) {
        const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0, bins = digit == 2 ? 1024 : 2048;
        for (int i = tid; i < kBins; i += kSelectThreads) hist[i] = 0;
        __syncthreads();
        each([&](int, uint32_t x, bool on) {
            if (on && (x & mask) == prefix) atomicAdd(&hist[(x >> shift) & (bins - 1)], 1u);
        });
        __syncthreads();
        // a few bins a thread, from the top: how many keys lie above and in them
        const int top = kBins - 1 - kMine * tid;
        uint32_t count[kMine], sum = 0;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            count[i] = hist[top - i];
            sum += count[i];
        }
        const uint32_t mine = sum;
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t up = __shfl_up(sum, d, 64);
            if (lane >= d) sum += up;
        }
        if (lane == 63) sums[wave] = sum;
        __syncthreads();
        uint32_t above = before(sums) + sum - mine;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            if (above < want && want <= above + count[i]) {
                found[0] = top - i;
                found[1] = want - above;
            }
            above += count[i];
        }
        __syncthreads();
        prefix |= found[0] << shift;
        mask |= (uint32_t)(bins - 1) << shift;
        want = found[1];
    }
    // `prefix` is the k-th largest key, `want` how many keys equal to it are kept
    uint32_t more = 0, same = 0;
    each([&](int, uint32_t x, bool on) {
        more += __popcll(__ballot(on && x > prefix));
        same += __popcll(__ballot(on && x == prefix));
    });
    if (lane == 0) {
        sums[wave] = more;
        sums[kSelectWaves + wave] = same;
    }
    __syncthreads();
    more = before(sums);
    same = before(sums + kSelectWaves);
    const uint64_t below = ((uint64_t)1 << lane) - 1;
    each([&](int j, uint32_t x, bool on) {
        const uint64_t gt = __ballot(on && x > prefix), eq = __ballot(on && x == prefix);
        const uint32_t g = more + __popcll(gt & below), e = same + __popcll(eq & below);
        if (on && (x > prefix || (x == prefix && e < want))) out[g + min(e, want)] = j;
        more += __popcll(gt);
        same += __popcll(eq);
    });
}

// A row of the cache: its number among all rows of all heads, or -1.
__device__ __forceinline__ int64_t row_at(const EvictArgs& a, const int32_t* table, int64_t stride, int s, int h, int i) {
    const int32_t e = table[s * stride + (i >> a.page_log2)];
    if ((uint32_t)e >= (uint32_t)a.c.num_pages) return -1;
    return ((int64_t)e * a.c.heads + h) * a.c.page_size + (i & (a.c.page_size - 1));
}

// A position read back from `kept`, which is the caller's memory: clamped, whatever it holds by now.
__device__ __forceinline__ int within(int from, int len) { return (int)min((uint32_t)from, (uint32_t)len - 1u); }

// A scale row (1, 2, 4 or 8 bytes; 0: there are none) from one row to another.
__device__ __forceinline__ void move_scale(void* p, int bytes, int64_t from, int64_t to) {
    if (bytes == 8)
        ((uint64_t*)p)[to] = ((const uint64_t*)p)[from];
    else if (bytes == 4)
        ((uint32_t*)p)[to] = ((const uint32_t*)p)[from];
    else if (bytes == 2)
        ((uint16_t*)p)[to] = ((const uint16_t*)p)[from];
}

// Into other pages: a workgroup takes kMoveRows kept rows of the keys or the values of one sequence and head.
constexpr int kMoveRows = 64, kMoveThreads = 256;
template <typename U>
__global__ __launch_bounds__(kMoveThreads) void evict_copy_kernel(EvictArgs a, int chunks) {
    __shared__ int64_t src[kMoveRows], dst[kMoveRows];
    const int tid = threadIdx.x, z = blockIdx.x & 1;
    const int chunk = (blockIdx.x >> 1) % chunks, sh = (blockIdx.x >> 1) / chunks;
    const int s = sh / a.c.heads, h = sh % a.c.heads, i0 = chunk * kMoveRows;
    const Kept kp(a, s);
    const int rows = min(kp.all - i0, kMoveRows);
    if (rows <= 0) return;
    if (tid < rows) {
        const int from = within(a.kept[((int64_t)s * a.c.heads + h) * a.keep + i0 + tid], kp.len);
        const int64_t p = page_at(a, a.table, a.table_stride, s, from >> a.page_log2);
        src[tid] = (p * a.c.heads + h) * a.c.page_size + (from & (a.c.page_size - 1));
        dst[tid] = row_at(a, a.to, a.to_stride, s, h, i0 + tid);
        if (dst[tid] >= 0) {
            if (z == 0) a.weight[dst[tid]] = a.weight[src[tid]];
            move_scale(z ? a.c.v_scale : a.c.k_scale, a.scale_bytes, src[tid], dst[tid]);
        }
    }
    __syncthreads();
    const int units = a.row_bytes / (int)sizeof(U), per = kMoveThreads / units;  // rows of a pass
    const int r0 = tid / units, u = tid % units;
    if (r0 >= per) return;
    U* data = (U*)(z ? a.c.v : a.c.k);
    constexpr int kAtOnce = 4;
    for (int r = r0; r < rows; r += kAtOnce * per) {  // (rows behind the last are read again and not written)
        U x[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) x[j] = data[src[min(r + j * per, rows - 1)] * units + u];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int64_t to = r + j * per < rows ? dst[r + j * per] : -1;
            if (to >= 0) data[to * units + u] = x[j];
        }
    }
}

// In place: see above.  blockIdx.x: sequence and head, and a column: kColumn bytes of the keys, of the values, or
// (the last) scales and weights.
constexpr int kInPlaceThreads = 1024, kColumn = 128, kAhead = 4;
template <typename U>
__global__ __launch_bounds__(kInPlaceThreads) void evict_in_place_kernel(EvictArgs a, int columns) {
    constexpr int kRows = kInPlaceThreads * kAhead;  // of one round at most
    __shared__ int64_t src[kRows], dst[kRows];
    const int tid = threadIdx.x;
    const int column = blockIdx.x % (2 * columns + 1), sh = blockIdx.x / (2 * columns + 1);
    const int s = sh / a.c.heads, h = sh % a.c.heads;
    const Kept kp(a, s);
    if (kp.len <= a.keep) return;
    const int32_t* kept = a.kept + ((int64_t)s * a.c.heads + h) * a.keep;
    auto source = [&](int i) {
        const int from = within(kept[i], kp.len);
        return (page_at(a, a.table, a.table_stride, s, from >> a.page_log2) * a.c.heads + h) * a.c.page_size +
               (from & (a.c.page_size - 1));
    };
    // Reads of a round are complete before its writes begin; nothing of a later round's reads is written before.
    auto all_read = [&]() {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    };
    if (column == 2 * columns) {
        for (int i0 = 0; i0 < kp.all; i0 += kInPlaceThreads) {
            const int i = i0 + tid;
            const int64_t to = i < kp.all ? row_at(a, a.table, a.table_stride, s, h, i) : -1;
            const int64_t from = to >= 0 ? source(i) : 0;
            float w = 0.f;
            uint64_t x[2] = {0, 0};
            if (to >= 0) {
                w = a.weight[from];
                for (int z = 0; z < 2; ++z) {
                    const void* p = z ? a.c.v_scale : a.c.k_scale;
                    if (a.scale_bytes == 8) x[z] = ((const uint64_t*)p)[from];
                    if (a.scale_bytes == 4) x[z] = ((const uint32_t*)p)[from];
                    if (a.scale_bytes == 2) x[z] = ((const uint16_t*)p)[from];
                }
            }
            all_read();
            if (to >= 0) {
                a.weight[to] = w;
                for (int z = 0; z < 2; ++z) {
                    void* p = z ? a.c.v_scale : a.c.k_scale;
                    if (a.scale_bytes == 8) ((uint64_t*)p)[to] = x[z];
                    if (a.scale_bytes == 4) ((uint32_t*)p)[to] = (uint32_t)x[z];
                    if (a.scale_bytes == 2) ((uint16_t*)p)[to] = (uint16_t)x[z];
                }
            }
        }
        return;
    }
    const int units = a.row_bytes / (int)sizeof(U), wide = kColumn / (int)sizeof(U);
    const int u0 = column % columns * wide, mine = min(wide, units - u0);  // units of this column
    const int r = tid / mine, u = u0 + tid % mine, per = kInPlaceThreads / mine;
    U* data = (U*)(column >= columns ? a.c.v : a.c.k);
    for (int i0 = 0; i0 < kp.all; i0 += kAhead * per) {
        // where the round's rows are and go, worked out together; rows behind the last repeat it and go nowhere
        for (int i = tid; i < kAhead * per; i += kInPlaceThreads) {
            src[i] = source(min(i0 + i, kp.all - 1));
            dst[i] = i0 + i < kp.all ? row_at(a, a.table, a.table_stride, s, h, i0 + i) : -1;
        }
        __syncthreads();
        U x[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) x[j] = data[src[j * per + min(r, per - 1)] * units + u];
        all_read();
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int64_t to = r < per ? dst[j * per + r] : -1;
            if (to >= 0) data[to * units + u] = x[j];
        }
        __syncthreads();  // (src and dst are read)
    }
}

int move_chunks(const EvictArgs& a) { return (a.keep + kMoveRows - 1) / kMoveRows; }
int move_columns(const EvictArgs& a) { return (a.row_bytes + kColumn - 1) / kColumn; }

template <typename U>
hipError_t move(const EvictArgs& a, hipStream_t s) {
    const unsigned groups = (unsigned)evict_workgroups(a);
    if (a.to)
        evict_copy_kernel<U><<<groups, kMoveThreads, 0, s>>>(a, move_chunks(a));
    else
        evict_in_place_kernel<U><<<groups, kInPlaceThreads, 0, s>>>(a, move_columns(a));
    return hipGetLastError();
}

}  // namespace

int64_t evict_workgroups(const EvictArgs& a) {
    return (int64_t)a.sequences * a.c.heads * (a.to ? 2 * (int64_t)move_chunks(a) : 2 * move_columns(a) + 1);
}

hipError_t launch_evict(const EvictArgs& a, hipStream_t s) {
    const unsigned pairs = (unsigned)((int64_t)a.sequences * a.c.heads);
    // (what the registers of 16 wavefronts hold; few where that is enough, as far as the tables' width tells)
    const int64_t span = (int64_t)a.table_pages * a.c.page_size;
    if (span <= 256 * 16)
        evict_select_kernel<256, 16><<<pairs, 256, 0, s>>>(a);
    else if (span <= 1024 * 16)
        evict_select_kernel<1024, 16><<<pairs, 1024, 0, s>>>(a);
    else
        evict_select_kernel<1024, 36><<<pairs, 1024, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return a.row_bytes % 16 ? move<u32x2v>(a, s) : move<u32x4v>(a, s);
}

}  // namespace lscd
