// Declarations shared by the serving operators (quantised product, paged cache, attention):
// kernel arguments, launchers, the objects behind their handles.  The sparse product's own
// declarations are in lscd_internal.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lscd.h"

namespace lscd {

// ---------------------------------------------------------------- paged cache
// How a cache holds its values: 16 bits, e4m3 with a float scale a token and head, e2m1 with a byte (exponent
// + 127) for every 32 channels.
enum CacheForm { kForm16 = 0, kForm8 = 1, kForm4 = 2 };
inline int cache_form(int type) { return type == LSCD_E4M3 ? kForm8 : type == LSCD_E2M1 ? kForm4 : kForm16; }
constexpr int form_bits(int form) { return form == kForm4 ? 4 : form == kForm8 ? 8 : 16; }
constexpr int kScaleGroup = 32;
// Bytes of one token's and head's scales of an e2m1 cache: one for 32 channels, so that a row is one aligned word.
constexpr int scale_row(int dim) { return dim <= 64 ? 2 : dim <= 128 ? 4 : 8; }
// Copies of T tokens between rows of `type` ([T][heads][dim], strides in elements) and slots.
struct CacheMoveArgs {
    lscd_cache_t c;
    const void* in[2];    // write: new keys, values
    void* out[2];         // read: where they go
    int64_t stride[2];    // elements from one token to the next
    const int32_t* slots;
    int64_t T;
};
hipError_t launch_cache_write(const CacheMoveArgs& a, int type, hipStream_t s);
hipError_t launch_cache_read(const CacheMoveArgs& a, int type, hipStream_t s);

// ---------------------------------------------------------------- attention
constexpr int kAttnMaxDim = 256;
constexpr int kFewRows = 16;      // query rows of the kernel for few rows: one MFMA tile
constexpr int kFewTokens = 128;   // cached tokens of one of its work units (32 per wavefront)
constexpr int kManyRows = 256;    // the kernel for many rows: 32 per wavefront
constexpr int kManyTokens = 64;

struct AttnArgs {
    lscd_cache_t c;
    const void* q;
    void* o;
    int64_t q_stride, o_stride, table_stride;
    const int32_t* start;    // sequences + 1
    const int32_t* length;   // sequences
    const int32_t* table;    // [sequences][table_stride]
    int32_t table_pages, sequences, q_heads, share, causal, window;
    int64_t T;
    float scale_log2;        // scale * log2(e)
    int32_t few_limit;       // sequences of at most this many query rows belong to the few-row kernel
    int32_t page_log2;
    float* part;             // partial results: two slots per workgroup
    uint32_t* count;         // arrivals, one per workgroup; zero between calls (few rows)
    int4* record;            // cut items, one per workgroup: parts - 1, sequence, key head, row tile (many rows)
    float* lse;              // [T][q_heads], or null
    const float* row_lse;    // the same as an input (weigh)
    uint32_t share_magic, share_shift;  // x / share = x * magic >> shift for x below 2^31 (weigh)
    float* weight;           // [num_pages][heads][page_size] (weigh)
};
// Workgroups of one launch at most, and floats of one partial result.
int attention_few_grid(int cus, int type, int dim);  // by the cache's type
int attention_many_grid(int cus);
int attention_many_tokens(int dim);  // positions of one of the many-row kernel's work units
int64_t attention_few_floats(int dim);
int64_t attention_many_floats(int dim);
hipError_t launch_attention_few(const AttnArgs& a, int type, int grid, hipStream_t s);
hipError_t launch_weigh(const AttnArgs& a, int type, int cus, int which, hipStream_t s);
constexpr int kWeighTokens = 32;  // positions of one of its work units
// Sequences of more query rows go to its kernel for many.  (The other one over 16-bit caches, 32 sequences over 3000
// positions: 128 rows 122 us against 170, 192 167 against 178, 256 213 against 188; 4 sequences: 128 rows 26 against
// 29, 256 47 against 31.)
constexpr int kWeighRows = 128;
hipError_t launch_attention_many(const AttnArgs& a, int type, int grid, hipStream_t s);

// ---------------------------------------------------------------- eviction
struct EvictArgs {
    lscd_cache_t c;
    float* weight;                // [num_pages][heads][page_size]
    const int32_t* length;
    const int32_t* table;
    const int32_t* to;            // other pages, or null: the same
    int64_t table_stride, to_stride;
    int32_t* kept;                // [sequences][heads][keep]
    int32_t table_pages, sequences, keep, recent;
    int32_t page_log2;
    int32_t row_bytes, scale_bytes;  // of one position and head of keys or values, and of its scales
};
// Workgroups of its largest launch.
int64_t evict_workgroups(const EvictArgs& a);
hipError_t launch_evict(const EvictArgs& a, hipStream_t s);

// ---------------------------------------------------------------- quantised product
// Device layout of the codes: row tiles of 16 rows, units of 128 columns, [row tile][unit][64 lanes]
// [4 words].  Lane l of a unit has row l % 16; word s its 8 codes of columns 32 s + 8 (l / 16) + 0..7,
// placed so that pairs come out of a word with one shift and one mask (quant_bit).  Scales and zero
// points: [row tile][unit][16 rows] records, one entry per group of the unit: with groups of 128
// columns and no zero points a 16-bit scale, else a word scale | zero << 16.  Rows past M and columns
// past K hold zero points (weights of zero).
constexpr int kQuantUnit = 128;
constexpr int kQuantRows = 16;
constexpr int kQuantMaxTokens = 64;  // tokens of one launch
// A dimension of a grid has fewer than 2^32 threads (more are cut off without an error): 512 per row tile in
// the products, one per result where K was split.
constexpr int64_t kQuantMostRows = (int64_t)1 << 25;
constexpr int kQuantWaves = 8;

// Position of bit `bit` (0..3) of code j (0..7) in its word: pair p = j / 2 of codes (low and high
// half) sits at bits 6-9 of each half for p = 0, 4 above for p = 1, 4 below for p = 2, and 8 above,
// wrapping around the word, for p = 3.
__host__ __device__ inline int quant_bit(int j, int bit) {
    const int p = j / 2, at = 6 + 16 * (j & 1) + bit + (p == 1 ? 4 : p == 2 ? -4 : p == 3 ? 8 : 0);
    return at & 31;
}

// How one product runs: the kernel (0: up to 16 tokens, 1: more), row tiles per wavefront, and the
// ranges of K that workgroups split it into.
struct QuantPlan {
    int shared, rt, splits;
};
QuantPlan plan_quant(int tiles, int units, int N, int kind, int cus);
// Units that a wavefront has in flight for up to 16 tokens: what the registers hold (records of four words
// take as many of them as the codes: one unit fewer for 2 and 3 row tiles, and no more than 4 row tiles).
constexpr int quant_ahead(int rt, int kind) { return rt == 1 ? 4 : (rt == 2 ? (kind == 4 ? 3 : 4) : (rt == 3 && kind < 4 ? 3 : 2)); }

struct QuantArgs {
    const uint32_t* codes;
    const void* aux;         // scales and zero points
    const uint16_t* x;
    uint16_t* y;
    float* part;
    int64_t ldx, ldy;
    int32_t M, K, N;
    int32_t tiles, units, splits;
    int32_t spare;           // the row that lanes without a token read
};
struct QuantEncodeArgs {
    const uint8_t* q;        // [M][row_bytes]
    const uint16_t* scales;  // [M][groups]
    const uint8_t* zeros;    // [M][groups] or null
    uint32_t* codes;
    void* aux;
    int64_t M, K, row_bytes, groups;
    int32_t group, per_unit; // columns of a group, groups of a unit (1, 2 or 4)
    int32_t short_aux;       // 16-bit records
    int32_t tiles, units;
};
// Kinds of records: one 16-bit scale, one word, two words, four words a unit and row.
inline int quant_kind(int per_unit, bool zeros) { return per_unit == 1 ? (zeros ? 1 : 0) : per_unit; }
inline int quant_aux_bytes(int kind) { return kind == 0 ? 2 : 4 * kind; }
hipError_t launch_quant_encode(const QuantEncodeArgs& a, hipStream_t s);
hipError_t launch_quant_decode(const QuantArgs& a, int type, int kind, uint16_t* w, hipStream_t s);
// (one source file per type)
hipError_t launch_quant_f16(const QuantArgs& a, int kind, const QuantPlan& p, hipStream_t s);
hipError_t launch_quant_bf16(const QuantArgs& a, int kind, const QuantPlan& p, hipStream_t s);

}  // namespace lscd

struct lscd_quant_s {
    int device = 0;
    int cus = 256;
    int64_t M = 0, K = 0;
    int32_t group = 0, type = 0, per_unit = 1;
    int32_t tiles = 0, units = 0;
    uint32_t* codes = nullptr;
    void* aux = nullptr;
    int kind = 0;
    float* part = nullptr;
    int64_t part_floats = 0;
};

struct lscd_attention_s {
    int device = 0;
    int cus = 256;
    int32_t q_heads = 0, kv_heads = 0, head_dim = 0;
    float* part = nullptr;
    uint32_t* count = nullptr;
    int4* record = nullptr;
};
