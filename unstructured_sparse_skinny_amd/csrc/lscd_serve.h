// Declarations shared by the serving operators (quantised product, paged cache, attention):
// kernel arguments, launchers, the objects behind their handles.  The sparse product's own
// declarations are in lscd_internal.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lscd.h"

namespace lscd {

// ---------------------------------------------------------------- paged cache
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
constexpr int kManyRows = 128;    // the kernel for many rows: 32 per wavefront
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
    uint32_t* count;         // arrivals, one per workgroup; zero between calls
};
// Workgroups of one launch at most, and floats of one partial result.
int attention_few_grid(int cus);
int attention_many_grid(int cus);
int64_t attention_few_floats(int dim);
int64_t attention_many_floats(int dim);
hipError_t launch_attention_few(const AttnArgs& a, int type, int grid, hipStream_t s);
hipError_t launch_attention_many(const AttnArgs& a, int type, int grid, hipStream_t s);

}  // namespace lscd

struct lscd_attention_s {
    int device = 0;
    int cus = 256;
    int32_t q_heads = 0, kv_heads = 0, head_dim = 0;
    float* part = nullptr;
    uint32_t* count = nullptr;
};
