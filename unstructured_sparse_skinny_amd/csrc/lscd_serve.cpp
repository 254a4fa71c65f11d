// C-ABI layer of the serving operators: argument checks, handles and launches.  Entry points are
// declared and documented in include/lscd.h.

#include <math.h>

#include <algorithm>
#include <new>

#include "lscd_serve.h"

namespace {

lscd_status_t status_of(hipError_t e) {
    if (e == hipSuccess) return LSCD_SUCCESS;
    return e == hipErrorOutOfMemory ? LSCD_ERROR_OUT_OF_MEMORY : LSCD_ERROR_HIP;
}
bool aligned(const void* p, uintptr_t n) { return p && ((uintptr_t)p & (n - 1)) == 0; }

bool scaled_form(int32_t type) { return type == LSCD_E4M3 || type == LSCD_E2M1; }

lscd_status_t check_cache(const lscd_cache_t* c) {
    if (!c || !aligned(c->k, 16) || !aligned(c->v, 16) || c->num_pages < 1 || c->heads < 1 || c->page_size < 1 ||
        c->head_dim < 1)
        return LSCD_ERROR_INVALID_VALUE;
    if (c->type != LSCD_F16 && c->type != LSCD_BF16 && !scaled_form(c->type)) return LSCD_ERROR_INVALID_VALUE;
    const bool scaled = scaled_form(c->type);
    if (scaled ? !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16) : c->k_scale || c->v_scale)
        return LSCD_ERROR_INVALID_VALUE;
    if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) || c->head_dim % 16 ||
        c->head_dim > lscd::kAttnMaxDim || c->heads > 65535 || c->num_pages > 0x7FFFFFFF / c->page_size)
        return LSCD_ERROR_NOT_SUPPORTED;
    return LSCD_SUCCESS;
}

// Rows of `width` values, `stride` apart.
bool bad_rows(const void* p, int64_t stride, int64_t width) {
    return !aligned(p, 16) || stride < width || stride % 8 || stride > ((int64_t)1 << 40);
}

lscd_status_t check_move(const lscd_cache_t* c, const void* k, int64_t ks, const void* v, int64_t vs, const int32_t* slots,
                         int64_t T, int32_t type) {
    lscd_status_t st = check_cache(c);
    if (st != LSCD_SUCCESS) return st;
    if (T < 0 || (type != LSCD_F16 && type != LSCD_BF16)) return LSCD_ERROR_INVALID_VALUE;
    if (!scaled_form(c->type) && c->type != type) return LSCD_ERROR_NOT_SUPPORTED;
    if (T == 0) return LSCD_SUCCESS;
    const int64_t width = (int64_t)c->heads * c->head_dim;
    if (bad_rows(k, ks, width) || bad_rows(v, vs, width) || !aligned(slots, 4)) return LSCD_ERROR_INVALID_VALUE;
    if (T > ((int64_t)1 << 30)) return LSCD_ERROR_NOT_SUPPORTED;
    return LSCD_SUCCESS;
}

void free_attention(lscd_attention_s* h) {
    if (!h) return;
    if (h->part) (void)hipFree(h->part);
    if (h->count) (void)hipFree(h->count);
    if (h->record) (void)hipFree(h->record);
    delete h;
}

void free_quant(lscd_quant_s* h) {
    if (!h) return;
    if (h->codes) (void)hipFree(h->codes);
    if (h->aux) (void)hipFree(h->aux);
    if (h->part) (void)hipFree(h->part);
    delete h;
}

lscd_status_t attend(lscd_attention_t h, const lscd_cache_t* cache, const void* q, int64_t q_stride, const int32_t* start,
                     const int32_t* length, const int32_t* table, int64_t table_stride, int32_t table_pages,
                     int32_t sequences, int64_t T, float scale, int32_t causal, int32_t window, void* o, int64_t o_stride,
                     float* lse, int32_t type, void* stream);

// The arguments of query rows over cached positions, checked and put into *a.  (Where there is nothing to do, the
// pointers are not looked at.)
lscd_status_t check_rows(const lscd_cache_t* cache, const void* q, int64_t q_stride, int32_t q_heads, const int32_t* start,
                         const int32_t* length, const int32_t* table, int64_t table_stride, int32_t table_pages,
                         int32_t sequences, int64_t T, float scale, int32_t causal, int32_t window, int32_t type,
                         lscd::AttnArgs* a) {
    lscd_status_t st = check_cache(cache);
    if (st != LSCD_SUCCESS) return st;
    if ((type != LSCD_F16 && type != LSCD_BF16) || T < 0 || sequences < 0 || table_pages < 0 || window < 0 ||
        !isfinite(scale) || q_heads < 1 || q_heads % cache->heads)
        return LSCD_ERROR_INVALID_VALUE;
    if (!scaled_form(cache->type) && cache->type != type) return LSCD_ERROR_NOT_SUPPORTED;
    if (T == 0 || sequences == 0) return LSCD_SUCCESS;
    if (bad_rows(q, q_stride, (int64_t)q_heads * cache->head_dim) || !aligned(start, 4) || !aligned(length, 4) ||
        !aligned(table, 4) || table_pages < 1 || table_stride < table_pages)
        return LSCD_ERROR_INVALID_VALUE;
    const int64_t share = q_heads / cache->heads, span = (int64_t)table_pages * cache->page_size;
    if (T > ((int64_t)1 << 30) / share || span > ((int64_t)1 << 30)) return LSCD_ERROR_NOT_SUPPORTED;
    a->c = *cache;
    a->q = q;
    a->q_stride = q_stride;
    a->table_stride = table_stride;
    a->start = start;
    a->length = length;
    a->table = table;
    a->table_pages = table_pages;
    a->sequences = sequences;
    a->q_heads = q_heads;
    a->share = (int32_t)share;
    a->causal = causal != 0;
    a->window = (int32_t)std::min<int64_t>(window, (int64_t)1 << 30);
    a->T = T;
    a->scale_log2 = scale * 1.4426950408889634f;
    a->page_log2 = __builtin_ctz((unsigned)cache->page_size);
    return LSCD_SUCCESS;
}

lscd_status_t check_quant(const lscd_quant_s* h) {
    int device = 0;
    if (hipGetDevice(&device) != hipSuccess) return LSCD_ERROR_HIP;
    return device == h->device ? LSCD_SUCCESS : LSCD_ERROR_INVALID_VALUE;
}

lscd::QuantArgs quant_args(const lscd_quant_s* h) {
    lscd::QuantArgs a = {};
    a.codes = h->codes;
    a.aux = h->aux;
    a.part = h->part;
    a.M = (int32_t)h->M;
    a.K = (int32_t)h->K;
    a.tiles = h->tiles;
    a.units = h->units;
    return a;
}

}  // namespace

extern "C" {

lscd_status_t lscd_quant_encode(const void* codes, int64_t row_bytes, const void* scales, const void* zeros, int64_t M,
                                int64_t K, int32_t group, int32_t type, void* stream, lscd_quant_t* out) {
    if (!out) return LSCD_ERROR_INVALID_VALUE;
    *out = nullptr;
    if (!codes || !aligned(scales, 2) || M < 1 || K < 1 || group < 1 || row_bytes < (K + 1) / 2 ||
        (type != LSCD_F16 && type != LSCD_BF16))
        return LSCD_ERROR_INVALID_VALUE;
    if (M > lscd::kQuantMostRows || K > ((int64_t)1 << 24)) return LSCD_ERROR_NOT_SUPPORTED;
    if (group < 32 || (group < 128 ? group != 32 && group != 64 : group % 128)) return LSCD_ERROR_NOT_SUPPORTED;
    const int32_t tiles = (int32_t)((M + lscd::kQuantRows - 1) / lscd::kQuantRows);
    const int32_t units = (int32_t)((K + lscd::kQuantUnit - 1) / lscd::kQuantUnit);
    if ((int64_t)tiles * ((units + 3) / 4) >= ((int64_t)1 << 24)) return LSCD_ERROR_NOT_SUPPORTED;  // (encoded by 256 threads each)
    lscd_quant_s* h = new (std::nothrow) lscd_quant_s();
    if (!h) return LSCD_ERROR_OUT_OF_MEMORY;
    int cus = 0;
    hipError_t e = hipGetDevice(&h->device);
    if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, h->device);
    if (e != hipSuccess || cus <= 0) {
        free_quant(h);
        return LSCD_ERROR_HIP;
    }
    h->cus = cus;
    h->M = M;
    h->K = K;
    h->group = group;
    h->type = type;
    h->per_unit = group >= 128 ? 1 : 128 / group;
    h->tiles = tiles;
    h->units = units;
    h->kind = lscd::quant_kind(h->per_unit, zeros != nullptr);
    // (every number of tokens has its own plan: fewer may split K further and need more room)
    for (int n = 1; n <= lscd::kQuantMaxTokens; ++n) {
        const lscd::QuantPlan p = lscd::plan_quant(h->tiles, h->units, n, h->kind, cus);
        if (p.splits > 1) h->part_floats = std::max(h->part_floats, (int64_t)p.splits * M * n);
    }
    lscd::QuantEncodeArgs a = {};
    const int64_t total = (int64_t)tiles * units;
    if ((e = hipMalloc((void**)&h->codes, (size_t)total * 1024)) == hipSuccess &&
        (e = hipMalloc((void**)&h->aux, (size_t)total * 16 * lscd::quant_aux_bytes(h->kind))) == hipSuccess &&
        (!h->part_floats || (e = hipMalloc((void**)&h->part, (size_t)h->part_floats * 4)) == hipSuccess)) {
        a.q = (const uint8_t*)codes;
        a.scales = (const uint16_t*)scales;
        a.zeros = (const uint8_t*)zeros;
        a.codes = h->codes;
        a.aux = h->aux;
        a.short_aux = h->kind == 0;
        a.M = M;
        a.K = K;
        a.row_bytes = row_bytes;
        a.groups = (K + group - 1) / group;
        a.group = group;
        a.per_unit = h->per_unit;
        a.tiles = h->tiles;
        a.units = h->units;
        e = lscd::launch_quant_encode(a, (hipStream_t)stream);
        if (e == hipSuccess) e = hipStreamSynchronize((hipStream_t)stream);
    }
    if (e != hipSuccess) {
        free_quant(h);
        return status_of(e);
    }
    *out = h;
    return LSCD_SUCCESS;
}

lscd_status_t lscd_quant_linear(lscd_quant_t h, const void* x, int64_t ldx, void* y, int64_t ldy, int32_t N,
                                void* stream) {
    if (!h || N < 0) return LSCD_ERROR_INVALID_VALUE;
    if (N == 0) return LSCD_SUCCESS;
    if (!aligned(x, 2) || !aligned(y, 2) || ldx < h->K || ldy < h->M) return LSCD_ERROR_INVALID_VALUE;
    if (N > LSCD_MAX_N) return LSCD_ERROR_NOT_SUPPORTED;
    lscd_status_t st = check_quant(h);
    if (st != LSCD_SUCCESS) return st;
    lscd::QuantArgs a = quant_args(h);
    a.ldx = ldx;
    a.ldy = ldy;
    // (rows of fewer than 8 values: the kernel for up to 16 tokens, which has no 16-byte loads then)
    const int32_t most = h->K < 8 ? 16 : lscd::kQuantMaxTokens;
    for (int32_t n = 0; n < N; n += most) {
        a.x = (const uint16_t*)x + n * ldx;
        a.y = (uint16_t*)y + n * ldy;
        a.N = std::min(N - n, most);
        const lscd::QuantPlan p = lscd::plan_quant(h->tiles, h->units, a.N, h->kind, h->cus);
        a.splits = p.splits;
        hipError_t e = h->type == LSCD_F16 ? lscd::launch_quant_f16(a, h->kind, p, (hipStream_t)stream)
                                           : lscd::launch_quant_bf16(a, h->kind, p, (hipStream_t)stream);
        if (e != hipSuccess) return status_of(e);
    }
    return LSCD_SUCCESS;
}

lscd_status_t lscd_quant_decode(lscd_quant_t h, void* w, void* stream) {
    if (!h || !aligned(w, 2)) return LSCD_ERROR_INVALID_VALUE;
    lscd_status_t st = check_quant(h);
    if (st != LSCD_SUCCESS) return st;
    return status_of(lscd::launch_quant_decode(quant_args(h), h->type, h->kind, (uint16_t*)w, (hipStream_t)stream));
}

lscd_status_t lscd_quant_destroy(lscd_quant_t h) {
    free_quant(h);
    return LSCD_SUCCESS;
}

lscd_status_t lscd_cache_write(const lscd_cache_t* cache, const void* k, int64_t k_stride, const void* v,
                               int64_t v_stride, const int32_t* slots, int64_t T, int32_t type, void* stream) {
    lscd_status_t st = check_move(cache, k, k_stride, v, v_stride, slots, T, type);
    if (st != LSCD_SUCCESS || T == 0) return st;
    lscd::CacheMoveArgs a = {};
    a.c = *cache;
    a.in[0] = k;
    a.in[1] = v;
    a.stride[0] = k_stride;
    a.stride[1] = v_stride;
    a.slots = slots;
    a.T = T;
    return status_of(lscd::launch_cache_write(a, type, (hipStream_t)stream));
}

lscd_status_t lscd_cache_read(const lscd_cache_t* cache, const int32_t* slots, int64_t T, void* k, int64_t k_stride,
                              void* v, int64_t v_stride, int32_t type, void* stream) {
    lscd_status_t st = check_move(cache, k, k_stride, v, v_stride, slots, T, type);
    if (st != LSCD_SUCCESS || T == 0) return st;
    lscd::CacheMoveArgs a = {};
    a.c = *cache;
    a.out[0] = k;
    a.out[1] = v;
    a.stride[0] = k_stride;
    a.stride[1] = v_stride;
    a.slots = slots;
    a.T = T;
    return status_of(lscd::launch_cache_read(a, type, (hipStream_t)stream));
}

lscd_status_t lscd_attention_create(int32_t q_heads, int32_t kv_heads, int32_t head_dim, lscd_attention_t* out) {
    if (!out) return LSCD_ERROR_INVALID_VALUE;
    *out = nullptr;
    if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads || head_dim < 1) return LSCD_ERROR_INVALID_VALUE;
    if (q_heads > 65535 || head_dim % 16 || head_dim > lscd::kAttnMaxDim) return LSCD_ERROR_NOT_SUPPORTED;
    lscd_attention_s* h = new (std::nothrow) lscd_attention_s();
    if (!h) return LSCD_ERROR_OUT_OF_MEMORY;
    h->q_heads = q_heads;
    h->kv_heads = kv_heads;
    h->head_dim = head_dim;
    int cus = 0;
    hipError_t e = hipGetDevice(&h->device);
    if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, h->device);
    if (e != hipSuccess || cus <= 0) {
        free_attention(h);
        return LSCD_ERROR_HIP;
    }
    h->cus = cus;
    const int few = lscd::attention_few_grid(cus, LSCD_E2M1, head_dim), many = lscd::attention_many_grid(cus);
    const int64_t floats = std::max(2 * few * lscd::attention_few_floats(head_dim),
                                    2 * many * lscd::attention_many_floats(head_dim));
    if ((e = hipMalloc((void**)&h->part, (size_t)floats * 4)) != hipSuccess ||
        (e = hipMalloc((void**)&h->count, (size_t)few * 4)) != hipSuccess ||
        (e = hipMalloc((void**)&h->record, (size_t)many * sizeof(int4))) != hipSuccess ||
        (e = hipMemset(h->count, 0, (size_t)few * 4)) != hipSuccess || (e = hipDeviceSynchronize()) != hipSuccess) {
        free_attention(h);
        return status_of(e);
    }
    *out = h;
    return LSCD_SUCCESS;
}

lscd_status_t lscd_attention_destroy(lscd_attention_t h) {
    free_attention(h);
    return LSCD_SUCCESS;
}

lscd_status_t lscd_attention(lscd_attention_t h, const lscd_cache_t* cache, const void* q, int64_t q_stride,
                             const int32_t* start, const int32_t* length, const int32_t* table, int64_t table_stride,
                             int32_t table_pages, int32_t sequences, int64_t T, float scale, int32_t causal,
                             int32_t window, void* o, int64_t o_stride, int32_t type, void* stream) {
    return attend(h, cache, q, q_stride, start, length, table, table_stride, table_pages, sequences, T, scale, causal, window,
                  o, o_stride, nullptr, type, stream);
}

lscd_status_t lscd_attention_lse(lscd_attention_t h, const lscd_cache_t* cache, const void* q, int64_t q_stride,
                                 const int32_t* start, const int32_t* length, const int32_t* table, int64_t table_stride,
                                 int32_t table_pages, int32_t sequences, int64_t T, float scale, int32_t causal,
                                 int32_t window, void* o, int64_t o_stride, float* lse, int32_t type, void* stream) {
    if (T > 0 && sequences > 0 && !aligned(lse, 4)) return LSCD_ERROR_INVALID_VALUE;
    return attend(h, cache, q, q_stride, start, length, table, table_stride, table_pages, sequences, T, scale, causal, window,
                  o, o_stride, lse, type, stream);
}

lscd_status_t lscd_cache_weigh(const lscd_cache_t* cache, const void* q, int64_t q_stride, int32_t q_heads,
                               const float* lse, const int32_t* start, const int32_t* length, const int32_t* table,
                               int64_t table_stride, int32_t table_pages, int32_t sequences, int64_t T, float scale,
                               int32_t causal, int32_t window, float* weight, int32_t type, void* stream) {
    lscd::AttnArgs a = {};
    lscd_status_t st = check_rows(cache, q, q_stride, q_heads, start, length, table, table_stride, table_pages, sequences, T,
                                  scale, causal, window, type, &a);
    if (st != LSCD_SUCCESS || T == 0 || sequences == 0) return st;
    if (!aligned(lse, 4) || !aligned(weight, 16)) return LSCD_ERROR_INVALID_VALUE;
    if (q_heads > 65535) return LSCD_ERROR_NOT_SUPPORTED;
    // Slots of work are counted in 31 bits on the device.
    const double span = (double)table_pages * cache->page_size;
    if (((double)(T * a.share) / lscd::kFewRows + sequences) * (span / lscd::kWeighTokens + 1) * cache->heads >= 2147483647.0)
        return LSCD_ERROR_NOT_SUPPORTED;
    int device = 0, cus = 0;
    hipError_t e = hipGetDevice(&device);
    if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, device);
    if (e != hipSuccess || cus <= 0) return LSCD_ERROR_HIP;
    a.row_lse = lse;
    uint32_t bits = 0;  // 2^bits >= share: magic = ceil(2^(31 + bits) / share) has 32 bits
    while (((int64_t)1 << bits) < a.share) ++bits;
    a.share_shift = 31 + bits;
    a.share_magic = (uint32_t)((((uint64_t)1 << a.share_shift) + a.share - 1) / a.share);
    a.weight = weight;
    // The same choice as for attention: one launch where no sequence can have many rows, or there is only one.
    const bool both = T * a.share > lscd::kWeighRows && T > sequences;
    a.few_limit = !both ? 0x7FFFFFFF : sequences > 1 ? lscd::kWeighRows : 0;
    return status_of(lscd::launch_weigh(a, type, cus, !both ? 1 : sequences > 1 ? 3 : 2, (hipStream_t)stream));
}

lscd_status_t lscd_cache_evict(const lscd_cache_t* cache, float* weight, const int32_t* length, const int32_t* table,
                               int64_t table_stride, int32_t table_pages, const int32_t* to, int64_t to_stride,
                               int32_t to_pages, int32_t sequences, int32_t keep, int32_t recent, int32_t* kept,
                               void* stream) {
    lscd_status_t st = check_cache(cache);
    if (st != LSCD_SUCCESS) return st;
    if (sequences < 0 || keep < 1 || recent < 0 || recent > keep) return LSCD_ERROR_INVALID_VALUE;
    if (sequences == 0) return LSCD_SUCCESS;
    if (!aligned(weight, 16) || !aligned(length, 4) || !aligned(table, 4) || !aligned(kept, 4) || table_pages < 1 ||
        table_stride < table_pages || ((uintptr_t)to & 3))
        return LSCD_ERROR_INVALID_VALUE;
    const int64_t page = cache->page_size;
    if (to && (to_pages < 1 || to_stride < to_pages || to_pages * page < keep)) return LSCD_ERROR_INVALID_VALUE;
    // (positions, and those that are kept, are counted in 31 bits with what a workgroup takes at a time behind them)
    if (table_pages * page > ((int64_t)1 << 30) || keep > (1 << 30)) return LSCD_ERROR_NOT_SUPPORTED;
    lscd::EvictArgs a = {};
    a.c = *cache;
    a.weight = weight;
    a.length = length;
    a.table = table;
    a.to = to == table ? nullptr : to;
    a.table_stride = table_stride;
    a.to_stride = to_stride;
    a.kept = kept;
    a.table_pages = table_pages;
    a.sequences = sequences;
    a.keep = keep;
    a.recent = recent;
    a.page_log2 = __builtin_ctz((unsigned)page);
    a.row_bytes = cache->head_dim * lscd::form_bits(lscd::cache_form(cache->type)) / 8;
    a.scale_bytes = cache->type == LSCD_E4M3 ? 4 : cache->type == LSCD_E2M1 ? lscd::scale_row(cache->head_dim) : 0;
    // (a dimension of a grid has fewer than 2^32 threads, 1024 of them a workgroup at most)
    if ((int64_t)sequences * cache->heads >= ((int64_t)1 << 22) || lscd::evict_workgroups(a) >= ((int64_t)1 << 22))
        return LSCD_ERROR_NOT_SUPPORTED;
    return status_of(lscd::launch_evict(a, (hipStream_t)stream));
}

}  // extern "C"

namespace {

lscd_status_t attend(lscd_attention_t h, const lscd_cache_t* cache, const void* q, int64_t q_stride, const int32_t* start,
                     const int32_t* length, const int32_t* table, int64_t table_stride, int32_t table_pages,
                     int32_t sequences, int64_t T, float scale, int32_t causal, int32_t window, void* o, int64_t o_stride,
                     float* lse, int32_t type, void* stream) {
    if (!h) return LSCD_ERROR_INVALID_VALUE;
    lscd_status_t st = check_cache(cache);
    if (st != LSCD_SUCCESS) return st;
    if (cache->heads != h->kv_heads || cache->head_dim != h->head_dim) return LSCD_ERROR_INVALID_VALUE;
    lscd::AttnArgs a = {};
    st = check_rows(cache, q, q_stride, h->q_heads, start, length, table, table_stride, table_pages, sequences, T, scale,
                    causal, window, type, &a);
    if (st != LSCD_SUCCESS) return st;
    if (T == 0 || sequences == 0) return LSCD_SUCCESS;
    if (bad_rows(o, o_stride, (int64_t)h->q_heads * h->head_dim)) return LSCD_ERROR_INVALID_VALUE;
    const int64_t share = a.share, span = (int64_t)table_pages * cache->page_size;
    int device = 0;
    if (hipGetDevice(&device) != hipSuccess) return LSCD_ERROR_HIP;
    if (device != h->device) return LSCD_ERROR_INVALID_VALUE;
    a.o = o;
    a.lse = lse;
    a.o_stride = o_stride;
    a.part = h->part;
    a.count = h->count;
    a.record = h->record;
    // Sequences of up to 16 query rows are the few-row kernel's, longer ones the other's.  Where no
    // sequence can be longer (or each has one new token, as far as the counts tell), the few-row
    // kernel takes all of them, whatever the device arrays hold.  A single sequence that may be long is the
    // other's, whatever its rows: one launch.
    const bool both = T * share > lscd::kFewRows && T > sequences;
    a.few_limit = !both ? 0x7FFFFFFF : sequences > 1 ? lscd::kFewRows : 0;
    // Workgroups: no more per item than pay.  An item of U units over W workgroups takes U / W units and
    // then, in its last one, W parts to join: best at W = sqrt(U * unit / part), with a unit's time over a
    // part's about 20 over the query rows where they are few (eight query rows over 32768 positions: 39 us with
    // the workgroups of one row, 26 with theirs) and 4 where they are 256.
    const double rows = std::min<double>(lscd::kFewRows, ceil((double)(T * share) / sequences));
    auto grid = [&](int most, int tile, int tokens, double ratio) {
        const double items = ((double)(T * share) / tile + sequences) * h->kv_heads, units = ceil((double)span / tokens);
        return (int)std::min<double>(most, items * std::min(units, 1.0 + ceil(sqrt(ratio * units))));
    };
    // Slots of work are counted in 31 bits on the device: a row tile has one for each stretch of positions and
    // two more at most.
    const bool few = sequences > 1 || !both;
    auto too_many = [&](int64_t tiles, int tokens) {
        return (double)(tiles + sequences) * (double)(span / tokens + 2) * h->kv_heads >= 2147483647.0;
    };
    if ((few && too_many(both ? 0 : T * share / lscd::kFewRows, lscd::kFewTokens)) ||
        (both && too_many(T * share / lscd::kManyRows, lscd::attention_many_tokens(h->head_dim))))
        return LSCD_ERROR_NOT_SUPPORTED;
    if (few) {
        hipError_t e = lscd::launch_attention_few(
            a, type, grid(lscd::attention_few_grid(h->cus, cache->type, h->head_dim), lscd::kFewRows, lscd::kFewTokens, 20.0 / rows), (hipStream_t)stream);
        if (e != hipSuccess) return status_of(e);
    }
    if (both) {
        hipError_t e = lscd::launch_attention_many(
            a, type, grid(lscd::attention_many_grid(h->cus), lscd::kManyRows, lscd::kManyTokens, 4.0), (hipStream_t)stream);
        if (e != hipSuccess) return status_of(e);
    }
    return LSCD_SUCCESS;
}

}  // namespace
