// Argument checks that the key/value cache's calls share.
#pragma once

#include <cstdint>

#include "kda.h"
#include "pool.h"
#include "../kda_internal.h"

namespace kda {
namespace host {

constexpr int64_t kMaxTokens = 1 << 30;   // of a sequence: the kernels' positions and their differences fit int32

inline int64_t elem_size(int32_t dtype) { return dtype == KDA_BF16 ? 2 : 4; }
inline int64_t align_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool valid_cache(int32_t Hkv, int32_t d, int32_t fmt, int32_t page_tokens) {
    return Hkv > 0 && Hkv <= 4096 && (d == 64 || d == 128) && (fmt == KDA_KV_BF16 || fmt == KDA_KV_I8) &&
           page_tokens >= 16 && page_tokens <= kda::kKvMaxPageTokens && page_tokens % 16 == 0;
}

inline int64_t record_bytes(int32_t d, int32_t fmt, int32_t page_tokens) {
    return 2 * (int64_t)page_tokens * d * (fmt == KDA_KV_I8 ? 1 : 2) + (fmt == KDA_KV_I8 ? 16 : 0);
}

// A [T][H][d] argument whose token rows lie `stride` elements apart: whole rows, 16-byte units.
inline bool valid_rows(const void *p, int64_t stride, int32_t H, int32_t d, int32_t dtype) {
    return p && aligned16(p) && stride >= (int64_t)H * d && stride * elem_size(dtype) % 16 == 0;
}

// The pool holds such a cache: its pages are large enough, and 16-byte accesses to them are aligned.
inline bool cache_view(const kda_pool *pool, int32_t Hkv, int32_t d, int32_t fmt, int32_t page_tokens, void *pool_base,
                const int32_t *table, int32_t max_pages, int32_t *status, kda::KvView &v) {
    if (!pool || !valid_cache(Hkv, d, fmt, page_tokens) || !pool_base || !aligned16(pool_base) || max_pages < 0 ||
        (max_pages > 0 && !table) || !status || (int64_t)max_pages * page_tokens > kMaxTokens)
        return false;
    const int64_t rec = record_bytes(d, fmt, page_tokens);
    if (pool->page_bytes < rec * Hkv) return false;
    v.base = static_cast<uint8_t *>(pool_base);
    v.page_bytes = pool->page_bytes;
    v.num_pages = pool->num_pages;
    v.page_tokens = page_tokens;
    v.Hkv = Hkv;
    v.d = d;
    v.fmt = fmt;
    v.rec_bytes = (int32_t)rec;
    v.table = table;
    v.max_pages = max_pages;
    v.status = status;
    return true;
}

inline bool valid_batch(int32_t nseq, int64_t T_tot, int32_t max_q, int32_t dtype) {
    return nseq > 0 && T_tot >= 0 && T_tot <= INT32_MAX - 1024 && max_q >= 0 && (dtype == KDA_F32 || dtype == KDA_BF16);
}

inline int status_of(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ECUDA; }

}  // namespace host
}  // namespace kda
