// C ABI of the key/value cache and its attention: argument checks and launches.  Every call is
// stream-ordered, allocates nothing and never waits for the device; lengths and page tables stay
// on the device and are checked there.
#include <algorithm>
#include <cmath>

#include "kda.h"
#include "pool.h"
#include "../kda_internal.h"

namespace {

constexpr int64_t kWholeUnits = 6;         // units up to which an item of the register kernel is not split
constexpr int64_t kMaxTokens = 1 << 30;   // of a sequence: the kernels' positions and their differences fit int32

int64_t elem_size(int32_t dtype) { return dtype == KDA_BF16 ? 2 : 4; }
int64_t align_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool valid_cache(int32_t Hkv, int32_t d, int32_t fmt, int32_t page_tokens) {
    return Hkv > 0 && Hkv <= 4096 && (d == 64 || d == 128) && (fmt == KDA_KV_BF16 || fmt == KDA_KV_I8) &&
           page_tokens >= 16 && page_tokens <= kda::kKvMaxPageTokens && page_tokens % 16 == 0;
}

int64_t record_bytes(int32_t d, int32_t fmt, int32_t page_tokens) {
    return 2 * (int64_t)page_tokens * d * (fmt == KDA_KV_I8 ? 1 : 2) + (fmt == KDA_KV_I8 ? 16 : 0);
}

// A [T][H][d] argument whose token rows lie `stride` elements apart: whole rows, 16-byte units.
bool valid_rows(const void *p, int64_t stride, int32_t H, int32_t d, int32_t dtype) {
    return p && aligned16(p) && stride >= (int64_t)H * d && stride * elem_size(dtype) % 16 == 0;
}

// The pool holds such a cache: its pages are large enough, and 16-byte accesses to them are aligned.
bool cache_view(const kda_pool *pool, int32_t Hkv, int32_t d, int32_t fmt, int32_t page_tokens, void *pool_base,
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

bool valid_batch(int32_t nseq, int64_t T_tot, int32_t max_q, int32_t dtype) {
    return nseq > 0 && T_tot >= 0 && T_tot <= INT32_MAX - 1024 && max_q >= 0 && (dtype == KDA_F32 || dtype == KDA_BF16);
}

int status_of(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ECUDA; }

// Rows of a tile.  The register kernel holds 16 rows; with more rows a sequence it reads the cache
// again for every 16, while a tile of the tensor-memory kernel takes 256 of them in the same time.  32
// sequences of 4096 tokens and 8 heads of 128, with 16, 32 and 64 rows a head: 8-bit cache 78, 134 and
// 253 us by the first, 167, 168 and 171 by the second; 16-bit cache with 16 and 32 rows 107 and 193
// against 116 and 117.  float32 calls stay on the register kernel: its products split an operand into
// terms.
int32_t attn_rows(int32_t dtype, int32_t fmt, int32_t max_q, int32_t G) {
    const int64_t most = fmt == KDA_KV_I8 ? 2 * kda::kAttnDecodeRows : kda::kAttnDecodeRows;
    return dtype == KDA_F32 || (int64_t)max_q * G <= most ? kda::kAttnDecodeRows : kda::kAttnPrefillRows;
}

// Workspace of an attention call: [AttnSplit per CTA][partial results].
struct AttnWs {
    int64_t o_part, total;
};
int32_t attn_ctas(int32_t rows) { return rows == kda::kAttnDecodeRows ? kda::kAttnMaxCtas : kda::kAttnSms; }
AttnWs attn_ws(int32_t d, int32_t rows) {
    AttnWs w;
    w.o_part = align_up(attn_ctas(rows) * (int64_t)sizeof(kda::AttnSplit), 256);
    w.total = w.o_part + (int64_t)attn_ctas(rows) * 2 * rows * (d + 4) * 4;
    return w;
}

}  // namespace

extern "C" {

int64_t kda_kv_page_bytes(int32_t Hkv, int32_t d, int32_t fmt, int32_t page_tokens) {
    if (!valid_cache(Hkv, d, fmt, page_tokens)) return KDA_EINVAL;
    return align_up(record_bytes(d, fmt, page_tokens) * Hkv, 256);
}

int kda_kv_append(const kda_pool *pool, int32_t Hq, int32_t Hkv, int32_t d, int32_t dtype, int32_t fmt,
                  int32_t page_tokens, int32_t nseq, int64_t T_tot, int32_t max_q, const int32_t *cu_q,
                  const int32_t *kv_len, const int32_t *page_table, int32_t max_pages, const void *q,
                  int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                  const float *cos_sin, int32_t max_pos, int32_t rot_dim, int32_t interleaved, void *q_out,
                  void *pool_base, int32_t *status_dev, void *stream) {
    kda::KvAppendArgs a{};
    if (!cache_view(pool, Hkv, d, fmt, page_tokens, pool_base, page_table, max_pages, status_dev, a.kv) ||
        !valid_batch(nseq, T_tot, max_q, dtype))
        return KDA_EINVAL;
    if ((q == nullptr) != (q_out == nullptr) || (q && (Hq <= 0 || Hq > 4096))) return KDA_EINVAL;
    if (cos_sin ? (rot_dim <= 0 || rot_dim > d || rot_dim % 16 || max_pos <= 0 || !aligned16(cos_sin)) : rot_dim != 0)
        return KDA_EINVAL;
    if (T_tot == 0 || max_q == 0) return KDA_OK;
    if (!cu_q || !kv_len || max_pages == 0 || !valid_rows(k, k_stride, Hkv, d, dtype) ||
        !valid_rows(v, v_stride, Hkv, d, dtype) || (q && (!valid_rows(q, q_stride, Hq, d, dtype) || !aligned16(q_out))))
        return KDA_EINVAL;
    a.Hq = q ? Hq : 0; a.dtype = dtype; a.nseq = nseq; a.max_q = max_q; a.T_tot = T_tot;
    a.cu_q = cu_q; a.kv_len = kv_len;
    a.q = q; a.k = k; a.v = v;
    a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.cos_sin = cos_sin; a.max_pos = max_pos; a.rot_dim = rot_dim; a.interleaved = interleaved;
    a.q_out = q_out;
    return status_of(kda::launch_kv_append(a, static_cast<cudaStream_t>(stream)));
}

int kda_kv_gather(const kda_pool *pool, int32_t Hkv, int32_t d, int32_t dtype, int32_t fmt, int32_t page_tokens,
                  int32_t nseq, int64_t T_out, const int32_t *cu_out, const int32_t *begin,
                  const int32_t *page_table, int32_t max_pages, void *k_out, void *v_out, const void *pool_base,
                  int32_t *status_dev, void *stream) {
    kda::KvGatherArgs a{};
    if (!cache_view(pool, Hkv, d, fmt, page_tokens, const_cast<void *>(pool_base), page_table, max_pages, status_dev,
                    a.kv) ||
        !valid_batch(nseq, T_out, 0, dtype))
        return KDA_EINVAL;
    if (T_out == 0) return KDA_OK;
    if (!cu_out || !begin || max_pages == 0 || !k_out || !v_out || !aligned16(k_out) || !aligned16(v_out))
        return KDA_EINVAL;
    a.dtype = dtype; a.nseq = nseq; a.T_out = T_out;
    a.cu_out = cu_out; a.begin = begin; a.k_out = k_out; a.v_out = v_out;
    return status_of(kda::launch_kv_gather(a, static_cast<cudaStream_t>(stream)));
}

int64_t kda_attn_workspace_bytes(int32_t Hq, int32_t Hkv, int32_t d, int32_t dtype, int32_t nseq, int64_t T_tot,
                                 int32_t max_q) {
    if (Hkv <= 0 || Hq <= 0 || Hq > 4096 || Hq % Hkv || (d != 64 && d != 128) || !valid_batch(nseq, T_tot, max_q, dtype))
        return KDA_EINVAL;
    return std::max(attn_ws(d, attn_rows(dtype, KDA_KV_BF16, max_q, Hq / Hkv)).total,
                    attn_ws(d, attn_rows(dtype, KDA_KV_I8, max_q, Hq / Hkv)).total);   // serves either format
}

int kda_attn_paged(const kda_pool *pool, int32_t Hq, int32_t Hkv, int32_t d, int32_t dtype, int32_t fmt,
                   int32_t page_tokens, int32_t nseq, int64_t T_tot, int32_t max_q, const int32_t *cu_q,
                   const int32_t *kv_len, const int32_t *page_table, int32_t max_pages, const void *q,
                   int64_t q_stride, float scale, int32_t window, int32_t sinks, void *o, float *lse,
                   const void *pool_base, void *workspace, int64_t ws_bytes, int32_t *status_dev, void *stream) {
    kda::AttnArgs a{};
    if (!cache_view(pool, Hkv, d, fmt, page_tokens, const_cast<void *>(pool_base), page_table, max_pages, status_dev,
                    a.kv) ||
        !valid_batch(nseq, T_tot, max_q, dtype) || Hq <= 0 || Hq > 4096 || Hq % Hkv || !std::isfinite(scale) ||
        window < 0 || sinks < 0)
        return KDA_EINVAL;
    if ((int64_t)max_q * (Hq / Hkv) > INT32_MAX - 1024) return KDA_EINVAL;
    if (T_tot == 0 || max_q == 0) return KDA_OK;
    const int64_t need = kda_attn_workspace_bytes(Hq, Hkv, d, dtype, nseq, T_tot, max_q);
    if (!cu_q || !kv_len || !o || !aligned16(o) || !valid_rows(q, q_stride, Hq, d, dtype) || !workspace ||
        !aligned16(workspace) || ws_bytes < need)
        return KDA_EINVAL;
    a.Hq = Hq; a.G = Hq / Hkv; a.dtype = dtype; a.nseq = nseq; a.max_q = max_q; a.T_tot = T_tot;
    a.g_magic = a.G > 1 ? (uint32_t)(((1ull << 32) + a.G - 1) / a.G) : 0u;
    a.cu_q = cu_q; a.kv_len = kv_len;
    a.q = q; a.q_stride = q_stride;
    // a window (or sinks) as long as a sequence can be is none (are all of it)
    const int32_t longest = max_pages * page_tokens;
    a.scale = scale; a.window = window >= longest ? 0 : window; a.sinks = std::min(sinks, longest);
    a.o = o; a.lse = lse;
    const int32_t rows = attn_rows(dtype, fmt, max_q, a.G);
    const AttnWs w = attn_ws(d, rows);
    // the most units that the call can have bounds the CTAs worth launching
    const int64_t tiles = T_tot * a.G / rows + nseq;
    int64_t tokens = (int64_t)max_pages * page_tokens;   // that a row tile can see: window, sinks, a unit cut at both ends
    if (a.window) tokens = std::min<int64_t>(tokens, (int64_t)a.window + a.sinks + max_q + 3 * kda::kAttnMinUnit);
    const int64_t units = std::max<int64_t>(1, (tokens + kda::kAttnMinUnit - 1) / kda::kAttnMinUnit);
    a.ctas = (int32_t)std::min<int64_t>(attn_ctas(rows), std::max<int64_t>(1, tiles * Hkv * units));
    // Few, short items: a CTA each; splitting them costs another launch to join the parts.  64 items of
    // 256, 640 and 1000 tokens of an 8-bit cache (2, 5 and 8 units): 6.7, 10.0 and 13.0 us whole, 10.0,
    // 12.9 and 14.2 split; of 384 tokens of a 16-bit one (6 units) 8.0 and 11.3; but 4 items of 8 units
    // 12.7 and 10.7.
    a.whole = rows == kda::kAttnDecodeRows && (int64_t)max_q * a.G <= rows && (int64_t)nseq * Hkv <= kda::kAttnSms &&
              tokens <= kWholeUnits * (fmt == KDA_KV_I8 ? 128 : 64);
    if (a.whole) a.ctas = nseq * Hkv;
    a.split = static_cast<kda::AttnSplit *>(workspace);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + w.o_part);
    return status_of(rows == kda::kAttnDecodeRows ? kda::launch_attn_decode(a, static_cast<cudaStream_t>(stream))
                                                  : kda::launch_attn_prefill(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
