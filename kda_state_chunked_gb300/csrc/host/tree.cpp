// C ABI of speculation with trees of drafts: the plan of a tree, keeping the accepted branch in the key/value
// cache, and verifying a tree against recurrent states.  As the cache's calls these are stream-ordered, allocate
// nothing and never wait for the device; trees, branches and lengths stay on the device and are checked there.
#include "kv_host.h"

namespace {

using namespace kda::host;

// A batch of trees: cu_q cuts T_tot drafts into sequences of at most max_q.
bool valid_trees(int32_t nseq, int64_t T_tot, int32_t max_q) {
    return valid_batch(nseq, T_tot, max_q, KDA_F32) && max_q <= KDA_TREE_MAX;
}

bool overlap(const void *a, const void *b, int64_t bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y ? y - x < (uintptr_t)bytes : x - y < (uintptr_t)bytes;
}

// What verifying and accepting share; false where the arguments do not fit.
bool tree_args(const kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t B, int64_t T_tot, int32_t max_q,
               const int32_t *cu_q, const void *q, const void *k, const void *v, const void *alpha, const void *beta,
               const float *conv_w, void *pool_base, const int32_t *state_pages, int32_t *status,
               kda::VerifyTreeArgs &a) {
    if (!cu_q || !q || !k || !v || !alpha || !beta || !conv_w || !pool_base || !state_pages || !aligned16(q) ||
        !aligned16(k) || !aligned16(v) || !aligned16(alpha) || !aligned16(conv_w) || !aligned16(pool_base))
        return false;
    a.H = H; a.d = d; a.dtype = dtype; a.B = B; a.max_q = max_q; a.T_tot = T_tot;
    a.cu_q = cu_q; a.q = q; a.k = k; a.v = v; a.alpha = alpha; a.beta = beta; a.conv_w = conv_w;
    a.pool = kda::pool_view(pool, pool_base, H, d, dtype);
    a.state_pages = state_pages;
    a.status = status;
    return true;
}

bool tree_shape(const kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t B, int64_t T_tot, int32_t max_q,
                const int32_t *status) {
    return pool && kda_object_bytes(H, d, dtype) > 0 && valid_trees(B, T_tot, max_q) && (int64_t)B * H <= INT32_MAX && status;
}

}  // namespace

extern "C" {

int kda_tree_plan(int32_t nseq, int64_t T_tot, int32_t max_q, const int32_t *cu_q, const int32_t *kv_len,
                  const int32_t *parent, uint64_t *mask, int32_t *pos, int32_t *status_dev, void *stream) {
    if (!valid_trees(nseq, T_tot, max_q) || !status_dev) return KDA_EINVAL;
    if (T_tot == 0 || max_q == 0) return KDA_OK;
    if (!cu_q || !kv_len || !parent || !mask || !pos) return KDA_EINVAL;
    kda::TreePlanArgs a{};
    a.nseq = nseq; a.max_q = max_q; a.T_tot = T_tot;
    a.cu_q = cu_q; a.kv_len = kv_len; a.parent = parent; a.mask = mask; a.pos = pos; a.status = status_dev;
    return status_of(kda::launch_tree_plan(a, static_cast<cudaStream_t>(stream)));
}

int kda_kv_accept(const kda_pool *pool, int32_t Hkv, int32_t d, int32_t fmt, int32_t page_tokens, int32_t nseq,
                  int64_t T_tot, int32_t max_q, const int32_t *cu_q, const int32_t *kv_len, const int32_t *page_table,
                  int32_t max_pages, const int32_t *path, const int32_t *accepted, int32_t *kv_len_out,
                  void *pool_base, int32_t *status_dev, void *stream) {
    kda::KvAcceptArgs a{};
    if (!cache_view(pool, Hkv, d, fmt, page_tokens, pool_base, page_table, max_pages, status_dev, a.kv) ||
        !valid_trees(nseq, T_tot, max_q) || !cu_q || !kv_len || !accepted || !kv_len_out || (T_tot > 0 && !path) ||
        overlap(kv_len, kv_len_out, (int64_t)nseq * 4) || overlap(accepted, kv_len_out, (int64_t)nseq * 4) || 2 * (int64_t)nseq * Hkv > INT32_MAX)
        return KDA_EINVAL;
    a.nseq = nseq; a.max_q = max_q; a.T_tot = T_tot;
    a.cu_q = cu_q; a.kv_len = kv_len; a.path = path; a.accepted = accepted; a.kv_len_out = kv_len_out;
    return status_of(kda::launch_kv_accept(a, static_cast<cudaStream_t>(stream)));
}

int kda_verify_tree(const kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t B, int64_t T_tot, int32_t max_q,
                    const int32_t *cu_q, const int32_t *parent, const void *q, const void *k, const void *v,
                    const void *alpha, const void *beta, const float *conv_w, void *o, const void *pool_base,
                    const int32_t *state_pages, int32_t *status_dev, void *stream) {
    if (!tree_shape(pool, H, d, dtype, B, T_tot, max_q, status_dev)) return KDA_EINVAL;
    if (T_tot == 0 || max_q == 0) return KDA_OK;
    kda::VerifyTreeArgs a{};
    if (!parent || !o || !aligned16(o) ||
        !tree_args(pool, H, d, dtype, B, T_tot, max_q, cu_q, q, k, v, alpha, beta, conv_w, const_cast<void *>(pool_base),
                   state_pages, status_dev, a))
        return KDA_EINVAL;
    a.parent = parent; a.o = o;
    return status_of(kda::launch_verify_tree(a, static_cast<cudaStream_t>(stream)));
}

int kda_verify_tree_accept(const kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t B, int64_t T_tot,
                           int32_t max_q, const int32_t *cu_q, const int32_t *path, const int32_t *accepted,
                           const void *q, const void *k, const void *v, const void *alpha, const void *beta,
                           const float *conv_w, void *pool_base, const int32_t *state_pages, int32_t *status_dev,
                           void *stream) {
    if (!tree_shape(pool, H, d, dtype, B, T_tot, max_q, status_dev)) return KDA_EINVAL;
    if (T_tot == 0 || max_q == 0) return KDA_OK;
    kda::VerifyTreeArgs a{};
    if (!path || !accepted ||
        !tree_args(pool, H, d, dtype, B, T_tot, max_q, cu_q, q, k, v, alpha, beta, conv_w, pool_base, state_pages,
                   status_dev, a))
        return KDA_EINVAL;
    a.path = path; a.accepted = accepted;
    return status_of(kda::launch_verify_tree_accept(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
