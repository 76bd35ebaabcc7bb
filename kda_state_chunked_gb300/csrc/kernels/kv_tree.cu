// Trees of drafts in the key/value cache: the plan of a tree, and keeping its accepted branch.
//
// Both are bound by latency: a plan reads a word a draft, a branch is some rows of a few blocks.  Keeping the branches of
// 256 requests (1 to 64 drafts, 8 heads of 128) takes 11.3 us over the 8-bit cache and 7.1 over the 16-bit one, one request's
// 2.9 us; a plan 2.6 to 2.9.
#include "kv_common.cuh"

namespace kda {
namespace {

// A CTA a sequence, a thread a draft.  mask_i = 1 << i | mask_parent and depth_i = depth_parent + 1, by pointer
// doubling: after step k a draft knows its 2^k nearest ancestors (itself among them) and the one behind them.
__global__ void __launch_bounds__(kTreeMost) tree_plan_kernel(TreePlanArgs a) {
    __shared__ uint64_t mask[kTreeMost];
    __shared__ int32_t up[kTreeMost];
    const int s = blockIdx.x, i = threadIdx.x;
    const int64_t first = __ldg(a.cu_q + s), end = __ldg(a.cu_q + s + 1), len = __ldg(a.kv_len + s), n = end - first;
    if (first < 0 || n < 0 || end > a.T_tot || n > a.max_q || len < n) {
        if (i == 0) flag_status(a.status, KDA_DEV_BAD_META);
        return;
    }
    int32_t p = -1;
    if (i < n) p = __ldg(a.parent + first + i);
    if (__syncthreads_or(p < -1 || (i < n && p >= i))) {
        if (i == 0) flag_status(a.status, KDA_DEV_BAD_META);
        // the calls behind see no parents: what an earlier plan (or nobody) wrote here must not pass for this tree's
        if (i < n && a.pos[first + i] >= 0) a.mask[first + i] = 0, a.pos[first + i] = -1;
        return;
    }
    uint64_t m = 1ull << i;
#pragma unroll 1
    for (int k = 1; k < kTreeMost; k *= 2) {
        mask[i] = m, up[i] = p;
        if (!__syncthreads_or(p >= 0)) break;
        if (p >= 0) m |= mask[p], p = up[p];
        __syncthreads();
    }
    if (i < n) {
        a.mask[first + i] = m;
        a.pos[first + i] = (int32_t)(len - n) + __popcll(m) - 1;
    }
}

// A CTA takes the keys or the values of one (sequence, head): the rows that move go through registers, all of them
// read before the first is written, for a row's new place may be another's old one.  In the 8-bit form the blocks
// that rows come to from other blocks get their scales first; what stays in such a block is coded anew where the
// scale grows.  Up to 63 rows move, over at most kBlocks blocks.
constexpr int kAcceptThreads = 128;
constexpr int kBlocks = (kTreeMost + 14) / 16 + 1;   // of 16 tokens, the drafts beginning anywhere in the first

template <int FMT, int D>
__global__ void __launch_bounds__(kAcceptThreads) kv_accept_kernel(KvAcceptArgs a) {
    constexpr int kRow = kKvRow<FMT, D>, kUnits = kRow / 16;            // 16-byte units a row
    constexpr int kHold = (kTreeMost * kUnits + kAcceptThreads - 1) / kAcceptThreads;
    __shared__ int32_t path[kTreeMost], page[kBlocks];
    __shared__ uint32_t top[kBlocks];                                   // largest |x| that comes from other blocks
    __shared__ float was[kBlocks];                                      // scales before
    __shared__ int32_t stays[kBlocks];                                  // an accepted token was there before
    const int tid = threadIdx.x, pt = a.kv.page_tokens;
    const bool is_v = blockIdx.x & 1;
    const int head = (int)(blockIdx.x / 2 % (uint32_t)a.kv.Hkv), s = (int)(blockIdx.x / 2 / (uint32_t)a.kv.Hkv);
    const int64_t first = __ldg(a.cu_q + s), end = __ldg(a.cu_q + s + 1), n = end - first;
    const int32_t len = __ldg(a.kv_len + s), m = __ldg(a.accepted + s);
    const bool one = tid == 0 && head == 0 && !is_v;                    // speaks for the sequence
    if (first < 0 || n < 0 || end > a.T_tot || n > a.max_q || len < n || len > (int64_t)a.kv.max_pages * pt || m < 0 || m > n) {
        if (one) flag_status(a.kv.status, KDA_DEV_BAD_META);
        return;
    }
    const int32_t base = len - (int32_t)n;
    int32_t from = -1;
    if (tid < m) path[tid] = from = __ldg(a.path + first + tid);
    if (tid < kBlocks) top[tid] = 0, stays[tid] = 0;
    __syncthreads();
    const bool wrong = tid < m && (from < (tid ? path[tid - 1] + 1 : 0) || from >= n);
    if (__syncthreads_or(wrong)) {
        if (one) flag_status(a.kv.status, KDA_DEV_BAD_META);
        return;
    }
    // path[i] >= i, and from the first row that moves on all do
    const int still = __syncthreads_count(tid < m && from == tid);
    if (still == m) {
        if (one) a.kv_len_out[s] = base + m;
        return;
    }
    const int block0 = (base + still) / pt, blocks = (base + path[m - 1]) / pt - block0 + 1;   // <= kBlocks
    bool lost = false;
    if (tid < blocks) {
        const int32_t id = __ldg(a.kv.table + (int64_t)s * a.kv.max_pages + block0 + tid);
        page[tid] = id;
        lost = (uint32_t)id >= (uint32_t)a.kv.num_pages;
    }
    if (__syncthreads_or(lost)) {
        if (one) flag_status(a.kv.status, KDA_DEV_BAD_PAGE);
        return;
    }
    if (one) a.kv_len_out[s] = base + m;
    auto record = [&](int b) { return a.kv.base + (int64_t)page[b] * a.kv.page_bytes + (int64_t)head * a.kv.rec_bytes; };
    auto tile = [&](int b) { return record(b) + (is_v ? pt * kRow : 0); };
    auto scale_at = [&](int b) { return reinterpret_cast<float *>(record(b) + 2 * pt * kRow) + (is_v ? 1 : 0); };
    if (FMT == KDA_KV_I8 && tid < blocks) was[tid] = fabsf(*scale_at(tid));
    uint4 u[kHold];
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
        const int i = still + (tid + k * kAcceptThreads) / kUnits, unit = (tid + k * kAcceptThreads) % kUnits;
        if (i < m) {
            const int at = base + path[i], b = at / pt;
            u[k] = *reinterpret_cast<const uint4 *>(tile(b - block0) + kv_tile_off<kRow>(pt, at - b * pt, 16 * unit));
        }
    }
    __syncthreads();
    if constexpr (FMT == KDA_KV_BF16) {
#pragma unroll
        for (int k = 0; k < kHold; ++k) {
            const int i = still + (tid + k * kAcceptThreads) / kUnits, unit = (tid + k * kAcceptThreads) % kUnits;
            if (i < m) {
                const int at = base + i, b = at / pt;
                *reinterpret_cast<uint4 *>(tile(b - block0) + kv_tile_off<kRow>(pt, at - b * pt, 16 * unit)) = u[k];
            }
        }
    } else {
        auto value = [](const uint4 &c, int j, float sc) {
            const uint32_t w = j < 4 ? c.x : j < 8 ? c.y : j < 12 ? c.z : c.w;
            return __fmul_rn((float)(int8_t)(w >> (8 * (j & 3))), sc);
        };
#pragma unroll
        for (int k = 0; k < kHold; ++k) {
            const int i = still + (tid + k * kAcceptThreads) / kUnits;
            if (i >= m) continue;
            const int to = (base + i) / pt - block0, of = (base + path[i]) / pt - block0;
            if (to == of) {
                stays[to] = 1;
                continue;
            }
            uint32_t most = 0;
#pragma unroll
            for (int j = 0; j < 16; ++j) most = max(most, __float_as_uint(value(u[k], j, was[of])) & 0x7FFFFFFFu);
            atomicMax(&top[to], most);
        }
        __syncthreads();
        auto scale_of = [&](int b) {   // of a block that rows go to, in bits
            const uint32_t came = __float_as_uint(__fdiv_rn(__uint_as_float(top[b]), 127.f)) & 0x7FFFFFFFu;
            const bool old = (block0 + b) * pt < base + still || stays[b];
            return old ? max(came, __float_as_uint(was[b])) : came;
        };
#pragma unroll
        for (int k = 0; k < kHold; ++k) {
            const int i = still + (tid + k * kAcceptThreads) / kUnits, unit = (tid + k * kAcceptThreads) % kUnits;
            if (i >= m) continue;
            const int at = base + i, to = at / pt - block0, of = (base + path[i]) / pt - block0;
            const uint32_t bits = scale_of(to);
            uint4 c = u[k];
            if (to != of || bits != __float_as_uint(was[to])) {
                float x[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = value(u[k], j, was[of]);
                const uint2 lo = codes8(x, __uint_as_float(bits)), hi = codes8(x + 8, __uint_as_float(bits));
                c = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
            *reinterpret_cast<uint4 *>(tile(to) + kv_tile_off<kRow>(pt, at - (block0 + to) * pt, 16 * unit)) = c;
        }
        // the rows in front of those that move: all in the first block, for a later one holds rows that move alone
        const uint32_t bits = scale_of(0);
        if (bits != __float_as_uint(was[0])) {
            const int rows = base + still - block0 * pt;
            for (int i = tid; i < rows * kUnits; i += kAcceptThreads) {
                uint4 *at = reinterpret_cast<uint4 *>(tile(0) + kv_tile_off<kRow>(pt, i / kUnits, 16 * (i % kUnits)));
                const uint4 c = *at;
                float x[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = value(c, j, was[0]);
                const uint2 lo = codes8(x, __uint_as_float(bits)), hi = codes8(x + 8, __uint_as_float(bits));
                *at = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
        }
        const int last = (base + m - 1) / pt - block0;
        if (tid <= last) *scale_at(tid) = __uint_as_float(scale_of(tid));
    }
}

template <int FMT, int D>
cudaError_t accept(const KvAcceptArgs &a, cudaStream_t st) {
    kv_accept_kernel<FMT, D><<<(unsigned)(2 * (int64_t)a.nseq * a.kv.Hkv), kAcceptThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_plan(const TreePlanArgs &a, cudaStream_t s) {
    tree_plan_kernel<<<(unsigned)a.nseq, kTreeMost, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv_accept(const KvAcceptArgs &a, cudaStream_t s) {
    if (a.kv.d == 128) return a.kv.fmt == KDA_KV_I8 ? accept<KDA_KV_I8, 128>(a, s) : accept<KDA_KV_BF16, 128>(a, s);
    return a.kv.fmt == KDA_KV_I8 ? accept<KDA_KV_I8, 64>(a, s) : accept<KDA_KV_BF16, 64>(a, s);
}

}  // namespace kda
