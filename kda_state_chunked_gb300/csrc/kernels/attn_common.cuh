// What the two attention kernels share: row tiles, the tokens each sees, the even split of all
// their units over the CTAs, and the joining of partial results.
//
// The split: every row tile of every sequence and head is an item of >= 1 units of UNIT cached
// tokens (an item that sees nothing has one, which writes its zeros).  With W units in all,
// CTA c takes units [c W / C, (c + 1) W / C) of the list ordered by sequence, row tile, head: each
// CTA has the same work however ragged the lengths are, and the lengths stay on the device.
#pragma once

#include <cmath>

#include "kv_common.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace attn {

// Trees of drafts are these kernels compiled again (attn_tree_decode.cu, attn_tree_prefill.cu), with masks in the place of
// the causal rule.  Known when compiling: a branch on the call's mask in what follows, taken by the warp that walks the units,
// cost the prompts' kernel registers (8-bit cache, 4096 tokens behind 12288: 1,103 us, 1,029 without).
#ifdef KDA_ATTN_TREE
constexpr bool kTree = true;
#else
constexpr bool kTree = false;
#endif

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Row tile rt of sequence s.  Row r of a sequence is (token r / G, head r % G of the group).
struct Tile {
    int32_t s, rt, tiles;         // tiles: row tiles of the sequence
    KvSeq q;
    int32_t row0, nrows;
    int32_t pmin, pmax;           // positions of its first and last row's token
    int32_t first, sinks, units;  // unit where its window begins, sink units before that, units in all
};

// Token r / G of row r of a sequence (r < 2^31): the high half of r ceil(2^32 / G) is that or one more.
__device__ __forceinline__ int32_t token_of(const AttnArgs &a, int32_t r) {
    if (a.G == 1) return r;
    const uint32_t q = __umulhi((uint32_t)r, a.g_magic);
    return (int32_t)(q * (uint32_t)a.G > (uint32_t)r ? q - 1 : q);
}

template <int ROWS>
__device__ __forceinline__ int32_t tiles_of(const AttnArgs &a, const KvSeq &q) {
    return (int32_t)(((int64_t)q.n * a.G + ROWS - 1) / ROWS);
}

template <int ROWS, int UNIT>
__device__ __forceinline__ Tile make_tile(const AttnArgs &a, int32_t s, const KvSeq &q, int32_t rt) {
    Tile t;
    t.s = s;
    t.rt = rt;
    t.q = q;
    t.tiles = tiles_of<ROWS>(a, q);
    t.row0 = rt * ROWS;
    t.nrows = min(ROWS, q.n * a.G - t.row0);
    const int32_t base = q.len - q.n;
    if (kTree) {                  // a tree's rows see what is before its drafts, and drafts by their own masks
        t.pmin = base - 1;
        t.pmax = base + q.n - 1;
    } else {
        t.pmin = base + token_of(a, t.row0);
        t.pmax = base + token_of(a, t.row0 + t.nrows - 1);
    }
    t.first = t.sinks = 0;
    if (t.pmax < 0) {             // more new tokens than the cache holds: these rows see nothing
        t.units = 1;
        return t;
    }
    if (a.window > 0) {
        t.first = max(0, t.pmin - a.window + 1) / UNIT;
        t.sinks = min(t.first, (a.sinks + UNIT - 1) / UNIT);
    }
    t.units = t.sinks + t.pmax / UNIT - t.first + 1;
    return t;
}

// First token of the tile's unit u.
template <int UNIT>
__device__ __forceinline__ int32_t unit_token(const Tile &t, int32_t u) {
    return (u < t.sinks ? u : t.first + u - t.sinks) * UNIT;
}

// Whether position p sees token j.
__device__ __forceinline__ bool sees(const AttnArgs &a, int32_t p, int32_t j) {
    return j <= p && (a.window <= 0 || j > p - a.window || j < a.sinks);
}
// A draft of a tree: what it sees of the drafts, and its position (between the first draft's place and the last's).
struct Draft {
    uint64_t mask;
    int32_t pos;
};
__device__ __forceinline__ Draft draft_of(const AttnArgs &a, int32_t tok0, int32_t n, int32_t base, int32_t tok) {
    Draft r;
    r.mask = __ldg(a.mask + tok0 + tok) & (~0ull >> (kTreeMost - n));   // (1 <= n <= kTreeMost)
    r.pos = a.window > 0 ? min(max(__ldg(a.pos + tok0 + tok), base), base + n - 1) : base;
    return r;
}
// Whether it sees token j, base being the first draft's place.
__device__ __forceinline__ bool draft_sees(const AttnArgs &a, const Draft &r, int32_t base, int32_t j) {
    if (j < base) return a.window <= 0 || j > r.pos - a.window || j < a.sinks;
    return j - base < kTreeMost && (r.mask >> (j - base) & 1u);
}

// Whether any / every row of the tile sees some / all of tokens [t0, t0 + n).
__device__ __forceinline__ bool any_sees(const AttnArgs &a, const Tile &t, int32_t t0, int32_t n) {
    return t0 <= t.pmax && (a.window <= 0 || t0 + n - 1 > t.pmin - a.window || t0 < a.sinks);
}
__device__ __forceinline__ bool all_see(const AttnArgs &a, const Tile &t, int32_t t0, int32_t n) {
    return t0 + n - 1 <= t.pmin && (a.window <= 0 || t0 > t.pmax - a.window || t0 + n <= a.sinks);
}

// CTA that holds unit u of W.
__device__ __forceinline__ int32_t cta_of(int64_t u, int64_t W, int32_t C) {
    return (int32_t)(((u + 1) * C - 1) / W);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ptx::mbar_wait with its loop kept rolled: these kernels wait in many places, and the unrolled
// loops alone came to 85 KB of code.  NS: nanoseconds between looks, for warps that run ahead and so
// mostly wait; a warp that looks all the time takes a third of its scheduler's issue slots.
template <int NS = 0>
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, volatile int *err) {
#pragma unroll 1
    for (uint32_t i = 0; i < ptx::kSpinLimit >> (NS ? 4 : 0); ++i) {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if (err && *err) return false;
        if (NS) __nanosleep(NS);
    }
    if (err) *err = 1;
    return false;
}

// A group of warps of which one looks, by look(), and the others stand at named barrier `id`.  All get
// its answer, and a wait that runs out sends the whole group out of its loop: were one warp to leave by
// itself, the others would stand at the group's next barrier for good.
template <int ID_THREADS, class F>
__device__ __forceinline__ bool wait_together(F look, bool looks, int id) {
    uint32_t ok = 1;
    if (looks) ok = look();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %0, 0;\n\tbarrier.cta.red.and.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "+r"(ok)
        : "r"(id), "n"(ID_THREADS)
        : "memory");
    return ok != 0;
}

// The matrix unit cuts its sums instead of rounding them: over 27,000 products on one accumulator (a context
// of a million tokens, where an item has a CTA for itself) outputs came out 2.5e-3 too small, more than
// half a bf16's step.  So an item is taken in pieces of that many units, whose results are added in
// rounded fp32 in the CTA's partial result: at most 2,048 products a piece, 1e-4.
constexpr int kPieceUnits = 256;

// What a warp that walks the list of units says of each (bits of a job's flags): first, last unit of a
// piece; every row sees every token; the item's own first, last unit is in this CTA; no unit, the end;
// the CTA has a further piece of the item, had one before.
enum : int32_t { kBegin = 1, kEnd = 2, kWhole = 4, kStop = 8, kStarts = 16, kEnds = 32, kMore = 64, kAgain = 128 };

// The flags of a piece's ends, for the i-th unit of an item in this CTA; last: the last one.
__device__ __forceinline__ int32_t piece_flags(int32_t i, bool last) {
    const int32_t k = i % kPieceUnits;
    return (k == 0 ? kBegin : 0) | (last || k + 1 == kPieceUnits ? kEnd : 0) | (!last && k + 1 == kPieceUnits ? kMore : 0) |
           (i >= kPieceUnits ? kAgain : 0);
}

// A place in the list of units.
struct Walk {
    Tile t;
    int32_t h, u;
    int64_t left;
};

__device__ __forceinline__ KvSeq seq_of(const AttnArgs &a, int s) {
    const KvSeq q = kv_seq(a.cu_q, a.kv_len, s, a.T_tot, a.max_q, a.kv);
    if (kTree && q.len < q.n) {   // drafts without a place
        flag_status(a.kv.status, KDA_DEV_BAD_META);
        return {0, 0, 0};
    }
    return q;
}

template <int ROWS, int UNIT>
__device__ __forceinline__ void next_item(const AttnArgs &a, Walk &w) {
    w.u = 0;
    if (++w.h < a.kv.Hkv) return;
    w.h = 0;
    int s = w.t.s, rt = w.t.rt + 1;
    KvSeq q = w.t.q;
    if (rt >= w.t.tiles) {
        rt = 0;
        do q = seq_of(a, ++s);
        while (q.n == 0 && s + 1 < a.nseq);
    }
    w.t = make_tile<ROWS, UNIT>(a, s, q, rt);
}

template <int D>
constexpr int kPartRow = D + 4;   // floats of a partial row: o, m, l, 2 free (rows stay 16-byte aligned)

__device__ __forceinline__ void store_row4(void *o, int dtype, int64_t at, float4 v) {
    if (dtype == KDA_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(o) + at) = v;
    } else {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
        uint2 u;
        u.x = *reinterpret_cast<const uint32_t *>(&x);
        u.y = *reinterpret_cast<const uint32_t *>(&y);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(o) + at) = u;
    }
}

// log-sum-exp from a base-2 maximum and the sum above it.
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2; }

// Join the partial results of the items that several CTAs touched: block (c, y) takes rows y,
// y + gridDim.y, ... of the item that starts in CTA c and ends later, a warp a row.  Few and small
// items, so this is bound by latency: a lane holds D / 32 columns, and the loads of four pieces are
// under way at a time.
template <int D, int ROWS>
__global__ void __launch_bounds__(128) attn_join_kernel(AttnArgs a) {
    ptx::grid_dep_wait();
    const AttnSplit sp = a.split[blockIdx.x];
    if (sp.last_cta < 0) return;
    const int c0 = blockIdx.x, c1 = sp.last_cta, lane = threadIdx.x % 32;
    constexpr int kCols = D / 32;
    for (int r = blockIdx.y * 4 + threadIdx.x / 32; r < sp.nrows; r += gridDim.y * 4) {
        auto piece = [&](int c) { return a.part + ((int64_t)(c * 2 + (c == c0)) * ROWS + r) * kPartRow<D>; };
        float m = -INFINITY;
        for (int c = c0 + lane; c <= c1; c += 32) m = fmaxf(m, piece(c)[D]);
        for (int i = 16; i; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, i));
        const float ref = m == -INFINITY ? 0.f : m;
        float l = 0.f, o[kCols];
#pragma unroll
        for (int j = 0; j < kCols; ++j) o[j] = 0.f;
#pragma unroll 4
        for (int c = c0; c <= c1; ++c) {
            const float *p = piece(c);
            const float w = exp2f(p[D] - ref);
            l += w * p[D + 1];
#pragma unroll
            for (int j = 0; j < kCols; ++j) o[j] += w * p[lane * kCols + j];
        }
        const int row = sp.row0 + r;
        const int32_t tok = token_of(a, row);
        const int64_t at = (int64_t)(sp.row_tok + tok) * a.Hq + sp.head * a.G + row - tok * a.G;
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            const float v = l == 0.f ? 0.f : o[j] * inv;
            if (a.dtype == KDA_F32) static_cast<float *>(a.o)[at * D + lane * kCols + j] = v;
            else static_cast<__nv_bfloat16 *>(a.o)[at * D + lane * kCols + j] = __float2bfloat16_rn(v);
        }
        if (a.lse && lane == 0) a.lse[at] = lse_of(m, l);
    }
}

}  // namespace attn
}  // namespace kda
