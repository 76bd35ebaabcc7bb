// Attention of many query rows over the paged cache (prompts, drafts of wide groups; bf16 calls).
//
//   S = Q K^T,  p = 2^(f S - m),  O += P V,  l += sum p,   f = scale log2 e (and the scales of the
//   8-bit form), m a running bound of the row's maximum
//
// on the fifth-generation tensor cores.  Bound: the matrix pipe, 4 D flops for each of the row
// tile's (row, token) pairs.  A row tile is 256 query rows of one key/value head, two halves of 128
// that take turns: while one half's warps turn scores into probabilities, the pipe works for the
// other.  Tensor memory holds S of both halves (128 columns each, P over its first half) and O of
// both: 512 columns.  Keys and values of a unit of 128 tokens are read once for both halves.
//
// One CTA of 28 warps an SM:
//   warps 0-15       softmax, eight to a half, two threads a row (64 tokens each): scores from tensor
//                    memory, probabilities back into it, at the end the output.  The probabilities
//                    are taken against a reference that follows the row's maximum only once that
//                    has grown by more than 2^8 (fp16 and bf16 have the room), so O is seldom
//                    rescaled.  With a thread a row a half took 3,300 cycles from its scores to its
//                    last probability where nothing is masked, with two 2,700.
//   warps 16-23      queries into shared memory; 8-bit cache: codes from global memory through
//                    registers to fp16 tiles (a page's bytes never lie in shared memory);
//                    16-bit cache: a look at values that not every row sees
//   warp 24          issues the products
//   warp 25          16-bit cache: bulk copies of pages, whose lines already lie as the matrix
//                    unit's 128-byte swizzle wants them
//   warp 26          walks the list of units and hands each on as a job: its tokens, records, scales
// The walk's divisions and table reads are in one place, up to eight units ahead: with a copy of it
// in every role the kernel was 220 KB of code and stood waiting for instructions, 9,700 cycles a
// unit instead of the 4,400 to 5,300 of now.
//
// Measured: 4096 queries of 32 heads of 128 behind 12288 tokens, 8-bit cache: 1,034 us, 930 TFLOP/s,
// 49% of the plain product's rate; four ragged prompts of up to 8192 tokens through a window of 1024:
// 283 us, 0.30 of that rate.  The pipe is busy 2,100 of a unit's cycles.  What stands in its way is a
// half's way from its scores to its probabilities (2,700 cycles) with the pipe's own 1,000 and two
// hand-overs behind it; the other half covers part of that only, as both use the same issue slots
// (63% taken).  One pass over the scores instead of two wants 32 more registers than there are:
// 20% slower, and 15% with registers taken from the other warps.
//
// Trees of drafts (compiled again, kTree): a job's pages are asked into L2 when it is handed on, keys and values of the
// 8-bit cache have registers of their own, probabilities over the 16-bit cache two terms.  32 ragged contexts of 512 to
// 32768 tokens, 32 heads (8 key/value), 16 drafts: 8-bit 512 us (618 without the first two), 16-bit 504 us (404 with one
// term); 16 trees of 33 to 64 drafts behind 4096 to 16384 tokens, 16-bit: 205 us.  For up to 128 rows a form was built in
// which the two halves take alternate units and join at an item's end: 608 us for the first, and not kept.
//
// 8-bit cache: as in the register kernel codes are exact in fp16 and query rows scaled by a power
// of two; the key scale of each 16 tokens multiplies f, the value scale goes into the exponent:
// p' = 2^(f S + log2 vs - b + 6), b a running bound of the row's own f S + log2 vs, and a group's sum
// of p' divided by 2^(log2 vs - b + m + 6) is its sum of p.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "tc_common.cuh"

namespace kda {
namespace {

using namespace attn;

constexpr int kRows = kAttnPrefillRows, kHalf = 128, kUnit = 128;
constexpr int kSoftWarps = 16, kLoadWarps = 8, kMmaWarp = 24, kCopyWarp = 25, kWalkWarp = 26, kThreads = 28 * 32;
constexpr float kGrow = 8.f;            // bits that a row's maximum may grow before O is rescaled
constexpr float kPBits = 6.f;           // 8-bit: bits that a probability is scaled up in fp16
// What an item (a row tile of a head) costs beyond its units, in units: the share of a CTA counts it.
// Its end stays in the pipe's way for one to two units' time, and its masked units take longer.  Four ragged
// windowed prompts, whose items have 1 to 11 units: 286 us, 375 with shares of equal units.
constexpr int kItem = 2;
constexpr int kJobs = 8;                // units handed out and not yet done with

// A unit of work.
struct __align__(16) Job {
    int32_t j0;                         // its first token
    int32_t flags;
    int32_t base;                       // position of the sequence's first query
    int32_t row0, nrows, tok0, head;    // the row tile
    uint32_t live;                      // groups of 16 tokens that are there
    int32_t last_cta, pmin, pmax;
    uint32_t nans;                      // 8-bit: groups whose value scale is no number
    int32_t slot[8];                    // of each group: first token's slot in its page,
    int64_t rec[8];                     // its record's place in the pool (the pool's first where it is not there),
    float ks[8], lg[8];                 // 8-bit: key scale, log2 of the value scale (-infinity for 0 and for no number)
};

template <int D>
struct Lay {
    static constexpr int half_q = kHalf * D * 2, tile = kUnit * D * 2, blk = kUnit * 128;   // 64-column blocks
    static constexpr int q = 0, k = 2 * half_q, v = k + 2 * tile, misc = v + 2 * tile;
    static constexpr int qs = misc;                        // [2][256] row factors
    static constexpr int jobs = qs + 2 * kRows * 4;        // [kJobs]
    static constexpr int pair = jobs + kJobs * (int)sizeof(Job);  // [2][2][256][2] what a row's two threads tell each other
    static constexpr int bad = pair + 2 * 2 * kRows * 8;   // [2][4] tokens taken out of a value tile
    static constexpr int plan = bad + 2 * 16;              // the split's scratch
    static constexpr int bar = plan + 4096;
    static constexpr int total = bar + 512;
};

enum Bar { QFULL, QEMPTY, KFULL, KEMPTY = KFULL + 2, VFULL = KEMPTY + 2, VEMPTY = VFULL + 2, VRAW = VEMPTY + 2,
           SFULL = VRAW + 2, PFULL = SFULL + 2, OFULL = PFULL + 2, DRAIN = OFULL + 2, JFULL, JEMPTY = JFULL + kJobs,
           NBAR = JEMPTY + kJobs };

template <int FMT>
__host__ __device__ constexpr uint32_t idesc(int M, int N, int b_mn) {
    const uint32_t d = ptx::idesc_bf16(M, N, 0, b_mn);
    return FMT == KDA_KV_I8 ? d & ~((1u << 7) | (1u << 10)) : d;   // fp16 operands instead of bf16
}

template <int FMT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (FMT == KDA_KV_I8) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        return tcx::f2_to_bf2(lo, hi);
    }
}

// 32 lanes x 16 columns, a lane a thread.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float (&v)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
                   "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
                 : "r"(addr)
                 : "memory");
}
// Wait for the loads of v from tensor memory; naming the registers keeps their uses behind it.
__device__ __forceinline__ void wait_ld(float (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                 :
                 : "memory");
}
__device__ __forceinline__ float tmem_ld1(uint32_t addr) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(addr) : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r)::"memory");
    return __uint_as_float(r);
}
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Sixteen codes as fp16, in two 16-byte units.
__device__ __forceinline__ void codes_to_half(uint4 c, uint4 &lo, uint4 &hi) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = w[i] ^ 0x80808080u;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const uint32_t u = __byte_perm(b, 0x64646464u, y ? 0x4342 : 0x4140);
            const uint32_t k = 0x64806480u;   // 1024 + 128 in both halves
            const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&u), *reinterpret_cast<const __half2 *>(&k));
            r[2 * i + y] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    lo = make_uint4(r[0], r[1], r[2], r[3]);
    hi = make_uint4(r[4], r[5], r[6], r[7]);
}

// Units of sequence s over all heads and what its items add, summed by a warp.
__device__ __forceinline__ int64_t seq_units(const AttnArgs &a, int s, int lane) {
    const KvSeq q = seq_of(a, s);
    const int n = tiles_of<kRows>(a, q);
    int64_t w = 0;
#pragma unroll 1
    for (int i = lane; i < n; i += 32) w += make_tile<kRows, kUnit>(a, s, q, i).units + kItem;
    for (int i = 16; i; i >>= 1) w += __shfl_xor_sync(0xFFFFFFFFu, w, i);
    return w * a.kv.Hkv;
}

// This CTA's share of the units, into *start (left = 0: none).  W and the number of CTAs that take
// part come back too.  All warps call it; sums[512] is shared scratch.
__device__ __forceinline__ void find_share(const AttnArgs &a, int64_t *sums, Walk *start, int64_t &W, int32_t &C) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int per = (a.nseq + 511) / 512, groups = (a.nseq + per - 1) / per;   // sequences a sum
#pragma unroll 1
    for (int i = warp; i < groups; i += kThreads / 32) {
        int64_t w = 0;
#pragma unroll 1
        for (int s = i * per; s < min(a.nseq, (i + 1) * per); ++s) w += seq_units(a, s, lane);
        if (lane == 0) sums[i] = w;
    }
    __syncthreads();
    if (warp == 0) {
        int64_t all = 0;
        for (int i = lane; i < groups; i += 32) all += sums[i];
        for (int i = 16; i; i >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, i);
        const int32_t c = (int32_t)min((int64_t)a.ctas, all);
        Walk w{};
        if ((int32_t)blockIdx.x < c) {
            const int64_t begin = (int64_t)blockIdx.x * all / c, end = (int64_t)(blockIdx.x + 1) * all / c;
            int64_t at = begin;
            int i = 0;
            while (at >= sums[i]) at -= sums[i++];
            int s = i * per;
#pragma unroll 1
            for (int64_t n; at >= (n = seq_units(a, s, lane)); ++s) at -= n;
            const KvSeq q = seq_of(a, s);
#pragma unroll 1
            for (int base = 0;; base += 32) {           // the tile: prefix sums over 32 tiles at a time
                const int rt = base + lane, n = tiles_of<kRows>(a, q);
                const int64_t mine = rt < n ? (int64_t)(make_tile<kRows, kUnit>(a, s, q, rt).units + kItem) * a.kv.Hkv : 0;
                int64_t x = mine;
                for (int j = 1; j < 32; j <<= 1) {
                    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, j);
                    if (lane >= j) x += y;
                }
                const uint32_t hit = __ballot_sync(0xFFFFFFFFu, at < x);
                if (hit) {
                    const int f = __ffs(hit) - 1;
                    at -= __shfl_sync(0xFFFFFFFFu, x - mine, f);
                    w.t = make_tile<kRows, kUnit>(a, s, q, base + f);
                    break;
                }
                at -= __shfl_sync(0xFFFFFFFFu, x, 31);
            }
            w.h = (int32_t)(at / (w.t.units + kItem));
            w.u = (int32_t)(at % (w.t.units + kItem));
            w.left = end - begin;
            if (w.u >= w.t.units) {                     // behind the units of an item: on to the next one
                w.left -= w.t.units + kItem - w.u;
                if (w.left > 0) next_item<kRows, kUnit>(a, w);
            }
        }
        __syncwarp();
        if (lane == 0) {
            *start = w;
            sums[0] = all;
        }
    }
    __syncthreads();
    W = sums[0];
    C = (int32_t)min((int64_t)a.ctas, W);
}

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads, 1) attn_prefill_kernel(const __grid_constant__ AttnArgs a) {
    using L = Lay<D>;
    constexpr int kBlks = D / 64, kRow = kKvRow<FMT, D>;
    // Trees over the 16-bit cache: probabilities in two bf16 terms, 16 bits, side by side in the columns of the scores
    // that they come from.  A choice of accuracy against time: outputs are 1.7e-3 off, as fp32 probabilities give them, and
    // 2.3e-3 with one term, which would take 404 us instead of 504 for the ragged contexts above and 177 instead of 205 for
    // the large trees.
    constexpr bool kTwo = kTree && FMT == KDA_KV_BF16;
    static_assert(NBAR * 8 <= 512, "barriers");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = ptx::smem_align1024(smem_raw);
    __shared__ uint32_t tmem_at;
    __shared__ int err_flag;
    __shared__ Walk start;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::bar);
    float *qs = reinterpret_cast<float *>(sm + L::qs);
    Job *jobs = reinterpret_cast<Job *>(sm + L::jobs);
    volatile uint32_t *bad = reinterpret_cast<uint32_t *>(sm + L::bad);
    volatile int *err = &err_flag;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

    if (tid == 0) {
        err_flag = 0;
        ptx::mbar_init(&bars[QFULL], kLoadWarps);
        ptx::mbar_init(&bars[QEMPTY], 1);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&bars[KFULL + i], FMT == KDA_KV_I8 ? kLoadWarps : 1);
            ptx::mbar_init(&bars[KEMPTY + i], 1);
            ptx::mbar_init(&bars[VFULL + i], kLoadWarps);
            ptx::mbar_init(&bars[VEMPTY + i], 1);
            ptx::mbar_init(&bars[VRAW + i], 1);
            ptx::mbar_init(&bars[SFULL + i], 1);
            ptx::mbar_init(&bars[PFULL + i], kSoftWarps / 2);
            ptx::mbar_init(&bars[OFULL + i], 1);
        }
        ptx::mbar_init(&bars[DRAIN], 1);
        for (int i = 0; i < kJobs; ++i) {
            ptx::mbar_init(&bars[JFULL + i], 1);
            ptx::mbar_init(&bars[JEMPTY + i], kSoftWarps + kLoadWarps + 1 + (FMT == KDA_KV_BF16 ? 1 : 0));
        }
    }
    ptx::fence_mbar_init();
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(&tmem_at, 512);
        ptx::tmem_relinquish();
        ptx::tc_fence_before();
    }
    ptx::grid_dep_wait();
    int64_t W;
    int32_t C;
    find_share(a, reinterpret_cast<int64_t *>(sm + L::plan), &start, W, C);
    ptx::tc_fence_after();
    const uint32_t tm = tmem_at;
    const int pt = a.kv.page_tokens;
    // Waits of a whole warp, of one thread; the next job, and being done with one.
    auto wait1 = [&](int b, uint32_t parity) { return wait_bar(&bars[b], parity, err); };
    auto wait = [&](int b, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait1(b, parity)) != 0; };
    auto wait_slow = [&](int b, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait_bar<64>(&bars[b], parity, err)) != 0; };
    auto job = [&](uint32_t n) -> const Job & { return jobs[n % kJobs]; };
    auto wait_job = [&](uint32_t n) { return wait(JFULL + n % kJobs, n / kJobs & 1); };
    auto done = [&](uint32_t n) { tcx::warp_arrive(&bars[JEMPTY + n % kJobs]); };

    // The roles run side by side out of one instruction cache, so their loops are kept small: rolled
    // where their register arrays allow it.
    if (warp < kSoftWarps) {
        // ====================================================== softmax and output
        const int half = warp / 8, side = warp / 4 % 2, row = half * kHalf + (warp % 4) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp % 4) * 32) << 16;
        const uint32_t tS = tm + lanes + half * 128 + side * 64;           // this thread's 64 scores
        const uint32_t tO = tm + lanes + 256 + half * 128 + side * (D / 2);   // and its half of the output
        float2 *pair = reinterpret_cast<float2 *>(sm + L::pair);
        auto meet = [&]() { tcx::named_bar(1 + half * 4 + warp % 4, 64); };    // the two warps of these rows
        auto together = [&](auto look) {                                       // the half's eight warps
            return wait_together<kSoftWarps / 2 * 32>(look, warp % 8 == 0, 9 + half);
        };
        auto wait_half = [&](int b, uint32_t parity) { return together([&]() { return wait1(b, parity); }); };
        uint32_t n_s = 0, n_item = 0, n_o = 0;   // units of this half, items so far, of this half: the barriers' parities
        int32_t pos = -1, p_lo = 0, p_hi = 0;   // positions of this row, of the warp's rows
        bool in = false, ok = true;
        float m = -INFINITY, big = -INFINITY, l = 0.f, f_row = 0.f;   // big: 8-bit, the reference with value scales
        auto lift = [&]() { return (big == -INFINITY ? 0.f : big - m) - kPBits; };
        auto next_job = [&](uint32_t n) { return wait1(JFULL + (n + 1) % kJobs, (n + 1) / kJobs & 1); };
        ok = wait_half(JFULL, 0);
        for (uint32_t n = 0; ok; ++n) {            // job n is there; the next is waited for beside its scores
            const Job &jb = job(n);
            const int32_t flags = jb.flags, nrows = jb.nrows, j0 = jb.j0;
            if (flags & kStop) break;
            if (half * kHalf >= nrows) {           // nothing in this half
                n_item += (flags & kEnd) != 0;
                done(n);
                ok = together([&]() { return next_job(n); });
                continue;
            }
            const int32_t at = jb.row0 + row;
            if (flags & kBegin) {
                in = row < nrows;
                pos = in ? jb.base + token_of(a, at) : -1;
                if (kTree) {
                    p_lo = jb.pmin, p_hi = jb.pmax;
                } else {
                    p_lo = __reduce_min_sync(0xFFFFFFFFu, in ? pos : INT32_MAX);
                    p_hi = __reduce_max_sync(0xFFFFFFFFu, pos);
                }
                m = big = -INFINITY, l = 0.f;
                float z[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) z[i] = 0.f;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) ptx::tmem_st16(tO + 16 * c, z);
            }
            ok = together([&]() { return next_job(n) && wait1(SFULL + half, n_s & 1); });
            if (!ok) break;
            ptx::tc_fence_after();
            if (flags & kBegin) f_row = qs[(n_item & 1) * kRows + row];
            // Of group c (16 tokens): the columns that this row sees, and whether every row of the warp sees
            // all of them or none any.  A warp's rows are few neighbouring tokens, so in a unit that a mask
            // cuts most groups still are the one or the other.
            auto seen = [&](int c) -> uint32_t {
                auto low = [](int32_t k) -> uint32_t { return k <= 0 ? 0u : k >= 16 ? 0xFFFFu : (1u << k) - 1u; };
                const int32_t b = j0 + 64 * side + 16 * c;
                if (kTree) {
                    if (!in) return 0;
                    const Draft r = draft_of(a, jb.tok0, jb.pmax + 1 - jb.base, jb.base, pos - jb.base);
                    uint32_t x = low(jb.base - b);
                    if (a.window > 0) x &= ~low(r.pos - a.window + 1 - b) | low(a.sinks - b);
                    const int32_t first = b - jb.base;        // of the group's tokens, among the drafts
                    if (first >= 0 && first < kTreeMost) x |= (uint32_t)(r.mask >> first) & 0xFFFFu;
                    if (first < 0 && first > -16) x |= (uint32_t)(r.mask << -first) & 0xFFFFu;
                    return x;
                }
                uint32_t x = low(pos + 1 - b);
                if (a.window > 0) x &= ~low(pos - a.window + 1 - b) | low(a.sinks - b);
                return x;
            };
            enum { kNone, kSome, kEvery };
            auto kind = [&](int c) -> int {
                const int32_t b = j0 + 64 * side + 16 * c;
                if (!(jb.live >> (4 * side + c) & 1u) || b > p_hi || (a.window > 0 && b + 15 <= p_lo - a.window && b >= a.sinks)) return kNone;
                return b + 15 <= p_lo && (a.window <= 0 || b > p_hi - a.window || b + 16 <= a.sinks) ? kEvery : kSome;
            };
            // 16 scores at a time, the next on their way from tensor memory
            auto groups = [&](auto step) {
                float x[2][16];
                tmem_ld16(tS, x[0]);
#pragma unroll 1
                for (int c = 0; c < 4; c += 2) {
                    wait_ld(x[0]);
                    tmem_ld16(tS + 16 * (c + 1), x[1]);
                    step(x[0], c);
                    wait_ld(x[1]);
                    if (c == 0) tmem_ld16(tS + 32, x[0]);
                    step(x[1], c + 1);
                }
            };
            // ---- the row's maximum, and (8-bit cache) that of its scores with log2 of their value scales added
            float top = -INFINITY, topv = -INFINITY;
            auto most = [&](auto all) {
                groups([&](const float (&x)[16], int c) {
                    const int k = decltype(all)::value ? kEvery : kind(c);
                    float gt = FMT == KDA_KV_I8 ? -INFINITY : top;
                    if (k == kEvery) {
#pragma unroll
                        for (int i = 0; i < 16; i += 2) gt = max3(gt, x[i], x[i + 1]);
                    } else if (k == kSome) {
                        const uint32_t see = seen(c);
#pragma unroll
                        for (int i = 0; i < 16; ++i) gt = fmaxf(gt, see & 1u << i ? x[i] : -INFINITY);
                    }
                    if constexpr (FMT == KDA_KV_I8) {
                        if (k != kNone) {
                            gt *= f_row * jb.ks[4 * side + c];   // factors are >= 0
                            top = fmaxf(top, gt);
                            topv = fmaxf(topv, gt + jb.lg[4 * side + c]);
                        }
                    } else {
                        top = gt;
                    }
                });
            };
            if (flags & kWhole) most(std::true_type{});
            else most(std::false_type{});
            if (FMT == KDA_KV_BF16 && top != -INFINITY) top *= f_row;
            {
                float2 *mine = pair + ((n_s & 1) * 2 + side) * kRows, *other = pair + ((n_s & 1) * 2 + (side ^ 1)) * kRows;
                mine[row] = make_float2(top, topv);
                meet();
                const float2 z = other[row];
                top = fmaxf(top, z.x), topv = fmaxf(topv, z.y);
            }
            // ---- the row's references, which lag behind its maxima (also from -infinity)
            float grown = 1.f;            // what O is to be multiplied by
            if (top > m + kGrow) {
                const float mn = FMT == KDA_KV_I8 ? ceilf(top) : top, f = ex2(m - mn);
                if (FMT == KDA_KV_BF16) grown = f;
                l *= f;
                m = mn;
            }
            if (FMT == KDA_KV_I8 && topv > big + kGrow) {
                const float bn = ceilf(topv);
                grown = ex2(big - bn);
                big = bn;
            }
            const float ms = m == -INFINITY ? 0.f : m;
            // ---- tokens whose values were taken out of the product (16-bit cache)
            bool odd = false;
            if (FMT == KDA_KV_BF16 && !(flags & kWhole)) {
                ok = wait_half(VFULL + (n & 1), n >> 1 & 1);
                if (!ok) break;
                const volatile uint32_t *out = bad + (n & 1) * 4;
                odd = (out[0] | out[1] | out[2] | out[3]) != 0;
            }
            // ---- O to the new references
            if (__any_sync(0xFFFFFFFFu, grown != 1.f || odd)) {
                // the products of the last unit are done, for the scores of this one came after them
                if (flags & kBegin) ptx::tmem_wait_st();
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float o[16];
                    tmem_ld16(tO + 16 * c, o);
                    wait_ld(o);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] *= grown;
                    if (FMT == KDA_KV_BF16 && odd) {
#pragma unroll 1
                        for (int j = 0; j < kUnit; ++j) {
                            if (!(bad[(n & 1) * 4 + (j >> 5)] >> (j & 31) & 1u)) continue;   // the same for all rows
                            const float x = tmem_ld1(tS - side * 64 + j);
                            const bool see = kTree ? in && draft_sees(a, draft_of(a, jb.tok0, jb.pmax + 1 - jb.base, jb.base, pos - jb.base), jb.base, j0 + j)
                                                   : sees(a, pos, j0 + j);
                            if (see) {
                                const float pj = ex2(x * f_row - ms);
                                const uint8_t *line = a.kv.base + jb.rec[j >> 4] + pt * kRow;
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const uint4 v = *reinterpret_cast<const uint4 *>(
                                        line + kv_tile_off<kRow>(pt, jb.slot[j >> 4] + (j & 15), side * D + 32 * c + 16 * i));
                                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                    for (int y = 0; y < 4; ++y) {
                                        const float2 z = tcx::bf2_to_f2(w[y]);
                                        o[8 * i + 2 * y] += pj * z.x;
                                        o[8 * i + 2 * y + 1] += pj * z.y;
                                    }
                                }
                            }
                            __syncwarp();
                        }
                    }
                    ptx::tmem_st16(tO + 16 * c, o);
                }
            }
            if (FMT == KDA_KV_BF16 && odd) meet();   // the other warp is done with these scores too
            // ---- the probabilities, over the scores that they come from: a group's 8 columns lie in
            // what an earlier group has read
            const float lifted = FMT == KDA_KV_I8 ? lift() : 0.f;
            auto weigh = [&](auto all) {
                groups([&](const float (&x)[16], int c) {
                    const int k = decltype(all)::value ? kEvery : kind(c);
                    float p[8], low[8];
                    if (k == kNone) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) p[i] = low[i] = 0.f;
                    } else {
                        const uint32_t see = k == kEvery ? ~0u : seen(c);
                        float fk = f_row, bias = -ms, back = 1.f;
                        if (FMT == KDA_KV_I8) {
                            // (a scale of 0 gives a product of 0 in fp16, and still its share of the sum)
                            const float e = fmaxf(jb.lg[4 * side + c] - lifted, -94.f);
                            fk *= jb.ks[4 * side + c];
                            bias += e;
                            back = ex2(-e);
                        }
                        const float2 ff = make_float2(fk, fk), bb = make_float2(bias, bias);
                        float2 part = make_float2(0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float2 y = tcx::ffma2(make_float2(x[2 * i], x[2 * i + 1]), ff, bb);
                            y.x = ex2(y.x), y.y = ex2(y.y);
                            if (k == kSome) {
                                y.x = see & 1u << 2 * i ? y.x : 0.f;
                                y.y = see & 2u << 2 * i ? y.y : 0.f;
                            }
                            part = tcx::fadd2(part, y);
                            p[i] = __uint_as_float(pack2<FMT>(y.x, y.y));
                            if (kTwo) {
                                const float2 z = tcx::bf2_to_f2(__float_as_uint(p[i]));
                                low[i] = __uint_as_float(pack2<FMT>(y.x - z.x, y.y - z.y));
                            }
                        }
                        l += (part.x + part.y) * back;
                        if (FMT == KDA_KV_I8 && (jb.nans >> (4 * side + c) & 1u)) {   // fp16 NaN where the row sees it
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                p[i] = __uint_as_float((see & 1u << 2 * i ? 0x7E00u : 0u) | (see & 2u << 2 * i ? 0x7E000000u : 0u));
                        }
                    }
                    ptx::tmem_st8(tS + (kTwo ? 16 : 8) * c, p);
                    if (kTwo) ptx::tmem_st8(tS + 16 * c + 8, low);
                });
            };
            if (flags & kWhole) weigh(std::true_type{});
            else weigh(std::false_type{});
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            tcx::warp_arrive(&bars[PFULL + half]);
            ++n_s;
            if (flags & kEnd) {
                // ---- the item's output, or this CTA's part of it, added to an earlier piece's
                const bool all = (flags & kStarts) && (flags & kEnds) && !(flags & kMore);
                float *part = a.part + ((int64_t)(blockIdx.x * 2 + (flags & kStarts ? 1 : 0)) * kRows + row) * kPartRow<D>;
                float unscale = FMT == KDA_KV_I8 ? exp2f(lift()) : 1.f, again = 0.f, l_was = 0.f;
                if (flags & kAgain) {
                    const float was = part[D], both = fmaxf(m, was), ref = both == -INFINITY ? 0.f : both;
                    const float f = ex2(m - ref);
                    again = ex2(was - ref);
                    l_was = part[D + 1] * again;
                    unscale *= f, l *= f;
                    m = both;
                }
                {
                    float2 *mine = pair + ((n_s & 1) * 2 + side) * kRows, *other = pair + ((n_s & 1) * 2 + (side ^ 1)) * kRows;
                    mine[row].x = l;
                    meet();
                    l += other[row].x + l_was;
                    meet();              // the next item's first maxima go to the same place
                }
                ok = wait_half(OFULL + half, n_o++ & 1);
                if (!ok) break;
                ptx::tc_fence_after();
                const int32_t tok = token_of(a, at);
                const int64_t orow = ((int64_t)jb.tok0 + tok) * a.Hq + jb.head * a.G + at - tok * a.G;
                const float norm = !all ? 1.f : l == 0.f ? 0.f : 1.f / l, f = unscale * norm;
                again *= norm;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float o[1][16];
                    tmem_ld16(tO + 16 * c, o[0]);
                    wait_ld(o[0]);
#pragma unroll
                    for (int y = 0; y < 1; ++y) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[y][i] = all && l == 0.f ? 0.f : o[y][i] * f;
                        const int col = side * (D / 2) + 16 * (c + y);
                        if (flags & kAgain)
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[y][i] += part[col + i] * again;
                        if (in && all) {
                            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + orow * D + col);
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                dst[i] = make_uint4(tcx::f2_to_bf2(o[y][8 * i], o[y][8 * i + 1]), tcx::f2_to_bf2(o[y][8 * i + 2], o[y][8 * i + 3]),
                                                    tcx::f2_to_bf2(o[y][8 * i + 4], o[y][8 * i + 5]), tcx::f2_to_bf2(o[y][8 * i + 6], o[y][8 * i + 7]));
                        } else if (in) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                reinterpret_cast<float4 *>(part + col)[i] =
                                    make_float4(o[y][4 * i], o[y][4 * i + 1], o[y][4 * i + 2], o[y][4 * i + 3]);
                        }
                    }
                    __syncwarp();
                }
                ptx::tc_fence_before();
                if (in && side == 0) {
                    if (!all) part[D] = m, part[D + 1] = l;
                    else if (a.lse) a.lse[orow] = lse_of(m, l);
                }
                if (tid == 0 && (flags & kStarts) && !(flags & kEnds)) {
                    AttnSplit sp{};
                    sp.last_cta = jb.last_cta;
                    sp.row_tok = jb.tok0;
                    sp.head = jb.head;
                    sp.row0 = jb.row0;
                    sp.nrows = nrows;
                    a.split[blockIdx.x] = sp;
                }
                ++n_item;
            }
            done(n);
        }
        if (!ok && lane == 0) flag_status(a.kv.status, KDA_DEV_TIMEOUT);
    } else if (warp < kSoftWarps + kLoadWarps) {
        // ====================================================== queries, and keys and values
        const int lw = warp - kSoftWarps, lt = tid - kSoftWarps * 32;
        auto together = [&](auto look) {                          // the eight warps
            return wait_together<kLoadWarps * 32>(look, lw == 0, 11);
        };
        auto wait_all = [&](int b, uint32_t parity) { return together([&]() { return wait1(b, parity); }); };
        auto with_next = [&](int b, uint32_t parity, uint32_t n) {   // and the job behind job n
            return together([&]() { return wait1(b, parity) && wait1(JFULL + (n + 1) % kJobs, (n + 1) / kJobs & 1); });
        };
        uint32_t n_item = 0;
        // 8-bit: the units' codes are read one unit ahead into registers.  A warp takes 16 tokens;
        // eight lanes take four units of token r and of token r ^ 5, which keeps both their reads
        // and their writes in different banks.
        constexpr int kRegs = kRow / 32;
        constexpr int kQuads = kRow / 64;                         // groups of four 16-byte units a row
        uint4 kc[kRegs] = {}, vc[kRegs] = {};
        const int r8 = (lane >> 3) ^ ((lane >> 2 & 1) * 5), ul = lane & 3;
        // A lane's places: its units' in a page's lines (rows 8 apart lie 1024 bytes apart, the upper
        // four units of a line opposite the lower), and those of their two halves in a tile.
        const uint32_t from = kv_tile_off<kRow>(pt, r8, 16 * ul), from4 = from ^ 64u;
        const uint32_t to = (16 * lw + r8) * 128 + (((2 * ul) ^ (r8 & 7)) << 4);
        auto fetch = [&](const Job &jb, bool values, uint4 (&c)[kRegs]) {
            const uint8_t *src = a.kv.base + (jb.rec[lw] + (values ? pt * kRow : 0) + jb.slot[lw] * (kRow < 128 ? kRow : 128));
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int x = 0; x < kQuads; ++x)
                    c[i * kQuads + x] =
                        __ldg(reinterpret_cast<const uint4 *>(src + (x ? from4 : from) + i * 8 * (kRow < 128 ? kRow : 128)));
        };
        auto put = [&](const uint4 (&c)[kRegs], uint8_t *tile) {
            uint8_t *lo_at = tile + to, *hi_at = tile + (to ^ 16u);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int x = 0; x < kQuads; ++x) {
                    uint4 lo, hi;
                    codes_to_half(c[i * kQuads + x], lo, hi);
                    *reinterpret_cast<uint4 *>(lo_at + x * L::blk + i * 1024) = lo;
                    *reinterpret_cast<uint4 *>(hi_at + x * L::blk + i * 1024) = hi;
                }
        };
        // An item's queries: a thread takes 16 columns of every kRpp-th row, kBatch rows' loads under way
        // at a time; the first batch is read while the last item's queries are still in use.
        auto queries = [&](const Job &jb) -> bool {
            constexpr int kTpr = D / 16, kRpp = kLoadWarps * 32 / kTpr, kBatch = FMT == KDA_KV_I8 ? 2 : 4;
            const float sign = a.scale < 0.f ? -1.f : 1.f;
            const int nrows = jb.nrows, rows = nrows > kHalf ? kRows : kHalf, c = lt % kTpr;
            uint4 x[kBatch][2];
#pragma unroll 1
            for (int r0 = lt / kTpr; r0 < rows; r0 += kBatch * kRpp) {
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int r = r0 + i * kRpp, at = jb.row0 + r, tok = token_of(a, at);
                    x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
                    if (r < nrows) {
                        const uint4 *src = reinterpret_cast<const uint4 *>(
                            static_cast<const __nv_bfloat16 *>(a.q) + ((int64_t)jb.tok0 + tok) * a.q_stride +
                            (int64_t)(jb.head * a.G + at - tok * a.G) * D + 16 * c);
                        x[i][0] = src[0], x[i][1] = src[1];
                    }
                }
                if (r0 == lt / kTpr && !wait_all(QEMPTY, (n_item & 1) ^ 1)) return false;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int r = r0 + i * kRpp;
                    if (r >= rows) break;
                    float f = a.scale * sign * kLog2e;
                    uint32_t y[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w, x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
                    if (sign < 0.f)
#pragma unroll
                        for (int j = 0; j < 8; ++j) y[j] ^= 0x80008000u;
                    if (FMT == KDA_KV_I8) {
                        // a power of two that brings the row's largest magnitude to [2^10, 2^11)
                        float e[16], top = 0.f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float2 v = tcx::bf2_to_f2(y[j]);
                            e[2 * j] = v.x, e[2 * j + 1] = v.y;
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j) top = fmaxf(top, fabsf(e[j]));
#pragma unroll
                        for (int j = 1; j < kTpr; j <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, j));
                        const int b = (int)(__float_as_uint(top) >> 23);
                        const int shift = b == 0 || b == 255 ? 0 : min(max(137 - b, -120), 120);
                        const float up = __uint_as_float((uint32_t)(127 + shift) << 23);
                        f *= __uint_as_float((uint32_t)(127 - shift) << 23);
#pragma unroll
                        for (int j = 0; j < 8; ++j) y[j] = pack2<FMT>(e[2 * j] * up, e[2 * j + 1] * up);
                    }
                    uint8_t *dst = sm + L::q + (r / kHalf) * L::half_q + (c >> 2) * (kHalf * 128);
                    const int rr = r % kHalf;
                    *reinterpret_cast<uint4 *>(dst + ptx::sw128_off(rr, 32 * (c & 3))) = make_uint4(y[0], y[1], y[2], y[3]);
                    *reinterpret_cast<uint4 *>(dst + ptx::sw128_off(rr, 32 * (c & 3) + 16)) = make_uint4(y[4], y[5], y[6], y[7]);
                    if (c == 0) qs[(n_item & 1) * kRows + r] = f;
                }
            }
            ptx::fence_proxy_async_smem();
            tcx::warp_arrive(&bars[QFULL]);
            return true;
        };
        bool ok = wait_all(JFULL, 0), stop = ok && (job(0).flags & kStop);
        if (kTree && FMT == KDA_KV_I8 && ok && !stop) {
            fetch(job(0), false, kc);
            fetch(job(0), true, vc);
        } else if (FMT == KDA_KV_I8 && ok && !stop) {
#pragma unroll 1
            for (int v = 0; v < 2; ++v) {
#pragma unroll
                for (int i = 0; i < kRegs; ++i) kc[i] = vc[i];
                fetch(job(0), v, vc);
            }
        }
        for (uint32_t n = 0; ok && !stop; ++n) {
            const Job &jb = job(n);
            const int st = n & 1;
            const uint32_t par = (n >> 1 & 1) ^ 1;
            if (jb.flags & kBegin) {
                ok = queries(jb);
                if (!ok) break;
                ++n_item;
            }
            if (kTree && FMT == KDA_KV_I8) {
                // Few rows: keys and values in registers of their own.  Moving one up, as below, waits for it to land,
                // which the time of a unit of a prompt hides.
                ok = with_next(KEMPTY + st, par, n);
                if (!ok) break;
                put(kc, sm + L::k + st * L::tile);
                ptx::fence_proxy_async_smem();
                tcx::warp_arrive(&bars[KFULL + st]);
                stop = job(n + 1).flags & kStop;
                if (!stop) fetch(job(n + 1), false, kc);
                ok = wait_all(VEMPTY + st, par);
                if (!ok) break;
                put(vc, sm + L::v + st * L::tile);
                ptx::fence_proxy_async_smem();
                tcx::warp_arrive(&bars[VFULL + st]);
                if (!stop) fetch(job(n + 1), true, vc);
            } else if (FMT == KDA_KV_I8) {
                // keys, then values: kc goes out, vc moves up, the same of the next unit is fetched
#pragma unroll 1
                for (int v = 0; v < 2; ++v) {
                    ok = v ? wait_all(VEMPTY + st, par) : with_next(KEMPTY + st, par, n);
                    if (!ok) break;
                    put(kc, sm + (v ? L::v : L::k) + st * L::tile);
                    ptx::fence_proxy_async_smem();
                    tcx::warp_arrive(&bars[(v ? VFULL : KFULL) + st]);
                    if (v == 0) stop = job(n + 1).flags & kStop;
#pragma unroll
                    for (int i = 0; i < kRegs; ++i) kc[i] = vc[i];
                    if (!stop) fetch(job(n + 1), v, vc);
                }
                if (!ok) break;
            } else {
                // values that not every row sees: a token that no row sees is cleared (0 times what a
                // stale slot holds need not be 0), and one with an infinity or a NaN is taken out and
                // left to the rows that see it
                ok = with_next(VRAW + st, n >> 1 & 1, n);
                if (!ok) break;
                stop = job(n + 1).flags & kStop;
                if (!(jb.flags & kWhole) && lt < kUnit) {
                    uint8_t *line = sm + L::v + st * L::tile + lt * 128;
                    const int32_t j = jb.j0 + lt;
                    const bool any = (jb.live >> (lt >> 4) & 1u) && j <= jb.pmax &&
                                     (a.window <= 0 || j > jb.pmin - a.window || j < a.sinks);
                    bool strange = false;
                    if (any) {
#pragma unroll 1
                        for (int b = 0; b < kBlks; ++b)
#pragma unroll 2
                            for (int i = 0; i < 8; ++i) {
                                const uint4 x = *reinterpret_cast<const uint4 *>(line + b * L::blk + ((i ^ (lt & 7)) << 4));
                                for (uint32_t y : {x.x, x.y, x.z, x.w})
                                    strange |= (y & 0x7F80u) == 0x7F80u || (y & 0x7F800000u) == 0x7F800000u;
                            }
                    }
                    if (!any || strange)
#pragma unroll 1
                        for (int b = 0; b < kBlks; ++b)
#pragma unroll 2
                            for (int i = 0; i < 8; ++i)
                                *reinterpret_cast<uint4 *>(line + b * L::blk + ((i ^ (lt & 7)) << 4)) = make_uint4(0, 0, 0, 0);
                    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, strange);
                    if (lane == 0) bad[st * 4 + lw] = mask;
                    ptx::fence_proxy_async_smem();
                }
                tcx::warp_arrive(&bars[VFULL + st]);
            }
            done(n);
        }
    } else {
        if (warp == kMmaWarp) {
            // ================================================== products
            // The whole warp walks along and one lane issues: addresses then stay in uniform registers,
            // and a product takes the 64 cycles that the pipe needs (about 100 from a lone lane).
            const uint32_t sb = ptx::smem_u32(sm);
            const uint32_t tu = __shfl_sync(0xFFFFFFFFu, tm, 0);
            uint32_t n_item = 0, n_p[2] = {0, 0};
            auto scores = [&](int half, int st) {                     // one lane
                const uint64_t qd = ptx::sdesc_sw128(sb + L::q + half * L::half_q, 16, 1024);
                const uint64_t kd = ptx::sdesc_sw128(sb + L::k + st * L::tile, 16, 1024);
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint32_t off = ((s >> 2) * L::blk + (s & 3) * 32) >> 4;
                    ptx::mma_bf16(tu + half * 128, qd + off, kd + off, idesc<FMT>(128, 128, 0), s > 0 ? 1u : 0u);
                }
                ptx::mma_commit(&bars[SFULL + half]);
            };
            auto outputs = [&](int half, int st) {
                const uint64_t vd = ptx::sdesc_sw128(sb + L::v + st * L::tile, L::blk, 1024);
#pragma unroll
                for (int s = 0; s < kUnit / 16; ++s) {   // probabilities: 32 columns (two terms: 64) in each half of the scores
                    const uint32_t from = tu + half * 128 + (s >> 2) * 64 + (s & 3) * (kTwo ? 16 : 8);
                    if (kTwo) ptx::mma_bf16_ta(tu + 256 + half * 128, from + 8, vd + (s * 2048 >> 4), idesc<FMT>(128, D, 1), 1u);
                    ptx::mma_bf16_ta(tu + 256 + half * 128, from, vd + (s * 2048 >> 4), idesc<FMT>(128, D, 1), 1u);
                }
            };
            // Wait for up to four barriers at once, lane i for the i-th: beside the other warps' work a wait
            // costs this one 250 cycles even where the barrier's phase is over, four of them a quarter of a unit.
            auto wait_set = [&](int count, int b0, uint32_t p0, int b1, uint32_t p1, int b2, uint32_t p2, int b3, uint32_t p3) {
                const int b = lane == 0 ? b0 : lane == 1 ? b1 : lane == 2 ? b2 : b3;
                const uint32_t par = (lane == 0 ? p0 : lane == 1 ? p1 : lane == 2 ? p2 : p3) & 1;
                bool there = lane >= count;
#pragma unroll 1
                for (uint32_t i = 0; i < ptx::kSpinLimit; ++i) {
                    if (!there) there = ptx::mbar_try_wait(&bars[b], par);
                    if (__all_sync(0xFFFFFFFFu, there)) return true;
                    if (__any_sync(0xFFFFFFFFu, *err != 0)) return false;
                }
                *err = 1;
                return false;
            };
            // a half's outputs of unit n, and its scores of the next, whose completion says both
            auto issue = [&](uint32_t n, int h, bool more, bool unit_done, bool item_done) {
                const int st = n & 1, nx = st ^ 1;
                ptx::tc_fence_after();
                if (elect()) {
                    outputs(h, st);
                    if (more) scores(h, nx);
                    else ptx::mma_commit(&bars[OFULL + h]);
                    if (unit_done) {
                        ptx::mma_commit(&bars[VEMPTY + st]);
                        if (more) ptx::mma_commit(&bars[KEMPTY + nx]);
                        if (item_done) ptx::mma_commit(&bars[QEMPTY]);
                    }
                }
                __syncwarp();
            };
            bool ok = wait_job(0);
            int32_t flags = ok ? job(0).flags : kStop, nrows = job(0).nrows;
            for (uint32_t n = 0; !(flags & kStop); ++n) {
                const int st = n & 1, nx = st ^ 1;
                const bool two = nrows > kHalf, more = !(flags & kEnd);
                // the scores of an item's first unit; those of the next follow each half's outputs
                if (flags & kBegin) {
                    if (!wait_set(2, QFULL, n_item, KFULL + st, n >> 1, 0, 0, 0, 0)) break;
                    ptx::tc_fence_after();
                    if (elect()) {
                        scores(0, st);
                        if (two) scores(1, st);
                        ptx::mma_commit(&bars[KEMPTY + st]);
                        if (flags & kEnd) ptx::mma_commit(&bars[QEMPTY]);
                    }
                    __syncwarp();
                    ++n_item;
                }
                if (!wait_set(more ? 4 : 3, PFULL, n_p[0]++, VFULL + st, n >> 1, JFULL + (n + 1) % kJobs, (n + 1) / kJobs,
                              KFULL + nx, (n + 1) >> 1))
                    break;
                // with the scores of an item's last unit done its queries may go
                const int32_t next_flags = job(n + 1).flags, next_nrows = job(n + 1).nrows;
                const bool last = more && (next_flags & kEnd);
                issue(n, 0, more, !two, last);
                if (two) {
                    if (!wait(PFULL + 1, n_p[1]++ & 1)) break;
                    issue(n, 1, more, true, last);
                }
                done(n);
                flags = next_flags, nrows = next_nrows;
            }
            if (elect()) ptx::mma_commit(&bars[DRAIN]);
            __syncwarp();
            wait_bar(&bars[DRAIN], 0, nullptr);
        } else if (FMT == KDA_KV_BF16 && warp == kCopyWarp) {
            // ================================================== copies (16-bit cache)
            uint32_t n_k = 0, n_v = 0;                            // tiles asked for
            for (uint32_t n = 0; wait_job(n); ++n) {
                const Job &jb = job(n);
                if (jb.flags & kStop) break;
                const int st = n & 1;
                const uint32_t par = (n >> 1 & 1) ^ 1, bytes = __popc(jb.live) * 16 * kRow;
                const bool there = lane < 8 && (jb.live >> lane & 1u);
                const uint8_t *src = there ? a.kv.base + jb.rec[lane] + jb.slot[lane] * 128 : nullptr;
                done(n);
                auto copy = [&](int bar, uint8_t *dst, const uint8_t *from) {
                    if (lane == 0) ptx::mbar_arrive_expect_tx(&bars[bar], bytes);
                    __syncwarp();
                    if (there)
#pragma unroll
                        for (int b = 0; b < kBlks; ++b)
                            ptx::bulk_load(dst + b * L::blk + lane * 2048, from + b * pt * 128, 2048, &bars[bar]);
                };
                if (!wait_slow(KEMPTY + st, par)) break;
                copy(KFULL + st, sm + L::k + st * L::tile, src);
                ++n_k;
                if (!wait_slow(VEMPTY + st, par)) break;
                copy(VRAW + st, sm + L::v + st * L::tile, src + pt * kRow);
                ++n_v;
            }
            // the last copies land before the block ends, whatever became of their readers
            __syncwarp();
            for (uint32_t i = n_k > 2 ? n_k - 2 : 0; i < n_k; ++i) wait_bar(&bars[KFULL + (i & 1)], i >> 1 & 1, nullptr);
            for (uint32_t i = n_v > 2 ? n_v - 2 : 0; i < n_v; ++i) wait_bar(&bars[VRAW + (i & 1)], i >> 1 & 1, nullptr);
        } else if (warp == kWalkWarp) {
            // ================================================== the list of units
            // Units go in batches of up to four of one item: lane i has group i % 8 of the batch's unit i / 8.
            // A batch's pages are read two batches ahead and its scales one ahead, so that the walk waits for
            // memory once in four units and not twice in each.
            struct Batch {
                Walk w;               // at its first unit
                int32_t n, page, slot;
                bool want;
            };
            auto look = [&](const Walk &x) {
                Batch r;
                r.w = x;
                r.n = x.left > 0 ? (int32_t)min((int64_t)min(4, x.t.units - x.u), x.left) : 0;
                r.page = r.slot = 0;
                r.want = false;
                if (r.n > 0) {
                    const int32_t j = unit_token<kUnit>(x.t, x.u + lane / 8) + lane % 8 * 16, b = j / pt;
                    r.slot = j - b * pt;
                    r.want = lane / 8 < r.n && any_sees(a, x.t, j, 16);
                    if (r.want) r.page = __ldg(a.kv.table + (int64_t)x.t.s * a.kv.max_pages + b);
                }
                return r;
            };
            auto after = [&](const Batch &x) {
                Walk w = x.w;
                w.left -= x.n;
                w.u += x.n;
                if (w.left > 0 && w.u == w.t.units) {
                    w.left -= kItem;
                    if (w.left > 0) next_item<kRows, kUnit>(a, w);
                }
                return w;
            };
            auto record = [&](const Batch &x) { return x.want ? kv_record(a.kv, x.page, x.w.h) : nullptr; };
            auto scales = [&](const uint8_t *rec) {
                return FMT == KDA_KV_I8 && rec ? __ldg(reinterpret_cast<const float2 *>(rec + 2 * pt * kRow)) : make_float2(0.f, 0.f);
            };
            if (lane == 0) a.split[blockIdx.x].last_cta = -1;
            const int64_t end = C > 0 ? (int64_t)(blockIdx.x + 1) * W / C : 0;
            Batch now = look(start), next = look(after(now));
            const uint8_t *rec = record(now);
            float2 sc = scales(rec);
            int32_t u_first = start.u;
            uint32_t n = 0;
            bool ok = true;
            while (ok && now.n > 0) {
                const uint8_t *next_rec = record(next);
                const float2 next_sc = scales(next_rec);
                const Batch then = look(after(next));
                const Tile &t = now.w.t;
                const int32_t k = lane / 8, u = now.w.u + k, j0 = unit_token<kUnit>(t, u);
                const int64_t left = now.w.left - k;
                const uint32_t live = __ballot_sync(0xFFFFFFFFu, rec != nullptr) >> (8 * k) & 0xFFu;
                const float x = fabsf(sc.y);
                const uint32_t nans = __ballot_sync(0xFFFFFFFFu, !(x < INFINITY)) >> (8 * k) & 0xFFu;
                for (int i = 0; ok && i < now.n; ++i) ok = wait_slow(JEMPTY + (n + i) % kJobs, ((n + i) / kJobs & 1) ^ 1);
                if (!ok) break;
                if (k < now.n) {
                    Job &jb = jobs[(n + k) % kJobs];
                    const int i = lane % 8;
                    jb.slot[i] = now.slot;
                    jb.rec[i] = rec ? rec - a.kv.base : 0;
                    if (FMT == KDA_KV_I8) {
                        // a value scale that is no number makes the probabilities NaN where they are seen; the sums,
                        // which have no part in the values, stay
                        jb.ks[i] = fabsf(sc.x) < INFINITY ? fabsf(sc.x) : NAN;   // an infinity reads as NaN whatever the codes
                        jb.lg[i] = x > 0.f && x < INFINITY ? fmaxf(log2f(x), -100.f) : -INFINITY;
                    }
                    if (i == 0) {
                        const bool ends = left >= t.units - u;   // the item's last unit is in this share
                        jb.j0 = j0;
                        jb.flags = piece_flags(u - u_first, u + 1 == t.units || left == 1) |
                                   (all_see(a, t, j0, kUnit) && live == 0xFFu ? kWhole : 0) | (u_first == 0 ? kStarts : 0) |
                                   (ends ? kEnds : 0);
                        jb.base = t.q.len - t.q.n;
                        jb.row0 = t.row0, jb.nrows = t.nrows, jb.tok0 = t.q.tok0, jb.head = now.w.h;
                        jb.live = live;
                        jb.last_cta = ends ? (int32_t)blockIdx.x : cta_of(end - left + (t.units - 1 - u), W, C);
                        jb.pmin = t.pmin, jb.pmax = t.pmax;
                        jb.nans = nans;
                    }
                }
                if (kTree && rec && k < now.n) {
                    // Few rows leave little time a unit, and a unit's copies are under way for one unit's time alone: what
                    // a job handed on needs is asked into L2, up to eight units before it is copied.
                    constexpr int kLine = kRow < 128 ? kRow : 128;
#pragma unroll
                    for (int v = 0; v < 2; ++v)
#pragma unroll
                        for (int y = 0; y < kRow / kLine; ++y)
                            ptx::prefetch_bulk(rec + v * pt * kRow + y * pt * kLine + now.slot * kLine, 16 * kLine);
                }
                __syncwarp();
                if (lane % 8 == 0 && k < now.n) ptx::mbar_arrive(&bars[JFULL + (n + k) % kJobs]);
                n += now.n;
                if (next.w.u == 0) u_first = 0;
                now = next, next = then;
                rec = next_rec, sc = next_sc;
            }
            if (ok && wait_slow(JEMPTY + n % kJobs, (n / kJobs & 1) ^ 1) && lane == 0) {
                jobs[n % kJobs].flags = kStop;
                ptx::mbar_arrive(&bars[JFULL + n % kJobs]);
            }
        }
    }
    __syncthreads();
    if (warp == kMmaWarp) ptx::tmem_dealloc(tm, 512);
}

template <int FMT, int D>
cudaError_t run(const AttnArgs &a, cudaStream_t st) {
    auto kern = attn_prefill_kernel<FMT, D>;
    constexpr int smem = Lay<D>::total + 1024;
    static_assert(smem <= 226 * 1024, "shared memory");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<a.ctas, kThreads, smem, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.ctas, 16);
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<D, kRows>, a);
}

}  // namespace

#ifdef KDA_ATTN_TREE
cudaError_t launch_attn_tree_prefill(const AttnArgs &a, cudaStream_t s) {
#else
cudaError_t launch_attn_prefill(const AttnArgs &a, cudaStream_t s) {
#endif
    if (a.kv.d == 128) return a.kv.fmt == KDA_KV_I8 ? run<KDA_KV_I8, 128>(a, s) : run<KDA_KV_BF16, 128>(a, s);
    return a.kv.fmt == KDA_KV_I8 ? run<KDA_KV_I8, 64>(a, s) : run<KDA_KV_BF16, 64>(a, s);
}

}  // namespace kda
