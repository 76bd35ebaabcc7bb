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
// One CTA of 14 warps an SM:
//   warps 0-3, 4-7   softmax of a half, a thread a row: scores from tensor memory, probabilities
//                    back into it, at the end the output.  O is only rescaled when a row's maximum
//                    has grown by more than 2^8 (fp16 and bf16 have the room).
//   warps 8-11       queries into shared memory; 8-bit cache: codes from global memory through
//                    registers to fp16 tiles (a page's bytes never lie in shared memory);
//                    16-bit cache: a look at values that not every row sees
//   warp 12          issues the products
//   warp 13          16-bit cache: bulk copies of pages, whose lines already lie as the matrix
//                    unit's 128-byte swizzle wants them
//
// 8-bit cache: as in the register kernel codes are exact in fp16 and query rows scaled by a power
// of two; the key scale of each 16 tokens multiplies f, the value scale goes into the exponent:
// p' = 2^(f S - m + log2(vs / ref 2^6)), and a group's sum of p' divided by that factor is its sum
// of p.  ref is the largest value scale so far, to within a factor of two.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "tc_common.cuh"

namespace kda {
namespace {

using namespace attn;

constexpr int kRows = kAttnPrefillRows, kHalf = 128, kUnit = 128;
constexpr int kSoftWarps = 8, kLoadWarps = 4, kMmaWarp = 12, kThreads = 14 * 32;
constexpr float kGrow = 8.f;            // bits that a row's maximum may grow before O is rescaled
constexpr float kPBits = 6.f;           // 8-bit: bits that a probability is scaled up in fp16
constexpr float kMinRef = 0x1p-100f;
constexpr int kRing = 4;                // units whose scales and live groups are kept

template <int D>
struct Lay {
    static constexpr int half_q = kHalf * D * 2, tile = kUnit * D * 2, blk = kUnit * 128;   // 64-column blocks
    static constexpr int q = 0, k = 2 * half_q, v = k + 2 * tile, misc = v + 2 * tile;
    static constexpr int qs = misc;                        // [2][256] row factors
    static constexpr int ks = qs + 2 * kRows * 4;          // [kRing][8] key scales, then value scales
    static constexpr int vs = ks + kRing * 8 * 4;
    static constexpr int live = vs + kRing * 8 * 4;        // [kRing] groups of 16 tokens that are there
    static constexpr int bad = live + kRing * 4;           // [2][4] tokens taken out of a value tile
    static constexpr int plan = bad + 2 * 16;              // the split's scratch
    static constexpr int bar = plan + 4096 + 64;
    static constexpr int total = bar + 256;
};

enum Bar { QFULL, QEMPTY, KFULL, KEMPTY = KFULL + 2, VFULL = KEMPTY + 2, VEMPTY = VFULL + 2, VRAW = VEMPTY + 2,
           SFULL = VRAW + 2, PFULL = SFULL + 2, OFULL = PFULL + 2, DRAIN = OFULL + 2, NBAR };

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

__device__ __forceinline__ float tmem_ld1(uint32_t addr) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(addr) : "memory");
    return __uint_as_float(r);
}
__device__ __forceinline__ void tmem_st16u(uint32_t addr, const uint32_t (&v)[16]) {
    float f[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(v[i]);
    ptx::tmem_st16(addr, f);
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

// A CTA's place in the list of units, walked by every role on its own.
struct Walk {
    Tile t;
    int32_t h, u;
    int64_t left;
};

__device__ __forceinline__ KvSeq seq_of(const AttnArgs &a, int s) {
    return kv_seq(a.cu_q, a.kv_len, s, a.T_tot, a.max_q, a.kv);
}

__device__ __forceinline__ void next_item(const AttnArgs &a, Walk &w) {
    w.u = 0;
    if (++w.h < a.kv.Hkv) return;
    w.h = 0;
    if (w.t.rt + 1 < w.t.tiles) {
        w.t = make_tile<kRows, kUnit>(a, w.t.s, w.t.q, w.t.rt + 1);
        return;
    }
    int s = w.t.s + 1;
    KvSeq q = seq_of(a, s);
    while (q.n == 0 && s + 1 < a.nseq) q = seq_of(a, ++s);
    w.t = make_tile<kRows, kUnit>(a, s, q, 0);
}

// Units of sequence s over all heads, summed by a warp.
__device__ __forceinline__ int64_t seq_units(const AttnArgs &a, int s, int lane) {
    const KvSeq q = seq_of(a, s);
    const int n = tiles_of<kRows>(a, q);
    int64_t w = 0;
    for (int i = lane; i < n; i += 32) w += make_tile<kRows, kUnit>(a, s, q, i).units;
    for (int i = 16; i; i >>= 1) w += __shfl_xor_sync(0xFFFFFFFFu, w, i);
    return w * a.kv.Hkv;
}

// This CTA's share of the units (left = 0: none).  W and the number of CTAs that take part come
// back too.  All warps call it; sums[512] and start are shared scratch.
__device__ __forceinline__ Walk find_share(const AttnArgs &a, int64_t *sums, Walk *start, int64_t &W, int32_t &C) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int per = (a.nseq + 511) / 512, groups = (a.nseq + per - 1) / per;   // sequences a sum
    for (int i = warp; i < groups; i += kThreads / 32) {
        int64_t w = 0;
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
            for (int64_t n; at >= (n = seq_units(a, s, lane)); ++s) at -= n;
            const KvSeq q = seq_of(a, s);
            for (int base = 0;; base += 32) {           // the tile: prefix sums over 32 tiles at a time
                const int rt = base + lane, n = tiles_of<kRows>(a, q);
                const int64_t mine = rt < n ? (int64_t)make_tile<kRows, kUnit>(a, s, q, rt).units * a.kv.Hkv : 0;
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
            w.h = (int32_t)(at / w.t.units);
            w.u = (int32_t)(at % w.t.units);
            w.left = end - begin;
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
    return *start;
}

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads, 1) attn_prefill_kernel(const __grid_constant__ AttnArgs a) {
    using L = Lay<D>;
    constexpr int kBlks = D / 64, kChunks = D / 32, kRow = kKvRow<FMT, D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = ptx::smem_align1024(smem_raw);
    __shared__ uint32_t tmem_at;
    __shared__ int err_flag;
    __shared__ Walk start;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::bar);
    float *qs = reinterpret_cast<float *>(sm + L::qs);
    float *ks = reinterpret_cast<float *>(sm + L::ks), *vs = reinterpret_cast<float *>(sm + L::vs);
    volatile uint32_t *live = reinterpret_cast<uint32_t *>(sm + L::live);
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
            ptx::mbar_init(&bars[PFULL + i], 4);
            ptx::mbar_init(&bars[OFULL + i], 1);
        }
        ptx::mbar_init(&bars[DRAIN], 1);
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
    const Walk mine = find_share(a, reinterpret_cast<int64_t *>(sm + L::plan), &start, W, C);
    ptx::tc_fence_after();
    const uint32_t tm = tmem_at;
    const int64_t end = C > 0 ? (int64_t)(blockIdx.x + 1) * W / C : 0;
    if (tid == 0) a.split[blockIdx.x].last_cta = -1;
    const int pt = a.kv.page_tokens;
    auto wait = [&](int b, uint32_t parity) { return ptx::mbar_wait(&bars[b], parity, err); };

    if (mine.left > 0) {
        if (warp < kSoftWarps) {
            // ================================================== softmax and output
            const int half = warp / 4, row = half * kHalf + (warp % 4) * 32 + lane;
            const uint32_t lanes = (uint32_t)((warp % 4) * 32) << 16;
            const uint32_t tS = tm + lanes + half * 128, tO = tm + lanes + 256 + half * 128;
            Walk w = mine;
            uint32_t n_s = 0;              // units of this half so far: the parity of its barriers
            uint32_t n_unit = 0, n_item = 0;
            bool ok = true;
            while (w.left > 0 && ok) {
                const Tile &t = w.t;
                const int32_t u_first = w.u, u_last = (int32_t)min((int64_t)t.units, w.u + w.left);
                if (half * kHalf >= t.nrows) {           // nothing in this half
                    n_unit += u_last - u_first;
                    w.left -= u_last - u_first;
                    ++n_item;
                    if (w.left > 0) next_item(a, w);
                    continue;
                }
                const bool in = row < t.nrows;
                const int32_t at = t.row0 + row, pos = in ? t.q.len - t.q.n + at / a.G : -1;
                float m = -INFINITY, l = 0.f, ref = 0.f, f_row = 0.f;
                {
                    float z[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) z[i] = 0.f;
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) ptx::tmem_st32(tO + 32 * c, z);
                }
                for (int32_t u = u_first; u < u_last; ++u, ++n_s, ++n_unit) {
                    const int32_t j0 = unit_token<kUnit>(t, u);
                    ok = __all_sync(0xFFFFFFFFu, wait(SFULL + half, n_s & 1));
                    if (!ok) break;
                    ptx::tc_fence_after();
                    if (u == u_first) f_row = qs[(n_item & 1) * kRows + row];
                    const uint32_t there = live[n_unit % kRing];
                    const bool whole = all_see(a, t, j0, kUnit) && there == 0xFFu;
                    // columns that this row sees, 32 at a time
                    auto seen = [&](int c) -> uint32_t {
                        auto low = [](int32_t n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; };
                        const int32_t b = j0 + 32 * c;
                        uint32_t s = low(pos + 1 - b);
                        if (a.window > 0) s &= ~low(pos - a.window + 1 - b) | low(a.sinks - b);
                        if (!(there >> (2 * c) & 1u)) s &= 0xFFFF0000u;
                        if (!(there >> (2 * c + 1) & 1u)) s &= 0x0000FFFFu;
                        return s;
                    };
                    float fk[8];
#pragma unroll
                    for (int g = 0; g < 8; ++g) fk[g] = FMT == KDA_KV_I8 ? f_row * ks[(n_unit % kRing) * 8 + g] : f_row;
                    // ---- the row's maximum (f >= 0, so it may be taken before the product)
                    float top = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float s[32];
                        ptx::tmem_ld32(tS + 32 * c, s);
                        ptx::tmem_wait_ld();
                        if (!whole) {
                            const uint32_t see = seen(c);
#pragma unroll
                            for (int i = 0; i < 32; ++i) s[i] = see >> i & 1u ? s[i] : -INFINITY;
                        }
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            float x = s[16 * g];
#pragma unroll
                            for (int i = 1; i < 16; ++i) x = fmaxf(x, s[16 * g + i]);
                            x = x == -INFINITY ? x : x * fk[2 * c + g];
                            top = fmaxf(top, x);
                        }
                    }
                    // ---- value scales
                    float vmax = 0.f;
                    if (FMT == KDA_KV_I8) {
#pragma unroll
                        for (int g = 0; g < 8; ++g) {
                            const float x = vs[(n_unit % kRing) * 8 + g];
                            if (x < INFINITY) vmax = fmaxf(vmax, x);
                        }
                    }
                    // ---- tokens whose values were taken out of the product (16-bit cache)
                    uint32_t out_of[4] = {0, 0, 0, 0};
                    bool odd = false;
                    if (FMT == KDA_KV_BF16 && !whole) {
                        ok = __all_sync(0xFFFFFFFFu, wait(VFULL + (n_unit & 1), n_unit >> 1 & 1));
                        if (!ok) break;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            out_of[i] = bad[(n_unit & 1) * 4 + i];
                            odd |= out_of[i] != 0;
                        }
                    }
                    // ---- O, where the row's reference moves
                    const bool grow = top > m + kGrow || (m == -INFINITY && top > -INFINITY);
                    const bool scaled = FMT == KDA_KV_I8 && vmax > 2.f * ref;
                    if (__any_sync(0xFFFFFFFFu, grow || scaled || odd)) {
                        float f = 1.f;
                        if (grow) {
                            f = m == -INFINITY ? 0.f : ex2(m - top);
                            l *= f;
                            m = top;
                        }
                        if (scaled) {
                            const float r = fmaxf(vmax, kMinRef);
                            f *= ref / r;
                            ref = r;
                        }
                        if (u > u_first || odd) {
                            if (u > u_first) {
                                ok = __all_sync(0xFFFFFFFFu, wait(OFULL + half, (n_s - 1) & 1));
                                if (!ok) break;
                                ptx::tc_fence_after();
                            } else {
                                ptx::tmem_wait_st();
                            }
#pragma unroll
                            for (int c = 0; c < kChunks; ++c) {
                                float o[32];
                                ptx::tmem_ld32(tO + 32 * c, o);
                                ptx::tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] *= f;
                                if (FMT == KDA_KV_BF16 && odd) {
                                    for (int j = 0; j < kUnit; ++j) {
                                        if (!(out_of[j >> 5] >> (j & 31) & 1u)) continue;   // the same for all rows
                                        const float s = tmem_ld1(tS + j);
                                        ptx::tmem_wait_ld();
                                        if (sees(a, pos, j0 + j)) {
                                            const float p = ex2(s * f_row - (m == -INFINITY ? 0.f : m));
                                            const int b = (j0 + j) / pt, slot = (j0 + j) % pt;
                                            const uint8_t *rec = kv_record(
                                                a.kv, __ldg(a.kv.table + (int64_t)t.s * a.kv.max_pages + b), w.h);
                                            if (rec)
#pragma unroll
                                                for (int i = 0; i < 32; ++i)
                                                    o[i] += p * __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(
                                                                    rec + pt * kRow +
                                                                    kv_tile_off<kRow>(pt, slot, 64 * c + 2 * i)));
                                        }
                                        __syncwarp();
                                    }
                                }
                                ptx::tmem_st32(tO + 32 * c, o);
                            }
                        }
                    }
                    // ---- probabilities, over the scores that they come from
                    const float ms = m == -INFINITY ? 0.f : m;
                    float bias[8], back[8];
#pragma unroll
                    for (int g = 0; g < 8; ++g) {
                        bias[g] = -ms;
                        back[g] = 1.f;
                        if (FMT == KDA_KV_I8) {
                            const float x = vs[(n_unit % kRing) * 8 + g];
                            const float lg = x == 0.f ? 0.f : x < INFINITY ? fmaxf(log2f(x / ref), -100.f) + kPBits : NAN;
                            bias[g] += lg;
                            back[g] = ex2(-lg);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float s[32];
                        ptx::tmem_ld32(tS + 32 * c, s);
                        ptx::tmem_wait_ld();
                        const uint32_t see = whole ? ~0u : seen(c);
                        uint32_t p[16];
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            float2 sum = make_float2(0.f, 0.f);
                            const float2 ff = make_float2(fk[2 * c + g], fk[2 * c + g]);
                            const float2 bb = make_float2(bias[2 * c + g], bias[2 * c + g]);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int e = 16 * g + 2 * i;
                                float2 y = tcx::ffma2(make_float2(s[e], s[e + 1]), ff, bb);
                                y.x = ex2(y.x), y.y = ex2(y.y);
                                if (!whole) {
                                    y.x = see >> e & 1u ? y.x : 0.f;
                                    y.y = see >> (e + 1) & 1u ? y.y : 0.f;
                                }
                                sum = tcx::fadd2(sum, y);
                                p[8 * g + i] = pack2<FMT>(y.x, y.y);
                            }
                            l += (sum.x + sum.y) * back[2 * c + g];
                        }
                        tmem_st16u(tS + 16 * c, p);
                    }
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before();
                    tcx::warp_arrive(&bars[PFULL + half]);
                }
                if (!ok) break;
                // ---- the item's output, or this CTA's part of it
                ok = __all_sync(0xFFFFFFFFu, wait(OFULL + half, (n_s - 1) & 1));
                if (!ok) break;
                ptx::tc_fence_after();
                const bool starts = u_first == 0, ends = u_last == t.units;
                const int64_t tok = (int64_t)t.q.tok0 + at / a.G, orow = tok * a.Hq + w.h * a.G + at % a.G;
                const float unscale = FMT == KDA_KV_I8 ? ref * 0x1p-6f : 1.f;
                const float f = starts && ends ? (l == 0.f ? 0.f : unscale / l) : unscale;
                float *part = a.part + ((int64_t)(blockIdx.x * 2 + (starts ? 1 : 0)) * kRows + row) * kPartRow<D>;
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    float o[32];
                    ptx::tmem_ld32(tO + 32 * c, o);
                    ptx::tmem_wait_ld();
                    if (in && starts && ends) {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + orow * D + 32 * c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t x[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float p0 = l == 0.f ? 0.f : o[8 * i + 2 * j] * f, p1 = l == 0.f ? 0.f : o[8 * i + 2 * j + 1] * f;
                                x[j] = tcx::f2_to_bf2(p0, p1);
                            }
                            dst[i] = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                    } else if (in) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            reinterpret_cast<float4 *>(part + 32 * c)[i] =
                                make_float4(o[4 * i] * f, o[4 * i + 1] * f, o[4 * i + 2] * f, o[4 * i + 3] * f);
                    }
                    __syncwarp();
                }
                ptx::tc_fence_before();
                if (in) {
                    if (!(starts && ends)) part[D] = m, part[D + 1] = l;
                    else if (a.lse) a.lse[orow] = lse_of(m, l);
                }
                if (tid == 0 && starts && !ends) {
                    AttnSplit sp{};
                    sp.last_cta = cta_of(end - 1 + (t.units - u_last), W, C);
                    sp.row_tok = t.q.tok0;
                    sp.head = w.h;
                    sp.row0 = t.row0;
                    sp.nrows = t.nrows;
                    a.split[blockIdx.x] = sp;
                }
                w.left -= u_last - u_first;
                ++n_item;
                if (w.left > 0) next_item(a, w);
            }
            if (!ok && lane == 0) flag_status(a.kv.status, KDA_DEV_TIMEOUT);
        } else if (warp < kSoftWarps + kLoadWarps) {
            // ================================================== queries, and keys and values
            const int lw = warp - kSoftWarps, lt = tid - kSoftWarps * 32;
            Walk w = mine;
            uint32_t n_unit = 0, n_item = 0;
            bool ok = true;
            // 8-bit: the units' codes are read one unit ahead into registers.  A warp takes 32 tokens;
            // eight lanes take four units of token r and of token r ^ 5, which keeps both their reads
            // and their writes in different banks.
            constexpr int kRegs = kRow / 16;
            constexpr int kQuads = kRow / 64;                         // groups of four 16-byte units a row
            uint4 kc[kRegs], vc[kRegs];
            const int r8 = (lane >> 3) ^ ((lane >> 2 & 1) * 5), ul = lane & 3;
            float2 sc = make_float2(0.f, 0.f);                        // lanes 0-7: scales of the unit's groups
            uint32_t there = 0;                                       // groups that are in the pool
            // the unit whose codes are fetched next, looked up one more unit ahead: its tokens, its
            // head and, in lanes 0-7, the pages of its groups
            Walk far = mine;
            int32_t f_tok = 0, f_head = 0, f_page = 0;
            uint32_t f_want = 0;
            bool f_any = false;
            auto look = [&]() {
                f_any = far.left > 0;
                if (!f_any) return;
                f_tok = unit_token<kUnit>(far.t, far.u);
                f_head = far.h;
                const int32_t j = f_tok + 16 * lane;
                const bool want = lane < 8 && any_sees(a, far.t, j, 16);
                if (want) f_page = __ldg(a.kv.table + (int64_t)far.t.s * a.kv.max_pages + j / pt);
                f_want = __ballot_sync(0xFFFFFFFFu, want);
                if (--far.left > 0 && ++far.u == far.t.units) next_item(a, far);
            };
            auto fetch = [&](bool values, uint4 (&c)[kRegs]) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {                         // eight tokens
                    const int32_t id = __shfl_sync(0xFFFFFFFFu, f_page, 2 * lw + (i >> 1));
                    const int32_t slot = (f_tok + 32 * lw + 8 * i) % pt + r8;
                    const bool real = (f_want >> (2 * lw + (i >> 1)) & 1u) && (uint32_t)id < (uint32_t)a.kv.num_pages;
                    const uint8_t *tile = a.kv.base + (int64_t)id * a.kv.page_bytes + (int64_t)f_head * a.kv.rec_bytes +
                                          (values ? pt * kRow : 0);
#pragma unroll
                    for (int y = 0; y < kQuads; ++y) {
                        c[i * kQuads + y] = make_uint4(0, 0, 0, 0);
                        if (real)
                            c[i * kQuads + y] = __ldg(reinterpret_cast<const uint4 *>(
                                tile + kv_tile_off<kRow>(pt, slot, 16 * (4 * y + ul))));
                    }
                }
            };
            auto scales = [&]() {                                     // lanes 0-7 of the first warp
                if (lw != 0) return;
                sc = make_float2(0.f, 0.f);
                const uint8_t *rec = lane < 8 && (f_want >> lane & 1u) ? kv_record(a.kv, f_page, f_head) : nullptr;
                if (rec) sc = __ldg(reinterpret_cast<const float2 *>(rec + 2 * pt * kRow));
                there = __ballot_sync(0xFFFFFFFFu, rec != nullptr);
            };
            auto put = [&](const uint4 (&c)[kRegs], uint8_t *tile) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int y = 0; y < kQuads; ++y) {
                        uint4 lo, hi;
                        codes_to_half(c[i * kQuads + y], lo, hi);
                        const int r = 32 * lw + 8 * i + r8, unit = 4 * y + ul;      // columns 16 unit ..
                        uint8_t *line = tile + (unit >> 2) * L::blk + r * 128;
                        *reinterpret_cast<uint4 *>(line + (((2 * unit) & 7) ^ (r & 7)) * 16) = lo;
                        *reinterpret_cast<uint4 *>(line + (((2 * unit + 1) & 7) ^ (r & 7)) * 16) = hi;
                    }
            };
            if (FMT == KDA_KV_I8) {
                look();
                scales();
                fetch(false, kc);
                fetch(true, vc);
                look();
            }
            while (w.left > 0 && ok) {
                const int32_t u_first = w.u, u_last = (int32_t)min((int64_t)w.t.units, w.u + w.left);
                // ---- queries
                ok = __all_sync(0xFFFFFFFFu, wait(QEMPTY, (n_item & 1) ^ 1));
                if (!ok) break;
                {
                    constexpr int kTpr = D / 16, kRpp = kLoadWarps * 32 / kTpr;
                    const float sign = a.scale < 0.f ? -1.f : 1.f;
                    const int rows = w.t.nrows > kHalf ? kRows : kHalf, c = lt % kTpr;
                    for (int r = lt / kTpr; r < rows; r += kRpp) {
                        const int at = w.t.row0 + r;
                        uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                        if (r < w.t.nrows) {
                            const uint4 *src = reinterpret_cast<const uint4 *>(
                                static_cast<const __nv_bfloat16 *>(a.q) + (int64_t)(w.t.q.tok0 + at / a.G) * a.q_stride +
                                (int64_t)(w.h * a.G + at % a.G) * D + 16 * c);
                            x[0] = src[0], x[1] = src[1];
                        }
                        float f = a.scale * sign * kLog2e;
                        float e[16];
                        const uint32_t xw[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 p = tcx::bf2_to_f2(xw[i]);
                            e[2 * i] = p.x * sign, e[2 * i + 1] = p.y * sign;
                        }
                        if (FMT == KDA_KV_I8) {
                            // a power of two that brings the row's largest magnitude to [2^10, 2^11)
                            float top = 0.f;
#pragma unroll
                            for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(e[i]));
#pragma unroll
                            for (int i = 1; i < kTpr; i <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));
                            const int b = (int)(__float_as_uint(top) >> 23);
                            const int shift = b == 0 || b == 255 ? 0 : min(max(137 - b, -120), 120);
                            const float up = __uint_as_float((uint32_t)(127 + shift) << 23);
#pragma unroll
                            for (int i = 0; i < 16; ++i) e[i] *= up;
                            f *= __uint_as_float((uint32_t)(127 - shift) << 23);
                        }
                        uint32_t y[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = pack2<FMT>(e[2 * i], e[2 * i + 1]);
                        uint8_t *dst = sm + L::q + (r / kHalf) * L::half_q + (c >> 2) * (kHalf * 128);
                        const int rr = r % kHalf;
                        *reinterpret_cast<uint4 *>(dst + ptx::sw128_off(rr, 32 * (c & 3))) = make_uint4(y[0], y[1], y[2], y[3]);
                        *reinterpret_cast<uint4 *>(dst + ptx::sw128_off(rr, 32 * (c & 3) + 16)) = make_uint4(y[4], y[5], y[6], y[7]);
                        if (c == 0) qs[(n_item & 1) * kRows + r] = f;
                    }
                    ptx::fence_proxy_async_smem();
                    tcx::warp_arrive(&bars[QFULL]);
                }
                for (int32_t u = u_first; u < u_last; ++u, ++n_unit) {
                    const int st = n_unit & 1;
                    const uint32_t par = (n_unit >> 1 & 1) ^ 1;
                    if (FMT == KDA_KV_I8) {
                        ok = __all_sync(0xFFFFFFFFu, wait(KEMPTY + st, par));
                        if (!ok) break;
                        put(kc, sm + L::k + st * L::tile);
                        if (lw == 0) {
                            if (lane < 8) {
                                ks[(n_unit % kRing) * 8 + lane] = fabsf(sc.x);
                                vs[(n_unit % kRing) * 8 + lane] = fabsf(sc.y);
                            }
                            if (lane == 0) live[n_unit % kRing] = there;
                        }
                        ptx::fence_proxy_async_smem();
                        tcx::warp_arrive(&bars[KFULL + st]);
                        if (f_any) {
                            fetch(false, kc);
                            scales();
                        }
                        ok = __all_sync(0xFFFFFFFFu, wait(VEMPTY + st, par));
                        if (!ok) break;
                        put(vc, sm + L::v + st * L::tile);
                        ptx::fence_proxy_async_smem();
                        tcx::warp_arrive(&bars[VFULL + st]);
                        if (f_any) {
                            fetch(true, vc);
                            look();
                        }
                    } else {
                        // values that not every row sees: a token that no row sees is cleared (0 times
                        // what a stale slot holds need not be 0), and one with an infinity or a NaN is
                        // taken out and left to the rows that see it
                        ok = __all_sync(0xFFFFFFFFu, wait(VRAW + st, n_unit >> 1 & 1));
                        if (!ok) break;
                        const int32_t j0 = unit_token<kUnit>(w.t, u);
                        const uint32_t groups = live[n_unit % kRing];
                        if (!all_see(a, w.t, j0, kUnit) || groups != 0xFFu) {
                            uint8_t *line = sm + L::v + st * L::tile + lt * 128;
                            const bool any = (groups >> (lt >> 4) & 1u) && any_sees(a, w.t, j0 + lt, 1);
                            bool strange = false;
                            if (any) {
#pragma unroll
                                for (int b = 0; b < kBlks; ++b)
                                    for (int i = 0; i < 8; ++i) {
                                        const uint4 x = *reinterpret_cast<const uint4 *>(line + b * L::blk + ((i ^ (lt & 7)) << 4));
                                        for (uint32_t y : {x.x, x.y, x.z, x.w})
                                            strange |= (y & 0x7F80u) == 0x7F80u || (y & 0x7F800000u) == 0x7F800000u;
                                    }
                            }
                            if (!any || strange)
#pragma unroll
                                for (int b = 0; b < kBlks; ++b)
                                    for (int i = 0; i < 8; ++i)
                                        *reinterpret_cast<uint4 *>(line + b * L::blk + ((i ^ (lt & 7)) << 4)) = make_uint4(0, 0, 0, 0);
                            const uint32_t mask = __ballot_sync(0xFFFFFFFFu, strange);
                            if (lane == 0) bad[st * 4 + lw] = mask;
                            ptx::fence_proxy_async_smem();
                        }
                        tcx::warp_arrive(&bars[VFULL + st]);
                    }
                }
                w.left -= u_last - u_first;
                ++n_item;
                if (w.left > 0 && ok) next_item(a, w);
            }
        } else if (warp == kMmaWarp) {
            // ================================================== products
            if (lane == 0) {
                const uint32_t sb = ptx::smem_u32(sm);
                Walk w = mine;
                uint32_t n_unit = 0, n_item = 0, n_p[2] = {0, 0};
                bool ok = true;
                auto scores = [&](int half, int st) {
#pragma unroll
                    for (int s = 0; s < D / 16; ++s) {
                        const uint32_t off = (s >> 2) * L::blk + (s & 3) * 32;
                        ptx::mma_bf16(tm + half * 128, ptx::sdesc_sw128(sb + L::q + half * L::half_q + off, 16, 1024),
                                      ptx::sdesc_sw128(sb + L::k + st * L::tile + off, 16, 1024), idesc<FMT>(128, 128, 0),
                                      s > 0 ? 1u : 0u);
                    }
                    ptx::mma_commit(&bars[SFULL + half]);
                };
                auto outputs = [&](int half, int st) {
#pragma unroll
                    for (int s = 0; s < kUnit / 16; ++s)
                        ptx::mma_bf16_ta(tm + 256 + half * 128, tm + half * 128 + s * 8,
                                         ptx::sdesc_sw128(sb + L::v + st * L::tile + s * 2048, L::blk, 1024),
                                         idesc<FMT>(128, D, 1), 1u);
                    ptx::mma_commit(&bars[OFULL + half]);
                };
                while (w.left > 0 && ok) {
                    const int32_t n = (int32_t)min((int64_t)w.t.units - w.u, w.left);
                    const int halves = w.t.nrows > kHalf ? 2 : 1;
                    ok = wait(QFULL, n_item & 1) && wait(KFULL + (n_unit & 1), n_unit >> 1 & 1);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    for (int h = 0; h < halves; ++h) scores(h, n_unit & 1);
                    ptx::mma_commit(&bars[KEMPTY + (n_unit & 1)]);
                    if (n == 1) ptx::mma_commit(&bars[QEMPTY]);
                    for (int32_t i = 0; i < n && ok; ++i, ++n_unit) {
                        const int st = n_unit & 1, nx = st ^ 1;
                        for (int h = 0; h < halves; ++h) {
                            ok = wait(PFULL + h, n_p[h] & 1) && (h || wait(VFULL + st, n_unit >> 1 & 1));
                            if (!ok) break;
                            ++n_p[h];
                            ptx::tc_fence_after();
                            outputs(h, st);
                            if (h + 1 == halves) ptx::mma_commit(&bars[VEMPTY + st]);
                            if (i + 1 < n) {
                                ok = h || wait(KFULL + nx, (n_unit + 1) >> 1 & 1);
                                if (!ok) break;
                                ptx::tc_fence_after();
                                scores(h, nx);
                                if (h + 1 == halves) {
                                    ptx::mma_commit(&bars[KEMPTY + nx]);
                                    if (i + 2 == n) ptx::mma_commit(&bars[QEMPTY]);
                                }
                            }
                        }
                    }
                    w.left -= n;
                    ++n_item;
                    if (w.left > 0) next_item(a, w);
                }
                ptx::mma_commit(&bars[DRAIN]);
                ptx::mbar_wait(&bars[DRAIN], 0, nullptr);
            }
            __syncwarp();
        } else if (FMT == KDA_KV_BF16) {
            // ================================================== copies (16-bit cache)
            Walk w = mine;
            bool ok = true;
            uint32_t n_k = 0, n_v = 0;                                // tiles asked for
            bool want;                                                // lanes 0-7: this group of 16 tokens is needed
            auto look = [&]() -> int32_t {                            // and its page
                const int32_t j = unit_token<kUnit>(w.t, w.u) + 16 * lane;
                want = lane < 8 && any_sees(a, w.t, j, 16);
                return want ? __ldg(a.kv.table + (int64_t)w.t.s * a.kv.max_pages + j / pt) : 0;
            };
            int32_t page = look();
            while (w.left > 0) {
                const int st = n_k & 1;
                const uint32_t par = (n_k >> 1 & 1) ^ 1;
                const int32_t slot = (unit_token<kUnit>(w.t, w.u) + 16 * lane) % pt;
                const uint8_t *rec = want ? kv_record(a.kv, page, w.h) : nullptr;
                const uint32_t there = __ballot_sync(0xFFFFFFFFu, rec != nullptr);
                if (--w.left > 0) {
                    if (++w.u == w.t.units) next_item(a, w);
                    page = look();                                    // the next unit's, while this one waits
                }
                ok = __all_sync(0xFFFFFFFFu, wait(KEMPTY + st, par));
                if (!ok) break;
                if (lane == 0) {
                    live[n_k % kRing] = there;
                    ptx::mbar_arrive_expect_tx(&bars[KFULL + st], __popc(there) * 16 * kRow);
                }
                __syncwarp();
                if (rec)
#pragma unroll
                    for (int b = 0; b < kBlks; ++b)
                        ptx::bulk_load(sm + L::k + st * L::tile + b * L::blk + lane * 2048, rec + b * pt * 128 + slot * 128, 2048,
                                       &bars[KFULL + st]);
                ++n_k;
                ok = __all_sync(0xFFFFFFFFu, wait(VEMPTY + st, par));
                if (!ok) break;
                if (lane == 0) ptx::mbar_arrive_expect_tx(&bars[VRAW + st], __popc(there) * 16 * kRow);
                __syncwarp();
                if (rec)
#pragma unroll
                    for (int b = 0; b < kBlks; ++b)
                        ptx::bulk_load(sm + L::v + st * L::tile + b * L::blk + lane * 2048,
                                       rec + pt * kRow + b * pt * 128 + slot * 128, 2048, &bars[VRAW + st]);
                ++n_v;
            }
            // the last copies land before the block ends, whatever became of their readers
            __syncwarp();
            for (uint32_t i = n_k > 2 ? n_k - 2 : 0; i < n_k; ++i) ptx::mbar_wait(&bars[KFULL + (i & 1)], i >> 1 & 1, nullptr);
            for (uint32_t i = n_v > 2 ? n_v - 2 : 0; i < n_v; ++i) ptx::mbar_wait(&bars[VRAW + (i & 1)], i >> 1 & 1, nullptr);
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

cudaError_t launch_attn_prefill(const AttnArgs &a, cudaStream_t s) {
    if (a.kv.d == 128) return a.kv.fmt == KDA_KV_I8 ? run<KDA_KV_I8, 128>(a, s) : run<KDA_KV_BF16, 128>(a, s);
    return a.kv.fmt == KDA_KV_I8 ? run<KDA_KV_I8, 64>(a, s) : run<KDA_KV_BF16, 64>(a, s);
}

}  // namespace kda
