// Attention of few query rows over the paged cache (decoding, drafts; every float32 call).
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j - m_i), j over the visible tokens
//
// in one pass over the cache with a running maximum and sum per row.  Bound: the cache's bytes.
// The rows of a group (query heads that share a key/value head, times the call's tokens) fill the
// M = 16 of a warp-level matrix product, so a cached byte is read once for all of them; wider
// tensor-memory tiles would stand empty here.
//
// Two CTAs of 4 warps an SM, so that one streams while the other joins its warps or starts an item.
// A warp takes a step of a unit's tokens (32 of the 8-bit cache, 16 of the 16-bit one: groups of 16
// tokens, each in one page) and runs alone: it copies its own tokens of later units into its own
// ring of shared-memory stages (bulk copies: a page's rows are contiguous) and keeps its own
// maxima, sums and 16 x D accumulators.  The warps meet only at an item's end.
//
// 8-bit cache: codes c become fp16 exactly (the byte under the exponent of 1024, less 1152), a
// query row is scaled by a power of two into fp16's range, so q . c carries no rounding beyond
// fp32 sums, and the block's key scale multiplies the score.  The value scale goes into the
// probabilities: p (vs / ref) 2^13 in fp16, ref the largest value scale so far.  float32 queries
// are split into 2 fp16 terms (3 bf16 terms over the 16-bit cache), and so are the probabilities:
// the products then keep 22 to 24 bits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"

namespace kda {
namespace {

using namespace attn;

constexpr int kWarps = 4;
constexpr float kPScale = 8192.f;                     // probabilities' scale in fp16
constexpr float kMinRef = 0x1p-100f;

template <int FMT, int D>
struct Shape {
    static constexpr int row = kKvRow<FMT, D>;
    static constexpr int step = FMT == KDA_KV_I8 ? 32 : 16, groups = step / 16, unit = kWarps * step;
    static constexpr int group = row * 16;            // K or V bytes of 16 tokens
    static constexpr int tile = groups * group;
    static constexpr int stage = 2 * tile + 128;      // keys, values, 16 bytes of scales a group
    static constexpr int stages = D == 128 ? 2 : 4;        // of a warp's ring, two CTAs an SM
    static constexpr int deep_stages = D == 128 ? 5 : 8;   // one CTA an SM
};

template <int FMT, int D, int NT>
struct Smem {
    // behind the rings
    static constexpr int o_acc = 0;                                      // [kWarps][16][D] fp32
    static constexpr int o_ml = o_acc + kWarps * 16 * D * 4;             // [2][kWarps][16][2] fp32
    static constexpr int o_q = o_ml + 2 * kWarps * 16 * 8;               // fragments of split queries
    static constexpr int o_bar = o_q + (NT > 1 ? NT * (D / 16) * 512 : 0);
    static constexpr int o_live = o_bar + kWarps * Shape<FMT, D>::deep_stages * 8;
    static constexpr int o_misc = o_live + kWarps * Shape<FMT, D>::deep_stages * 4;
    static constexpr int total(int stages) { return kWarps * stages * Shape<FMT, D>::stage + o_misc + 128; }
};

// Fragment loads and products are plain functions of their operands to the compiler, which may so
// place them as their latencies want.  What keeps the loads between a stage's arrival and its release
// is the address (pinned behind the wait) and the accumulators (pinned before the release).
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(addr));
}
template <int N>
__device__ __forceinline__ void pin(float (&o)[N][4]) {
#pragma unroll
    for (int j = 0; j < N; j += 2)
        asm volatile("" : "+f"(o[j][0]), "+f"(o[j][1]), "+f"(o[j][2]), "+f"(o[j][3]), "+f"(o[j + 1][0]), "+f"(o[j + 1][1]),
                     "+f"(o[j + 1][2]), "+f"(o[j + 1][3])::"memory");
}

// D (16x8) += A (16x16) B (16x8), fp32 sums.
template <int FMT>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (FMT == KDA_KV_I8)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two biased bytes (selected by SEL, under the exponent byte 0x64) as fp16: 1024 + b - 1152 = code.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t half2_of(uint32_t biased) {
    const uint32_t u = __byte_perm(biased, 0x64646464u, SEL);
    const uint32_t k = 0x64806480u;   // 1152, 1152
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&u), *reinterpret_cast<const __half2 *>(&k));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// x (already in range) as NT packed terms of the product's type whose sum is x to NT times its bits.
template <int FMT, int NT>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&out)[NT]) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        if constexpr (FMT == KDA_KV_I8) {
            const __half2 h = __floats2half2_rn(x, y);
            out[i] = *reinterpret_cast<const uint32_t *>(&h);
            if (i + 1 < NT) x -= __low2float(h), y -= __high2float(h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
            out[i] = *reinterpret_cast<const uint32_t *>(&h);
            if (i + 1 < NT) x -= __low2float(h), y -= __high2float(h);
        }
    }
}

// Place of the 4-float unit u of a row of the warps' accumulators in shared memory, so that the
// fragment stores of a warp fall into different banks.
template <int FMT, int D>
__device__ __forceinline__ int acc_unit(int row, int u) {
    return FMT == KDA_KV_BF16 ? u ^ ((row & 7) << 1) : u ^ ((row & 1) << 2);
}

// Where a warp's loads stand: the unit whose copy comes next; lane i's group i of it, its page id
// already on the way.
struct Cursor {
    Tile t;
    int32_t h, u;
    bool want;
    int32_t page, slot;
};

template <int FMT, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, 2) attn_decode_kernel(const __grid_constant__ AttnArgs a) {
    using S = Shape<FMT, D>;
    using M = Smem<FMT, D, NT>;
    constexpr int kKs = D / 16;   // 16-wide slices of a row
    constexpr int kNt = D / 8;    // 8-wide output tiles
    constexpr int kGr = S::groups;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *rings = ptx::smem_align1024(smem_raw);
    const int stages = a.deep ? S::deep_stages : S::stages;
    uint8_t *sm = rings + kWarps * stages * S::stage;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane >> 2, t = lane & 3;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + M::o_bar) + warp * stages;
    volatile uint32_t *live = reinterpret_cast<uint32_t *>(sm + M::o_live) + warp * stages;
    uint8_t *ring = rings + warp * stages * S::stage;
    float *ml = reinterpret_cast<float *>(sm + M::o_ml);   // of this item; the last one's may still be read
    int ml_next = kWarps * 32;
    float *acc = reinterpret_cast<float *>(sm + M::o_acc);
    uint32_t *qfrag = reinterpret_cast<uint32_t *>(sm + M::o_q);
    volatile int *err = reinterpret_cast<int *>(sm + M::o_misc);
    int64_t *share = reinterpret_cast<int64_t *>(sm + M::o_misc + 16);   // warps' sums, then the start

    if (lane == 0)
        for (int i = 0; i < stages; ++i) ptx::mbar_init(&bars[i], 1);
    if (tid == 0) *err = 0;
    ptx::fence_mbar_init();
    ptx::grid_dep_wait();

    // ---- this CTA's units: sum the units of every sequence, then find where its share begins
    const int32_t Hkv = a.kv.Hkv;
    auto seq = [&](int s) { return kv_seq(a.cu_q, a.kv_len, s, a.T_tot, a.max_q, a.kv); };
    auto seq_units = [&](int s) {
        const KvSeq q = seq(s);
        const int n = tiles_of<kAttnDecodeRows>(a, q);
        int64_t w = 0;
        for (int i = 0; i < n; ++i) w += make_tile<kAttnDecodeRows, S::unit>(a, s, q, i).units;
        return w * Hkv;
    };
    auto block_sum = [&](int64_t v, int64_t &before) {   // exclusive prefix over threads; returns the sum
        int64_t x = v;
        for (int i = 1; i < 32; i <<= 1) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, i);
            if (lane >= i) x += y;
        }
        __syncthreads();
        if (lane == 31) share[warp] = x;
        __syncthreads();
        int64_t base = 0, all = 0;
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) base += share[i];
            all += share[i];
        }
        before = base + x - v;
        return all;
    };
    int64_t W = 0, begin = 0, end;
    int32_t C = 0, h0, u0 = 0;
    Tile t0;
    if (a.whole) {
        // CTA i is item i: key/value head i % Hkv of sequence i / Hkv (one row tile a sequence)
        const KvSeq q = seq(blockIdx.x / Hkv);
        if (q.n == 0) return;
        h0 = blockIdx.x % Hkv;
        t0 = make_tile<kAttnDecodeRows, S::unit>(a, blockIdx.x / Hkv, q, 0);
        end = t0.units;
    } else {
        int64_t mine0 = 0, mine = 0, before;
        for (int s = tid; s < a.nseq; s += kWarps * 32) {
            const int64_t w = seq_units(s);
            if (s == tid) mine0 = w;
            mine += w;
        }
        W = block_sum(mine, before);
        if (tid == 0) a.split[blockIdx.x].last_cta = -1;
        C = (int32_t)min((int64_t)a.ctas, W);   // no CTA that takes part is without a unit
        if ((int32_t)blockIdx.x >= C) return;
        begin = (int64_t)blockIdx.x * W / C, end = (int64_t)(blockIdx.x + 1) * W / C;
        int64_t *found = share + kWarps;
        int64_t base = 0;
        for (int s = 0; s < a.nseq; s += kWarps * 32) {
            const int64_t w = s == 0 ? mine0 : (s + tid < a.nseq ? seq_units(s + tid) : 0);
            const int64_t all = block_sum(w, before);
            if (begin >= base + before && begin < base + before + w) {
                found[0] = s + tid;
                found[1] = begin - base - before;
            }
            base += all;
            if (begin < base) break;
        }
        __syncthreads();
        const int32_t s0 = (int32_t)found[0];
        int64_t left0 = found[1];   // units before `begin` in sequence s0
        const KvSeq q = seq(s0);
        for (int rt = 0;; ++rt) {
            t0 = make_tile<kAttnDecodeRows, S::unit>(a, s0, q, rt);
            if (left0 < (int64_t)t0.units * Hkv) break;
            left0 -= (int64_t)t0.units * Hkv;
        }
        h0 = (int32_t)(left0 / t0.units);
        u0 = (int32_t)(left0 % t0.units);
    }

    // the next item after (tile, head)
    auto next_item = [&](Tile &x, int32_t &h) {
        if (++h < Hkv) return;
        h = 0;
        if (x.rt + 1 < x.tiles) {
            x = make_tile<kAttnDecodeRows, S::unit>(a, x.s, x.q, x.rt + 1);
            return;
        }
        int s = x.s + 1;
        KvSeq q = seq(s);
        while (q.n == 0 && s + 1 < a.nseq) q = seq(++s);
        x = make_tile<kAttnDecodeRows, S::unit>(a, s, q, 0);
    };

    // ---- loads
    const int pt = a.kv.page_tokens;
    auto aim = [&](Cursor &c) {   // this warp's step of the cursor's unit
        const int32_t j = unit_token<S::unit>(c.t, c.u) + warp * S::step + lane * 16;
        c.want = lane < kGr && any_sees(a, c.t, j, 16);
        if (!c.want) return;
        const int32_t b = j / pt;
        c.slot = j - b * pt;
        c.page = __ldg(a.kv.table + (int64_t)c.t.s * a.kv.max_pages + b);
    };
    auto load = [&](const Cursor &c, int stage) {
        const uint8_t *rec = c.want ? kv_record(a.kv, c.page, c.h) : nullptr;
        const uint32_t there = __ballot_sync(0xFFFFFFFFu, rec != nullptr);
        if (lane == 0) {
            live[stage] = there;
            ptx::mbar_arrive_expect_tx(&bars[stage], __popc(there) * (2 * S::group + (FMT == KDA_KV_I8 ? 16 : 0)));
        }
        __syncwarp();
        if (!rec) return;
        // a group's lines follow one another in the page; a stage has them by line block, like a page
        constexpr uint32_t kLine = S::row < 128 ? S::row : 128, kRun = kLine * 16;
        uint8_t *dst = ring + stage * S::stage + lane * kRun;
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int b = 0; b < S::group / (int)kRun; ++b)
                ptx::bulk_load(dst + v * S::tile + b * kGr * kRun, rec + v * pt * S::row + b * pt * 128 + c.slot * kLine, kRun,
                               &bars[stage]);
        if (FMT == KDA_KV_I8)
            ptx::bulk_load(ring + stage * S::stage + 2 * S::tile + 16 * lane, rec + 2 * pt * S::row, 16, &bars[stage]);
    };
    Cursor cur;
    cur.t = t0;
    cur.h = h0;
    cur.u = u0;
    int64_t to_load = end - begin;
    aim(cur);
    auto load_next = [&](int stage) {
        if (to_load == 0) return;
        load(cur, stage);
        if (--to_load == 0) return;
        if (++cur.u == cur.t.units) {
            cur.u = 0;
            next_item(cur.t, cur.h);
        }
        aim(cur);
    };
    for (int i = 0; i < stages; ++i) load_next(i);

    // ---- items
    Tile tile = t0;
    int32_t head = h0, u = u0, stage = 0;
    uint32_t phase = 0;
    int64_t left = end - begin;
    while (left > 0) {
        const int32_t u_first = u, u_last = (int32_t)min((int64_t)tile.units, u + left);

        // query fragments, rows g and g + 8
        uint32_t qa[NT == 1 ? kKs : 1][4];
        float rs[2];
        int32_t pos[2];
        {
            float x[2][kKs * 4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = g + 8 * r, at = tile.row0 + row;
                const bool in = row < tile.nrows;
                pos[r] = in ? tile.q.len - tile.q.n + at / a.G : -1;
                const int64_t off = (int64_t)(tile.q.tok0 + at / a.G) * a.q_stride + (int64_t)(head * a.G + at % a.G) * D;
#pragma unroll
                for (int k = 0; k < kKs; ++k) {
                    // the four columns of slice k that this lane feeds: neighbours for the 8-bit
                    // cache (a lane's four bytes of a key), the fragment's own for the 16-bit one
                    const int c0 = 16 * k + (FMT == KDA_KV_I8 ? 4 * t : 2 * t);
                    const int c1 = FMT == KDA_KV_I8 ? c0 + 2 : c0 + 8;
                    float2 lo = make_float2(0.f, 0.f), hi = lo;
                    if (in) {
                        if (NT > 1) {
                            const float *p = static_cast<const float *>(a.q) + off;
                            lo = *reinterpret_cast<const float2 *>(p + c0);
                            hi = *reinterpret_cast<const float2 *>(p + c1);
                        } else {
                            const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(a.q) + off;
                            lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(p + c0));
                            hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(p + c1));
                        }
                    }
                    x[r][4 * k] = lo.x, x[r][4 * k + 1] = lo.y, x[r][4 * k + 2] = hi.x, x[r][4 * k + 3] = hi.y;
                }
                rs[r] = a.scale * kLog2e;
                if (FMT == KDA_KV_I8) {
                    // a power of two that brings the row's largest magnitude to [2^10, 2^11)
                    float top = 0.f;
#pragma unroll
                    for (int i = 0; i < kKs * 4; ++i) top = fmaxf(top, fabsf(x[r][i]));
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                    const int e = (int)(__float_as_uint(top) >> 23);
                    const int shift = e == 0 || e == 255 ? 0 : min(max(137 - e, -120), 120);
                    const float up = __uint_as_float((uint32_t)(127 + shift) << 23);
#pragma unroll
                    for (int i = 0; i < kKs * 4; ++i) x[r][i] *= up;
                    rs[r] *= __uint_as_float((uint32_t)(127 - shift) << 23);
                }
            }
#pragma unroll
            for (int k = 0; k < kKs; ++k) {
                uint32_t f[4][NT];
                split2<FMT, NT>(x[0][4 * k], x[0][4 * k + 1], f[0]);
                split2<FMT, NT>(x[1][4 * k], x[1][4 * k + 1], f[1]);
                split2<FMT, NT>(x[0][4 * k + 2], x[0][4 * k + 3], f[2]);
                split2<FMT, NT>(x[1][4 * k + 2], x[1][4 * k + 3], f[3]);
                if constexpr (NT == 1) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) qa[k][i] = f[i][0];
                } else if (k % kWarps == warp) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        *reinterpret_cast<uint4 *>(qfrag + ((n * kKs + k) * 32 + lane) * 4) =
                            make_uint4(f[0][n], f[1][n], f[2][n], f[3][n]);
                }
            }
            if constexpr (NT > 1) __syncthreads();
        }

        float o[kNt][4];
#pragma unroll
        for (int j = 0; j < kNt; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float ref = 0.f, inv_ref = 0.f;   // 8-bit: largest value scale so far

        for (; u < u_last; ++u, --left) {
            const bool ok = __all_sync(0xFFFFFFFFu, wait_bar(&bars[stage], phase, err));
            if (!ok) flag_status(a.kv.status, KDA_DEV_TIMEOUT);
            const uint32_t there = ok ? live[stage] : 0u;
            if (there) {
                const int32_t j0 = unit_token<S::unit>(tile, u) + warp * S::step;
                const uint8_t *buf = ring + stage * S::stage;
                uint32_t kb = ptx::smem_u32(buf);
                asm volatile("" : "+r"(kb)::"memory");
                const uint32_t vb = kb + S::tile;
                float sc[kGr][2], vs[kGr];   // a group's score factors (by row half) and value scale
#pragma unroll
                for (int y = 0; y < kGr; ++y) {
                    sc[y][0] = rs[0], sc[y][1] = rs[1], vs[y] = 0.f;
                    if (FMT == KDA_KV_I8) {
                        const float2 f = *reinterpret_cast<const float2 *>(buf + 2 * S::tile + 16 * y);
                        if (there >> y & 1u) sc[y][0] *= fabsf(f.x), sc[y][1] *= fabsf(f.x), vs[y] = fabsf(f.y);
                    }
                }
                // ---- scores: c[n] of tokens j0 + 8 n ..
                float c[2 * kGr][4] = {};
                const int mr = lane & 7, mm = lane >> 3;   // row and matrix whose address this lane gives
                auto slice = [&](float (&d)[4], int k, uint32_t b0, uint32_t b1) {
                    if constexpr (NT == 1) {
                        mma<FMT>(d, qa[k], b0, b1);
                    } else {
#pragma unroll
                        for (int z = NT - 1; z >= 0; --z) {
                            const uint4 f = *reinterpret_cast<const uint4 *>(qfrag + ((z * kKs + k) * 32 + lane) * 4);
                            const uint32_t qf[4] = {f.x, f.y, f.z, f.w};
                            mma<FMT>(d, qf, b0, b1);
                        }
                    }
                };
                if constexpr (FMT == KDA_KV_I8) {
#pragma unroll
                    for (int i = 0; i < kKs / 4; ++i)
#pragma unroll
                        for (int n = 0; n < 2 * kGr; ++n) {
                            uint32_t w[4];
                            ldsm4(w, kb + kv_tile_off<S::row>(S::step, 8 * n + mr, 16 * (4 * i + mm)));
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t b = w[k] ^ 0x80808080u;
                                slice(c[n], 4 * i + k, half2_of<0x4140>(b), half2_of<0x4342>(b));
                            }
                        }
                } else {
#pragma unroll
                    for (int i = 0; i < kKs / 2; ++i)
#pragma unroll
                        for (int n = 0; n < 2 * kGr; ++n) {
                            uint32_t w[4];
                            ldsm4(w, kb + kv_tile_off<S::row>(S::step, 8 * n + mr, 16 * (4 * i + mm)));
#pragma unroll
                            for (int k = 0; k < 2; ++k) slice(c[n], 2 * i + k, w[2 * k], w[2 * k + 1]);
                        }
                }
                // ---- softmax: element (n, e) is row g + 8 (e / 2), token j0 + 8 n + 2 t + e % 2
                const bool whole = there == (1u << kGr) - 1u && all_see(a, tile, j0, S::step);
                float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int n = 0; n < 2 * kGr; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[n][e] *= sc[n >> 1][e >> 1];
                if (!whole)   // rows not in use may see what they like
#pragma unroll
                    for (int n = 0; n < 2 * kGr; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!(there >> (n >> 1) & 1u) || !sees(a, pos[e >> 1], j0 + 8 * n + 2 * t + (e & 1)))
                                c[n][e] = -INFINITY;
#pragma unroll
                for (int n = 0; n < 2 * kGr; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], c[n][e]);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    top[r] = fmaxf(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], 1));
                    top[r] = fmaxf(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], 2));
                }
                float vmax = 0.f;
                if (FMT == KDA_KV_I8)
#pragma unroll
                    for (int y = 0; y < kGr; ++y) vmax = vs[y] < INFINITY ? fmaxf(vmax, vs[y]) : vmax;
                const bool scaled = FMT == KDA_KV_I8 && vmax > ref;
                if (__any_sync(0xFFFFFFFFu, top[0] > m[0] || top[1] > m[1] || scaled)) {
                    float f[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float mn = fmaxf(m[r], top[r]);
                        f[r] = mn == -INFINITY ? 1.f : ex2(m[r] - mn);
                        l[r] *= f[r];
                        m[r] = mn;
                    }
                    if (scaled) {
                        const float rn = fmaxf(vmax, kMinRef), k = ref / rn;
                        f[0] *= k, f[1] *= k;
                        ref = rn;
                        inv_ref = kPScale / rn;
                    }
#pragma unroll
                    for (int j = 0; j < kNt; ++j) o[j][0] *= f[0], o[j][1] *= f[0], o[j][2] *= f[1], o[j][3] *= f[1];
                }
                const float mx[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
                bool strange = false;   // a value scale that is no number: 0 times it must stay 0
                float pv[kGr];          // what a group's probabilities are multiplied by before rounding
#pragma unroll
                for (int y = 0; y < kGr; ++y) {
                    pv[y] = 1.f;
                    if (FMT == KDA_KV_I8) {
                        pv[y] = vs[y] * inv_ref;
                        if (!(vs[y] < INFINITY)) strange = true, pv[y] = NAN;
                    }
                }
                uint32_t pa[kGr][4][NT];
#pragma unroll
                for (int n = 0; n < 2 * kGr; ++n) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        c[n][e] = ex2(c[n][e] - mx[e >> 1]);
                        l[e >> 1] += c[n][e];
                    }
                    if (FMT == KDA_KV_I8) {
                        if (strange)
#pragma unroll
                            for (int e = 0; e < 4; ++e) c[n][e] = c[n][e] == 0.f ? 0.f : c[n][e] * pv[n >> 1];
                        else
#pragma unroll
                            for (int e = 0; e < 4; ++e) c[n][e] *= pv[n >> 1];
                    }
                    split2<FMT, NT>(c[n][0], c[n][1], pa[n >> 1][2 * (n & 1)]);
                    split2<FMT, NT>(c[n][2], c[n][3], pa[n >> 1][2 * (n & 1) + 1]);
                }
                // ---- values
                auto values = [&]() {
#pragma unroll
                    for (int y = 0; y < kGr; ++y) {
#pragma unroll
                        for (int i = 0; i < S::row / 32; ++i) {
                            uint32_t w[4];   // (tokens 0-7, 8-15) of 16-byte units 2 i and 2 i + 1
                            ldsm4t(w, vb + kv_tile_off<S::row>(S::step, 16 * y + 8 * (mm & 1) + mr, 16 * (2 * i + (mm >> 1))));
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                if constexpr (FMT == KDA_KV_I8) {
                                    // a register holds columns 2 g, 2 g + 1 of two tokens: the even ones
                                    // make one output tile, the odd ones the next
                                    const uint32_t b0 = w[2 * x] ^ 0x80808080u, b1 = w[2 * x + 1] ^ 0x80808080u;
#pragma unroll
                                    for (int z = NT - 1; z >= 0; --z) {
                                        const uint32_t f[4] = {pa[y][0][z], pa[y][1][z], pa[y][2][z], pa[y][3][z]};
                                        mma<FMT>(o[2 * (2 * i + x)], f, half2_of<0x4240>(b0), half2_of<0x4240>(b1));
                                        mma<FMT>(o[2 * (2 * i + x) + 1], f, half2_of<0x4341>(b0), half2_of<0x4341>(b1));
                                    }
                                } else {
#pragma unroll
                                    for (int z = NT - 1; z >= 0; --z) {
                                        const uint32_t f[4] = {pa[y][0][z], pa[y][1][z], pa[y][2][z], pa[y][3][z]};
                                        mma<FMT>(o[2 * i + x], f, w[2 * x], w[2 * x + 1]);
                                    }
                                }
                            }
                        }
                    }
                };
                bool odd = false;
                if constexpr (FMT == KDA_KV_BF16) {
                    // A token that a row does not see has probability 0, but 0 times an infinity or a
                    // NaN is not 0 (stale slots past the end, or a value the row must not know of).
                    // Where a step is not seen whole, look for such a value first.
                    if (!whole) {
                        uint32_t bad = 0;
                        for (int i = lane; i < S::tile / 16; i += 32) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(buf + S::tile + 16 * i);
                            for (uint32_t y : {x.x, x.y, x.z, x.w})
                                bad |= (uint32_t)((y & 0x7F80u) == 0x7F80u) | (uint32_t)((y & 0x7F800000u) == 0x7F800000u);
                        }
                        odd = __any_sync(0xFFFFFFFFu, bad != 0);
                    }
                }
                if (!odd) {
                    values();
                } else if constexpr (FMT == KDA_KV_BF16) {
                    // one product for each query token, without the tokens it does not see, of which
                    // only that token's rows are kept
                    for (int32_t q = tile.pmin; q <= tile.pmax; ++q) {
                        uint32_t keep[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int j = j0 + 8 * i + 2 * t;
                            keep[i] = (sees(a, q, j) ? 0xFFFFu : 0u) | (sees(a, q, j + 1) ? 0xFFFF0000u : 0u);
                        }
#pragma unroll
                        for (int i = 0; i < kNt; ++i) {
                            uint32_t w[4];
                            ldsm4t(w, vb + kv_tile_off<S::row>(S::step, 8 * (mm & 1) + mr, 16 * i));
                            float d[4] = {};
#pragma unroll
                            for (int z = NT - 1; z >= 0; --z) {
                                const uint32_t f[4] = {pa[0][0][z], pa[0][1][z], pa[0][2][z], pa[0][3][z]};
                                mma<FMT>(d, f, w[0] & keep[0], w[1] & keep[1]);
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (pos[e >> 1] == q) o[i][e] += d[e];
                        }
                    }
                }
            }
            pin(o);
            __syncwarp();
            load_next(stage);
            if (++stage == stages) stage = 0, phase ^= 1;
        }

        // ---- the warps' results together
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
            if (t == 0) {
                ml[(warp * 16 + g + 8 * r) * 2] = m[r];
                ml[(warp * 16 + g + 8 * r) * 2 + 1] = l[r];
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = g + 8 * r;
            if (row >= tile.nrows) continue;
            float mt = -INFINITY;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) mt = fmaxf(mt, ml[(i * 16 + row) * 2]);
            float f = mt == -INFINITY ? 1.f : exp2f(m[r] - mt);
            if (FMT == KDA_KV_I8) f *= ref * (1.f / kPScale);
            float *dst = acc + (warp * 16 + row) * D;
            if constexpr (FMT == KDA_KV_I8) {
#pragma unroll
                for (int i = 0; i < kNt / 2; ++i)   // columns 16 i + 4 t ..: even and odd ones from two tiles
                    *reinterpret_cast<float4 *>(dst + 4 * acc_unit<FMT, D>(row, 4 * i + t)) =
                        make_float4(o[2 * i][2 * r] * f, o[2 * i + 1][2 * r] * f, o[2 * i][2 * r + 1] * f,
                                    o[2 * i + 1][2 * r + 1] * f);
            } else {
#pragma unroll
                for (int j = 0; j < kNt; ++j)
                    *reinterpret_cast<float2 *>(dst + 4 * acc_unit<FMT, D>(row, 2 * j + (t >> 1)) + 2 * (t & 1)) =
                        make_float2(o[j][2 * r] * f, o[j][2 * r + 1] * f);
            }
        }
        __syncthreads();
        const bool starts = u_first == 0, ends = u_last == tile.units;
        const int part_slot = starts ? 1 : 0;
        for (int i = tid; i < tile.nrows * (D / 4); i += kWarps * 32) {
            const int row = i / (D / 4), unit = i % (D / 4);
            float mt = -INFINITY, lt = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, ml[(w * 16 + row) * 2]);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float lw = ml[(w * 16 + row) * 2 + 1];
                lt += mt == -INFINITY ? lw : lw * exp2f(ml[(w * 16 + row) * 2] - mt);
                const float4 x = *reinterpret_cast<const float4 *>(acc + (w * 16 + row) * D + 4 * acc_unit<FMT, D>(row, unit));
                v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
            }
            if (starts && ends) {
                const int at_row = tile.row0 + row;
                const int64_t at = (int64_t)(tile.q.tok0 + at_row / a.G) * a.Hq + head * a.G + at_row % a.G;
                const float inv = 1.f / lt;
                if (lt == 0.f) v = make_float4(0.f, 0.f, 0.f, 0.f);
                else v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
                store_row4(a.o, a.dtype, at * D + 4 * unit, v);
                if (a.lse && unit == 0) a.lse[at] = lse_of(mt, lt);
            } else {
                float *dst = a.part + ((int64_t)(blockIdx.x * 2 + part_slot) * 16 + row) * kPartRow<D>;
                *reinterpret_cast<float4 *>(dst + 4 * unit) = v;
                if (unit == 0) dst[D] = mt, dst[D + 1] = lt;
            }
        }
        if (tid == 0 && starts && !ends) {
            AttnSplit sp{};
            sp.last_cta = cta_of(end - 1 + (tile.units - u_last) , W, C);
            sp.row_tok = tile.q.tok0;
            sp.head = head;
            sp.row0 = tile.row0;
            sp.nrows = tile.nrows;
            a.split[blockIdx.x] = sp;
        }
        ml += ml_next;
        ml_next = -ml_next;
        if (left > 0) {
            u = 0;
            next_item(tile, head);
        }
    }
}

template <int FMT, int D, int NT>
cudaError_t run(const AttnArgs &a, cudaStream_t st) {
    using M = Smem<FMT, D, NT>;
    static_assert(M::total(Shape<FMT, D>::deep_stages) + 1024 <= 227 * 1024, "shared memory");
    static_assert(M::total(Shape<FMT, D>::stages) <= 113 * 1024, "two CTAs an SM");
    const int smem = M::total(a.deep ? Shape<FMT, D>::deep_stages : Shape<FMT, D>::stages) + 1024;
    auto kern = attn_decode_kernel<FMT, D, NT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<a.ctas, kWarps * 32, smem, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess || a.whole) return e;
    // the join is placed while the last CTAs run and waits for them in hardware
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.ctas, 4);
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<D, kAttnDecodeRows>, a);
}

}  // namespace

cudaError_t launch_attn_decode(const AttnArgs &a, cudaStream_t s) {
    const bool i8 = a.kv.fmt == KDA_KV_I8, f32 = a.dtype == KDA_F32;
    if (a.kv.d == 128) {
        if (i8) return f32 ? run<KDA_KV_I8, 128, 2>(a, s) : run<KDA_KV_I8, 128, 1>(a, s);
        return f32 ? run<KDA_KV_BF16, 128, 3>(a, s) : run<KDA_KV_BF16, 128, 1>(a, s);
    }
    if (i8) return f32 ? run<KDA_KV_I8, 64, 2>(a, s) : run<KDA_KV_I8, 64, 1>(a, s);
    return f32 ? run<KDA_KV_BF16, 64, 3>(a, s) : run<KDA_KV_BF16, 64, 1>(a, s);
}

}  // namespace kda
