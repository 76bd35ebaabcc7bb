// Attention of few query rows over the paged cache (decoding, drafts; every float32 call).
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j - m_i), j over the visible tokens
//
// in one pass over the cache with a running maximum and sum per row.  Bound: the cache's bytes.
// The rows of a group (query heads that share a key/value head, times the call's tokens) are the
// N = 8 of a warp-level matrix product (twice, for up to 16 rows), tokens and columns its M = 16:
//   S^T = K Q^T,  O^T += V^T P^T
// so a cached byte is read once for all rows; wider tensor-memory tiles would stand empty here.  With
// the rows as M, eight of them left half of every product empty, and 64 products a step at 11
// cycles each (measured, saturated) took half of the time that the bytes take.
//
// Two CTAs an SM, so that one streams while the other joins its warps or starts an item.  A fifth
// warp walks the list of units and copies them into a ring of stages (bulk copies: 16 tokens lie in
// one page, and a page's rows are contiguous); with each warp aiming its own copies the bookkeeping
// was 40% of the instructions.  The other four take a step of a unit's tokens each (32 of the 8-bit
// cache, 16 of the 16-bit one) and run alone, with their own maxima, sums and 16 x D accumulators.
// They meet only at a piece's beginning, to split its queries, and at its end.
//
// Measured (d = 128): 32 contexts of 512 to 32768 tokens, 8-bit: 202 us, 6.0 TB/s, 90% of the copy
// rate; one of 1,048,576 tokens: 185 us, 87%; 256 requests through a window of 1024, 16-bit: 172 us,
// 87%.  4 float32 drafts of 24 requests, 8-bit, d = 64: 33 us, where the products count (three or six
// for each of the 16-bit forms' one) and the split leaves 1.5 steps a warp.
//
// 8-bit cache: codes c become fp16 exactly (the byte under the exponent of 1024, less 1152), a
// query row is scaled by a power of two into fp16's range, so q . c carries no rounding beyond
// fp32 sums, and the block's key scale multiplies the score.  The value scale goes into the
// probabilities: p vs 2^6 in fp16, relative to the largest p vs that the row has seen (to within 2^8).
// A token 2^19 times below that loses bits and one 2^30 below adds nothing; what a row does not see, or
// sees without weight, costs it none.
//
// float32 calls: queries and probabilities are split into three bf16 terms, which keep all 24 bits over
// fp32's range; codes are exact in bf16.  (Two fp16 terms hold 22, and fewer the further a
// probability times its value scale lies below the largest.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"

namespace kda {
namespace {

using namespace attn;

constexpr int kWarps = 4;                             // that compute; one more walks and copies
constexpr float kPBits = 6.f;                         // bits that a probability is scaled up in fp16
constexpr float kGrow = 8.f;                          // bits that a row's maximum may grow before O is rescaled
constexpr float kTiny = 0x1p-149f;                    // stands for a score's factor of 0

template <int FMT, int D>
struct Shape {
    static constexpr int row = kKvRow<FMT, D>;
    static constexpr int line = row < 128 ? row : 128, blocks = row / line;
    static constexpr int step = FMT == KDA_KV_I8 ? 32 : 16, groups = step / 16, unit = kWarps * step;
    static constexpr int tile = row * unit;           // keys or values of a unit, by line block as in a page
    static constexpr int stage = 2 * tile + 128;      // and 16 bytes of scales for each 16 tokens
    static constexpr int stages = D == 128 ? 3 : 6;        // of the ring, two CTAs an SM
};

// A unit of work.
struct Job {
    int32_t j0, flags, base, row0, nrows, tok0, head;   // first token; the row tile
    uint32_t live, whole;                               // groups that are there; warps whose rows see all of theirs
    uint32_t lead;                                      // 4 bits a group: the group that its scales came with
    int32_t pmin, pmax;
};

template <int FMT, int D, int NT, int NR>
struct Smem {
    // behind the ring
    static constexpr int o_acc = 0;                                      // [kWarps][4][D] fp32
    static constexpr int o_ml = o_acc + kWarps * 4 * D * 4;             // [2][kWarps][16][2] fp32
    static constexpr int o_q = o_ml + 2 * kWarps * 16 * 8;               // fragments of the queries
    static constexpr int o_qs = o_q + NT * NR * (D / 16) * 256;          // [16] row factors
    static constexpr int o_drafts = o_qs + 64;                           // trees: [16] what each row sees
    static constexpr int o_job = o_drafts + (kTree ? 16 * (int)sizeof(Draft) : 0);
    static constexpr int o_bar = o_job + Shape<FMT, D>::stages * (int)sizeof(Job);   // full, empty
    static constexpr int o_err = o_bar + 2 * Shape<FMT, D>::stages * 8;
    static constexpr int total(int stages) { return stages * Shape<FMT, D>::stage + o_err + 64; }
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
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
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

// Two codes (bytes selected by SEL) as the product's type, both exact.  fp16: under the exponent byte 0x64
// a biased code, b = code + 128, is 1024 + b, less 1152.  bf16: under 0x43 a code's low seven bits are
// 128 + those, less 128 or, where the sign bit is set, 256.
template <bool F16, uint32_t SEL>
__device__ __forceinline__ uint32_t codes2(uint32_t c) {
    if constexpr (F16) {
        const uint32_t u = __byte_perm(c, 0x64646464u, SEL);
        const uint32_t k = 0x64806480u;   // 1152, 1152
        const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&u), *reinterpret_cast<const __half2 *>(&k));
        return *reinterpret_cast<const uint32_t *>(&r);
    } else {
        const uint32_t x = __byte_perm(c, 0x43434343u, SEL), u = x & 0xFF7FFF7Fu, k = x & 0xFF80FF80u;
        const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&u), *reinterpret_cast<const __nv_bfloat162 *>(&k));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
}

// x (already in range) as NT packed terms of the product's type whose sum is x to NT times its bits.
template <bool F16, int NT>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&out)[NT]) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        if constexpr (F16) {
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

// Place of the 4-float unit u of a row of the warps' accumulators in shared memory: a warp stores 64
// bytes of four pairs of rows at a time, which so fall into different banks.
__device__ __forceinline__ int acc_unit(int row, int u) { return u ^ (row >> 1 & 3) << 2; }

// The transpose of an 8 x 8 tile of 16-bit values, held as a product's fragment.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// The share of this CTA (left = 0: none), found by one warp: the units of all sequences summed, then
// the sequence, row tile, head and unit where the share begins.
template <int UNIT>
__device__ __forceinline__ Walk find_share(const AttnArgs &a, int lane, int64_t &W, int32_t &C) {
    constexpr int R = kAttnDecodeRows;
    auto seq_units = [&](int s) {
        const KvSeq q = seq_of(a, s);
        const int n = tiles_of<R>(a, q);
        int64_t w = 0;
#pragma unroll 1
        for (int i = 0; i < n; ++i) w += make_tile<R, UNIT>(a, s, q, i).units;
        return w * a.kv.Hkv;
    };
    Walk w{};
    W = 0;
#pragma unroll 1
    for (int s = lane; s < a.nseq; s += 32) W += seq_units(s);
    for (int i = 16; i; i >>= 1) W += __shfl_xor_sync(0xFFFFFFFFu, W, i);
    C = (int32_t)min((int64_t)a.ctas, W);   // no CTA that takes part is without a unit
    if ((int32_t)blockIdx.x >= C) return w;
    const int64_t begin = (int64_t)blockIdx.x * W / C, end = (int64_t)(blockIdx.x + 1) * W / C;
    w.left = end - begin;
    int64_t at = begin;
    int s0 = 0;
#pragma unroll 1
    for (int base = 0;; base += 32) {
        const int64_t mine = base + lane < a.nseq ? seq_units(base + lane) : 0;
        int64_t x = mine;
        for (int i = 1; i < 32; i <<= 1) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, i);
            if (lane >= i) x += y;
        }
        const uint32_t hit = __ballot_sync(0xFFFFFFFFu, at < x);
        const int f = hit ? __ffs(hit) - 1 : 31;
        at -= __shfl_sync(0xFFFFFFFFu, hit ? x - mine : x, f);
        s0 = base + f;
        if (hit) break;
    }
    const KvSeq q = seq_of(a, s0);
#pragma unroll 1
    for (int rt = 0;; ++rt) {
        w.t = make_tile<R, UNIT>(a, s0, q, rt);
        if (at < (int64_t)w.t.units * a.kv.Hkv) break;
        at -= (int64_t)w.t.units * a.kv.Hkv;
    }
    w.h = (int32_t)(at / w.t.units);
    w.u = (int32_t)(at % w.t.units);
    return w;
}

// NT: terms of a split operand; NR: tiles of eight rows.
template <int FMT, int D, int NT, int NR>
__global__ void __launch_bounds__((kWarps + 1) * 32, 2) attn_decode_kernel(const __grid_constant__ AttnArgs a) {
    using S = Shape<FMT, D>;
    using M = Smem<FMT, D, NT, NR>;
    constexpr int kKs = D / 16;   // 16-wide slices of a row
    constexpr int kDt = D / 16;   // 16-column output tiles
    constexpr int kGr = S::groups;
    constexpr bool kRegQ = NT == 1;   // query fragments stay in registers
    constexpr bool kF16 = FMT == KDA_KV_I8 && NT == 1;   // the products' type: fp16, or bf16
    // Terms of a probability.  bf16 calls over the 16-bit cache split them in two, which keep 16 bits: one term
    // of 8 took a third of the outputs off their nearest bf16 (2.2e-3 of their size instead of 1.66e-3) and
    // saved nothing, as the bytes bound these calls (256 windowed requests 173.4 and 173.7 us; 16 rows a head
    // 103 and 107).
    constexpr int kPt = NT == 1 && !kF16 ? 2 : NT;
    constexpr uint32_t kBias = kF16 ? 0x80808080u : 0u;  // of a code that codes2() takes
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = ptx::smem_align1024(smem_raw);
    constexpr int stages = S::stages - (NT > 1);
    uint8_t *sm = ring + stages * S::stage;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane >> 2, t = lane & 3;
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + M::o_bar), *empty = full + S::stages;
    Job *jobs = reinterpret_cast<Job *>(sm + M::o_job);
    volatile int *err = reinterpret_cast<int *>(sm + M::o_err);
    if (tid == 0) {
        for (int i = 0; i < stages; ++i) {
            ptx::mbar_init(&full[i], 1);
            ptx::mbar_init(&empty[i], kWarps);
        }
        *err = 0;
    }
    ptx::fence_mbar_init();
    __syncthreads();
    ptx::grid_dep_wait();

    if (warp == kWarps) {
        // ====================================================== the list of units, and their copies
        constexpr int kGroups = kWarps * kGr;
        const int pt = a.kv.page_tokens;
        Walk w{};
        int64_t W = 0;
        int32_t C = 0;
        if (a.whole) {
            // CTA i is item i: key/value head i % Hkv of sequence i / Hkv (one row tile a sequence)
            const KvSeq q = seq_of(a, blockIdx.x / a.kv.Hkv);
            if (q.n > 0) {
                w.h = blockIdx.x % a.kv.Hkv;
                w.t = make_tile<kAttnDecodeRows, S::unit>(a, blockIdx.x / a.kv.Hkv, q, 0);
                w.left = w.t.units;
            }
        } else {
            w = find_share<S::unit>(a, lane, W, C);
            if (lane == 0) a.split[blockIdx.x].last_cta = -1;
        }
        // Units go in batches of up to kBatch of one item: lane i looks up the page of group i % kGroups of
        // the batch's unit i / kGroups, and the next batch is looked up while this one is copied.
        constexpr int kBatch = 32 / kGroups;
        struct Look {
            int32_t n, page, slot;
            bool want;
        };
        auto look = [&](const Walk &x) {
            Look r{0, 0, 0, false};
            if (x.left <= 0) return r;
            r.n = (int32_t)min((int64_t)min(kBatch, x.t.units - x.u), x.left);
            const int32_t j = unit_token<S::unit>(x.t, x.u + lane / kGroups) + lane % kGroups * 16, b = j / pt;
            r.slot = j - b * pt;
            r.want = lane / kGroups < r.n && any_sees(a, x.t, j, 16);
            if (r.want) r.page = __ldg(a.kv.table + (int64_t)x.t.s * a.kv.max_pages + b);
            return r;
        };
        int32_t u_first = w.u;
        Look now = look(w);
        int stage = 0;
        uint32_t phase = 1;
        int64_t asked = 0;   // units whose copies were started
        bool ok = true;
        while (ok && now.n > 0) {
            Walk next = w;
            next.left -= now.n;
            next.u += now.n;
            if (next.left > 0 && next.u == w.t.units) next_item<kAttnDecodeRows, S::unit>(a, next);
            const Look then = look(next);
            const Tile &x = w.t;
#pragma unroll 1
            for (int k = 0; k < now.n; ++k) {
                ok = __all_sync(0xFFFFFFFFu, wait_bar(&empty[stage], phase, err));
                if (!ok) break;
                const int32_t u = w.u + k, j0 = unit_token<S::unit>(x, u), from = k * kGroups + lane;
                const int64_t left = w.left - k;
                const int32_t page = __shfl_sync(0xFFFFFFFFu, now.page, from), slot = __shfl_sync(0xFFFFFFFFu, now.slot, from);
                const bool want = __shfl_sync(0xFFFFFFFFu, (int)now.want, from) && lane < kGroups;
                const uint8_t *rec = want ? kv_record(a.kv, page, w.h) : nullptr;
                const uint32_t live = __ballot_sync(0xFFFFFFFFu, rec != nullptr);
                // A page's groups that follow one another go in one copy, which the first of them starts: a
                // copy costs some 100 cycles to start, whatever its size.
                const bool leads = rec && (lane == 0 || slot == 0 || !(live >> (lane - 1) & 1u));
                const uint32_t leaders = __ballot_sync(0xFFFFFFFFu, leads);
                const int first = 31 - __clz(leaders & (2u << lane) - 1u | 1u);   // this group's leader
                const uint32_t stop = (leaders | ~live) & ~((2u << lane) - 1u) | 1u << kGroups;
                const uint32_t run = __ffs(stop) - 1 - lane;                      // a leader's groups
                uint32_t lead = lane < kGroups ? (uint32_t)first << (4 * lane) : 0u;
                lead = __reduce_or_sync(0xFFFFFFFFu, lead);
                const uint32_t whole = __ballot_sync(0xFFFFFFFFu, lane < kWarps && all_see(a, x, j0 + lane * S::step, S::step));
                if (lane == 0) {
                    Job &jb = jobs[stage];
                    const bool ends = left >= x.units - u;   // the item's last unit is in this share
                    jb.j0 = j0;
                    jb.flags = piece_flags(u - u_first, u + 1 == x.units || left == 1) | (u_first == 0 ? kStarts : 0) | (ends ? kEnds : 0);
                    jb.base = x.q.len - x.q.n;
                    jb.row0 = x.row0, jb.nrows = x.nrows, jb.tok0 = x.q.tok0, jb.head = w.h;
                    jb.live = live, jb.whole = whole, jb.lead = lead;
                    jb.pmin = x.pmin, jb.pmax = x.pmax;
                    if (u_first == 0 && !ends && left == 1) {
                        AttnSplit sp{};
                        sp.last_cta = cta_of((int64_t)(blockIdx.x + 1) * W / C - 1 + (x.units - 1 - u), W, C);
                        sp.row_tok = x.q.tok0;
                        sp.head = w.h;
                        sp.row0 = x.row0;
                        sp.nrows = x.nrows;
                        a.split[blockIdx.x] = sp;
                    }
                    ptx::mbar_arrive_expect_tx(&full[stage], __popc(live) * 2 * 16 * S::row + (FMT == KDA_KV_I8 ? __popc(leaders) * 16 : 0));
                }
                __syncwarp();
                if (leads) {
                    uint8_t *dst = ring + stage * S::stage + lane * 16 * S::line;
                    const uint8_t *src = rec + slot * S::line;
#pragma unroll
                    for (int v = 0; v < 2; ++v)
#pragma unroll
                        for (int b = 0; b < S::blocks; ++b)
                            ptx::bulk_load(dst + v * S::tile + b * S::unit * S::line, src + v * pt * S::row + b * pt * S::line,
                                           run * 16 * S::line, &full[stage]);
                    if (FMT == KDA_KV_I8)
                        ptx::bulk_load(ring + stage * S::stage + 2 * S::tile + 16 * lane, rec + 2 * pt * S::row, 16, &full[stage]);
                }
                ++asked;
                if (++stage == stages) stage = 0, phase ^= 1;
            }
            if (next.u == 0) u_first = 0;
            w = next;
            now = then;
        }
        ok = ok && __all_sync(0xFFFFFFFFu, wait_bar(&empty[stage], phase, err));
        if (ok) {
            if (lane == 0) {
                jobs[stage].flags = kStop;
                ptx::mbar_arrive(&full[stage]);
            }
        } else {   // the copies under way land before the block ends
            for (int64_t i = max((int64_t)0, asked - stages); i < asked; ++i)
                wait_bar(&full[i % stages], (uint32_t)(i / stages) & 1u, nullptr);
        }
        return;
    }

    // ========================================================== the warps that compute
    float *ml = reinterpret_cast<float *>(sm + M::o_ml);   // of this item; the last one's may still be read
    int ml_next = kWarps * 32;
    float *acc = reinterpret_cast<float *>(sm + M::o_acc);
    uint32_t *qfrag = reinterpret_cast<uint32_t *>(sm + M::o_q);
    float *qs = reinterpret_cast<float *>(sm + M::o_qs);
    Draft *drafts = reinterpret_cast<Draft *>(sm + M::o_drafts);
    // The four warps meet; false where one has left, or is about to.  A warp that leaves sets the error
    // first and then arrives once more: the others, each at this meeting or on its way there, get through
    // it and find the error, so that no barrier holds anyone for good.
    auto meet = [&]() {
        asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
        return *err == 0;
    };
    bool ok = true;
    // Where a lane's addresses for the fragment loads lie in a stage.  Row mr of matrix mm: for the keys
    // of the 8-bit cache, tokens 8 (mm % 2) + mr and unit mm / 2 (two slices); of the 16-bit one, the
    // same (a slice is two units); for its values, tokens 8 (mm / 2) + mr and unit mm % 2; for those of
    // the 8-bit cache, tokens 8 (mm % 2) + mr and unit mm / 2.  Other units are an exclusive-or away.
    const int mr = lane & 7, mm = lane >> 3;
    const uint32_t k_at = kv_tile_off<S::row>(S::unit, warp * S::step + 8 * (mm & 1) + mr, 16 * (mm >> 1));
    const uint32_t v_at = S::tile + (FMT == KDA_KV_I8 ? k_at : kv_tile_off<S::row>(S::unit, warp * S::step + 8 * (mm >> 1) + mr, 16 * (mm & 1)));
    constexpr uint32_t kLine = S::line;
    auto unit = [](uint32_t at, int u) { return (at ^ (u & 7) << 4) + (u >> 3) * S::unit * 128; };   // u even or a multiple of 4
    int stage = 0;
    uint32_t phase = 0;
    // This lane's rows are 8 x + 2 t and the one after, x < NR.
    uint32_t qb[kRegQ ? kKs : 1][NR][2];
    float rs[NR][2];
    int32_t pos[NR][2], nrows = 0, row0 = 0, tok0 = 0, head = 0;   // the item
    float o[NR][kDt][4], m[NR][2], l[NR][2], big[NR][2];   // big: 8-bit, the reference of probability times value scale
    for (;;) {
        ok = __all_sync(0xFFFFFFFFu, wait_bar(&full[stage], phase, err));
        if (!ok) break;
        const Job &jb = jobs[stage];
        const int32_t flags = jb.flags;
        if (flags & kStop) break;
        if (flags & kBegin) {
            nrows = jb.nrows, row0 = jb.row0, tok0 = jb.tok0, head = jb.head;
            // The item's queries as fragments: eight threads a row, who agree on its factor.  Columns go
            // where the fragment wants them: pairs of a lane's four bytes of a key for the 8-bit cache.
            constexpr int kCols = D / 8;
            const int row = tid / 8, c0 = tid % 8 * kCols, at = row0 + row;
            float x[kCols];
#pragma unroll
            for (int i = 0; i < kCols; ++i) x[i] = 0.f;
            if (row < nrows) {
                const int32_t tok = token_of(a, at);
                const int64_t off = (int64_t)(tok0 + tok) * a.q_stride + (int64_t)(head * a.G + at - tok * a.G) * D + c0;
#pragma unroll
                for (int i = 0; i < kCols; i += 8) {
                    if (NT > 1) {
                        const float4 u = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + off + i);
                        const float4 v = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + off + i + 4);
                        x[i] = u.x, x[i + 1] = u.y, x[i + 2] = u.z, x[i + 3] = u.w;
                        x[i + 4] = v.x, x[i + 5] = v.y, x[i + 6] = v.z, x[i + 7] = v.w;
                    } else {
                        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) + off + i);
                        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            x[i + 2 * y] = __uint_as_float(w[y] << 16);
                            x[i + 2 * y + 1] = __uint_as_float(w[y] & 0xFFFF0000u);
                        }
                    }
                }
            }
            const float sign = a.scale < 0.f ? -1.f : 1.f;   // goes to the query: factors are positive
            float f = a.scale * sign * kLog2e;
            if (FMT == KDA_KV_BF16 && f == 0.f) f = kTiny;
#pragma unroll
            for (int i = 0; i < kCols; ++i) x[i] *= sign;
            if (FMT == KDA_KV_I8) {
                // a power of two that brings the row's largest magnitude to [2^10, 2^11)
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < kCols; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
                for (int i = 1; i < 8; i <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));
                const int e = (int)(__float_as_uint(top) >> 23);
                const int shift = e == 0 || e == 255 ? 0 : min(max(137 - e, -120), 120);
                const float up = __uint_as_float((uint32_t)(127 + shift) << 23);
#pragma unroll
                for (int i = 0; i < kCols; ++i) x[i] *= up;
                f *= __uint_as_float((uint32_t)(127 - shift) << 23);
            }
            if (tid % 8 == 0) qs[row] = f;
            if (kTree && tid % 8 == 1)
                drafts[row] = row < nrows ? draft_of(a, tok0, jb.pmax + 1 - jb.base, jb.base, token_of(a, at)) : Draft{0, jb.base};
#pragma unroll
            for (int i = 0; i < kCols; i += 2) {
                const int c = (c0 + i) % 16, k = (c0 + i) / 16;
                const int tt = FMT == KDA_KV_I8 ? c / 4 : c % 8 / 2, half = FMT == KDA_KV_I8 ? c / 2 % 2 : c / 8;
                uint32_t z[NT];
                split2<kF16, NT>(x[i], x[i + 1], z);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (row < 8 * NR) qfrag[(((n * kKs + k) * NR + row / 8) * 32 + row % 8 * 4 + tt) * 2 + half] = z[n];
            }
            ok = meet();
            if (!ok) break;
            if constexpr (kRegQ) {
#pragma unroll
                for (int k = 0; k < kKs; ++k)
#pragma unroll
                    for (int x = 0; x < NR; ++x) {
                        const uint2 u = *reinterpret_cast<const uint2 *>(qfrag + ((k * NR + x) * 32 + lane) * 2);
                        qb[k][x][0] = u.x, qb[k][x][1] = u.y;
                    }
            }
#pragma unroll
            for (int x = 0; x < NR; ++x) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int row = 8 * x + 2 * t + r;
                    rs[x][r] = qs[row];
                    pos[x][r] = row < nrows ? (kTree ? 0 : jb.base) + token_of(a, row0 + row) : -1;   // trees: the draft
                    m[x][r] = big[x][r] = -INFINITY, l[x][r] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < kDt; ++j) o[x][j][0] = o[x][j][1] = o[x][j][2] = o[x][j][3] = 0.f;
            }
        }
        const uint32_t there = jb.live >> (warp * kGr) & ((1u << kGr) - 1u);
        if (there) {
            const int32_t j0 = jb.j0 + warp * S::step;
            const uint8_t *buf = ring + stage * S::stage;
            uint32_t kb = ptx::smem_u32(buf);
            asm volatile("" : "+r"(kb)::"memory");
            float ks[kGr], vs[kGr];   // a group's scales; the key's goes into the score factors
            bool strange = false;     // a scale that is no number: what a row does not see must stay 0
#pragma unroll
            for (int y = 0; y < kGr; ++y) {
                ks[y] = 1.f, vs[y] = 0.f;
                if (FMT == KDA_KV_I8 && (there >> y & 1u)) {
                    const float2 f = *reinterpret_cast<const float2 *>(buf + 2 * S::tile +
                                                                       16 * (jb.lead >> (4 * (warp * kGr + y)) & 15u));
                    ks[y] = fabsf(f.x) < INFINITY ? fabsf(f.x) : NAN;   // an infinity reads as NaN whatever the codes
                    vs[y] = fabsf(f.y);
                    strange |= !(ks[y] < INFINITY && vs[y] < INFINITY);
                }
            }
            // ---- scores: c[y][x][e] is token j0 + 16 y + g + 8 (e / 2), row 8 x + 2 t + e % 2
            float c[kGr][NR][4] = {};
            auto slice = [&](int y, int k, const uint32_t (&af)[4]) {
#pragma unroll
                for (int x = 0; x < NR; ++x) {
                    if constexpr (kRegQ) {
                        mma<kF16>(c[y][x], af, qb[k][x][0], qb[k][x][1]);
                    } else {
#pragma unroll
                        for (int z = NT - 1; z >= 0; --z) {
                            const uint2 f = *reinterpret_cast<const uint2 *>(qfrag + (((z * kKs + k) * NR + x) * 32 + lane) * 2);
                            mma<kF16>(c[y][x], af, f.x, f.y);
                        }
                    }
                }
            };
#pragma unroll
            for (int i = 0; i < S::row / 32; ++i) {
                uint32_t w[kGr][4];   // 16-byte units 2 i and 2 i + 1 of tokens 0-7 and 8-15
#pragma unroll
                for (int y = 0; y < kGr; ++y) ldsm4(w[y], kb + unit(k_at, 2 * i) + y * 16 * kLine);
                if constexpr (FMT == KDA_KV_I8) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int y = 0; y < kGr; ++y) {
                            const uint32_t b0 = w[y][2 * k] ^ kBias, b1 = w[y][2 * k + 1] ^ kBias;
                            const uint32_t af[4] = {codes2<kF16, 0x4140>(b0), codes2<kF16, 0x4140>(b1), codes2<kF16, 0x4342>(b0),
                                                    codes2<kF16, 0x4342>(b1)};
                            slice(y, 2 * i + k, af);
                        }
                } else {
#pragma unroll
                    for (int y = 0; y < kGr; ++y) slice(y, i, w[y]);
                }
            }
            // ---- softmax
            // A score's factor.  It is never 0, for a masked score, -infinity, has to stay that.
            auto factor = [&](int y, int x, int r) {
                const float f = rs[x][r] * ks[y];
                return FMT == KDA_KV_I8 && f == 0.f ? kTiny : f;
            };
            const bool whole = there == (1u << kGr) - 1u && (jb.whole >> warp & 1u);
            if (!whole)   // rows not in use may see what they like
#pragma unroll
                for (int y = 0; y < kGr; ++y)
#pragma unroll
                    for (int x = 0; x < NR; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = j0 + 16 * y + g + 8 * (e >> 1);
                            const bool see = kTree ? draft_sees(a, drafts[8 * x + 2 * t + (e & 1)], jb.base, j) : sees(a, pos[x][e & 1], j);
                            if (!(there >> y & 1u) || !see) c[y][x][e] = -INFINITY;
                        }
            // m lags: it only follows a row's maximum when that has grown by more than 2^8.  So does big, which
            // is the same for the scores with log2 of the value scales added: what enters the product stays in
            // fp16's range by what the row itself sees, whatever scales its other blocks have.  Either is a whole
            // number, so that moving it rounds nothing, and moves by the row's own scores alone.
            float top[NR][2], topv[NR][2], lv[kGr];
            bool grown = false;
#pragma unroll
            for (int y = 0; y < kGr; ++y) lv[y] = vs[y] > 0.f && vs[y] < INFINITY ? fmaxf(__log2f(vs[y]), -100.f) : -INFINITY;
#pragma unroll
            for (int x = 0; x < NR; ++x)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    top[x][r] = topv[x][r] = -INFINITY;
#pragma unroll
                    for (int y = 0; y < kGr; ++y) {
                        const float s = fmaxf(c[y][x][r], c[y][x][r + 2]) * factor(y, x, r);
                        top[x][r] = fmaxf(top[x][r], s);
                        if (FMT == KDA_KV_I8) topv[x][r] = fmaxf(topv[x][r], s + lv[y]);
                    }
                    grown |= top[x][r] > m[x][r] + kGrow;
                    if (FMT == KDA_KV_I8) grown |= topv[x][r] > big[x][r] + kGrow;
                }
            if (__any_sync(0xFFFFFFFFu, grown)) {
#pragma unroll
                for (int x = 0; x < NR; ++x) {
                    float f[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
#pragma unroll
                        for (int i = 4; i < 32; i <<= 1) {
                            top[x][r] = fmaxf(top[x][r], __shfl_xor_sync(0xFFFFFFFFu, top[x][r], i));
                            if (FMT == KDA_KV_I8) topv[x][r] = fmaxf(topv[x][r], __shfl_xor_sync(0xFFFFFFFFu, topv[x][r], i));
                        }
                        f[r] = 1.f;
                        if (top[x][r] > m[x][r] + kGrow) {
                            const float mn = ceilf(top[x][r]);
                            f[r] = ex2(m[x][r] - mn);
                            l[x][r] *= f[r];
                            m[x][r] = mn;
                        }
                        if (FMT == KDA_KV_I8) {
                            f[r] = 1.f;
                            if (topv[x][r] > big[x][r] + kGrow) {
                                const float bn = ceilf(topv[x][r]);
                                f[r] = ex2(big[x][r] - bn);
                                big[x][r] = bn;
                            }
                        }
                    }
#pragma unroll
                    for (int j = 0; j < kDt; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[x][j][e] *= f[e & 1];
                }
            }
            // 8-bit: what a probability is multiplied by beside its value scale
            float up[NR][2];
#pragma unroll
            for (int x = 0; x < NR; ++x)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    up[x][r] = FMT == KDA_KV_I8 && big[x][r] != -INFINITY ? ex2(m[x][r] - big[x][r] + kPBits) : 0.f;
            uint32_t pb[kGr][NR][2][kPt];
#pragma unroll
            for (int y = 0; y < kGr; ++y) {
                // probabilities, and what of them is rounded: 8-bit, p vs 2^(m - big + 6).  (Where vs 2^(m - big)
                // is beyond fp32, p is 0.)
#pragma unroll
                for (int x = 0; x < NR; ++x) {
                    float p[4], pv[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) pv[r] = vs[y] < INFINITY ? fminf(vs[y] * up[x][r], 0x1p127f) : NAN;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int r = e & 1;
                        p[e] = ex2(fmaf(c[y][x][e], factor(y, x, r), m[x][r] == -INFINITY ? 0.f : -m[x][r]));
                        if (FMT == KDA_KV_I8 && strange && c[y][x][e] == -INFINITY) p[e] = 0.f;
                        l[x][r] += p[e];
                        if (FMT == KDA_KV_I8) p[e] = strange && c[y][x][e] == -INFINITY ? 0.f : p[e] * pv[r];
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {   // tokens 0-7, 8-15: rows of the transposed operand
                        split2<kF16, kPt>(p[2 * h], p[2 * h + 1], pb[y][x][h]);
#pragma unroll
                        for (int z = 0; z < kPt; ++z) pb[y][x][h][z] = transpose8(pb[y][x][h][z]);
                    }
                }
            }
            // ---- values
            bool odd = false;
            if constexpr (FMT == KDA_KV_BF16) {
                // A token that a row does not see has probability 0, but 0 times an infinity or a NaN is
                // not 0 (stale slots past the end, or a value the row must not know of).  Where a step is
                // not seen whole, look for such a value first.
                if (!whole) {
                    uint32_t bad = 0;
                    for (int i = lane; i < S::step * S::blocks * 8; i += 32) {   // 16-byte units of the warp's rows
                        const uint4 v = *reinterpret_cast<const uint4 *>(buf + S::tile + i / (S::step * 8) * S::unit * 128 +
                                                                         warp * S::step * 128 + 16 * (i % (S::step * 8)));
                        for (uint32_t y : {v.x, v.y, v.z, v.w})
                            bad |= (uint32_t)((y & 0x7F80u) == 0x7F80u) | (uint32_t)((y & 0x7F800000u) == 0x7F800000u);
                    }
                    odd = __any_sync(0xFFFFFFFFu, bad != 0);
                }
            }
            if (!odd) {
#pragma unroll
                for (int y = 0; y < kGr; ++y)
#pragma unroll
                    for (int i = 0; i < S::row / 32; ++i) {
                        uint32_t w[4];   // 16-byte units 2 i and 2 i + 1 of tokens 0-7 and 8-15
                        ldsm4t(w, kb + unit(v_at, 2 * i) + y * 16 * kLine);
                        auto columns = [&](int j, const uint32_t (&af)[4]) {
#pragma unroll
                            for (int x = 0; x < NR; ++x) {
                                if constexpr (NT == 1) {
#pragma unroll
                                    for (int z = kPt - 1; z >= 0; --z) mma<kF16>(o[x][j], af, pb[y][x][0][z], pb[y][x][1][z]);
                                } else {
                                    // the matrix unit's sums are cut, not rounded: over a long context their
                                    // bias came to 2e-6 of a float32 result, so each group's is added here
                                    float d[4] = {};
#pragma unroll
                                    for (int z = kPt - 1; z >= 0; --z) mma<kF16>(d, af, pb[y][x][0][z], pb[y][x][1][z]);
#pragma unroll
                                    for (int e = 0; e < 4; ++e) o[x][j][e] += d[e];
                                }
                            }
                        };
                        if constexpr (FMT == KDA_KV_I8) {
                            // a register holds columns 2 g, 2 g + 1 of two tokens: output tile j has the even
                            // columns of its 16 in rows 0-7 and the odd ones in rows 8-15
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint32_t b0 = w[2 * k] ^ kBias, b1 = w[2 * k + 1] ^ kBias;
                                const uint32_t af[4] = {codes2<kF16, 0x4240>(b0), codes2<kF16, 0x4341>(b0), codes2<kF16, 0x4240>(b1),
                                                        codes2<kF16, 0x4341>(b1)};
                                columns(2 * i + k, af);
                            }
                        } else {
                            columns(i, w);
                        }
                    }
            } else if constexpr (FMT == KDA_KV_BF16) {
                // one product for each query token, without the tokens it does not see, of which only
                // that token's rows are kept
#pragma unroll 1
                for (int32_t q = kTree ? token_of(a, row0) : jb.pmin; q <= (kTree ? token_of(a, row0 + nrows - 1) : jb.pmax); ++q) {
                    uint32_t keep[2];
                    Draft dr{};
                    if (kTree) dr = draft_of(a, tok0, jb.pmax + 1 - jb.base, jb.base, q);
                    auto sees_it = [&](int32_t j) { return kTree ? draft_sees(a, dr, jb.base, j) : sees(a, q, j); };
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int j = j0 + 8 * i + 2 * t;
                        keep[i] = (sees_it(j) ? 0xFFFFu : 0u) | (sees_it(j + 1) ? 0xFFFF0000u : 0u);
                    }
#pragma unroll
                    for (int i = 0; i < kDt; ++i) {
                        uint32_t w[4];
                        ldsm4t(w, kb + unit(v_at, 2 * i));
                        w[0] &= keep[0], w[1] &= keep[0], w[2] &= keep[1], w[3] &= keep[1];
#pragma unroll
                        for (int x = 0; x < NR; ++x) {
                            float d[4] = {};
#pragma unroll
                            for (int z = kPt - 1; z >= 0; --z) mma<kF16>(d, w, pb[0][x][0][z], pb[0][x][1][z]);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (pos[x][e & 1] == q) o[x][i][e] += d[e];
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int x = 0; x < NR; ++x) pin(o[x]);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&empty[stage]);
        if (++stage == stages) stage = 0, phase ^= 1;
        if (!(flags & kEnd)) continue;

        // ---- the warps' results together
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int i = 4; i < 32; i <<= 1) l[x][r] += __shfl_xor_sync(0xFFFFFFFFu, l[x][r], i);
                if (g == 0) {
                    ml[(warp * 16 + 8 * x + 2 * t + r) * 2] = m[x][r];
                    ml[(warp * 16 + 8 * x + 2 * t + r) * 2 + 1] = l[x][r];
                }
            }
        ok = meet();
        // four rows at a time, so that the ring has the room
        const bool starts = flags & kStarts, ends = flags & kEnds;
#pragma unroll
        for (int x = 0; x < NR; ++x) {
            float f[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float mt = -INFINITY;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) mt = fmaxf(mt, ml[(i * 16 + 8 * x + 2 * t + r) * 2]);
                f[r] = mt == -INFINITY ? 1.f : ex2(m[x][r] - mt);
                if (FMT == KDA_KV_I8) f[r] = big[x][r] == -INFINITY ? 0.f : ex2(big[x][r] - kPBits - mt);
            }
#pragma unroll 1
            for (int half = 0; ok && half < 2; ++half) {
                const int base = 8 * x + 4 * half;
                if (base >= nrows) break;
                if (t >> 1 == half) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int row = 2 * (t & 1) + r;
                        float *dst = acc + (warp * 4 + row) * D;
#pragma unroll
                        for (int j = 0; j < kDt; ++j) {
                            const float v0 = o[x][j][r] * f[r], v1 = o[x][j][r + 2] * f[r];
                            if constexpr (FMT == KDA_KV_I8) {   // columns 16 j + 2 g, 2 g + 1
                                *reinterpret_cast<float2 *>(dst + 4 * acc_unit(base + row, 4 * j + (g >> 1)) + 2 * (g & 1)) = make_float2(v0, v1);
                            } else {                            // columns 16 j + g, 16 j + 8 + g
                                dst[4 * acc_unit(base + row, 4 * j + (g >> 2)) + (g & 3)] = v0;
                                dst[4 * acc_unit(base + row, 4 * j + 2 + (g >> 2)) + (g & 3)] = v1;
                            }
                        }
                    }
                }
                ok = meet();
                if (!ok) break;
                // a thread sums 4 columns of a row: D / 4 threads a row
                const int sum_row = base + tid / (D / 4), unit4 = tid % (D / 4);
                if (sum_row < min(nrows, base + 4)) {
                    auto partial = [&]() { return a.part + ((int64_t)(blockIdx.x * 2 + (starts ? 1 : 0)) * 16 + sum_row) * kPartRow<D>; };
                    float top = -INFINITY, lt = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[(w * 16 + sum_row) * 2]);
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float lw = ml[(w * 16 + sum_row) * 2 + 1];
                        lt += top == -INFINITY ? lw : lw * ex2(ml[(w * 16 + sum_row) * 2] - top);
                        const float4 x = *reinterpret_cast<const float4 *>(acc + (w * 4 + (sum_row & 3)) * D +
                                                                           4 * acc_unit(sum_row, unit4));
                        v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
                    }
                    if (flags & kAgain) {   // to an earlier piece's
                        const float *was = partial();
                        const float4 u = *reinterpret_cast<const float4 *>(was + 4 * unit4);
                        const float both = fmaxf(top, was[D]), ref = both == -INFINITY ? 0.f : both;
                        const float fv = ex2(top - ref), fu = ex2(was[D] - ref);
                        v = make_float4(v.x * fv + u.x * fu, v.y * fv + u.y * fu, v.z * fv + u.z * fu, v.w * fv + u.w * fu);
                        lt = lt * fv + was[D + 1] * fu;
                        top = both;
                        // a row's threads, of one warp, have read what one of them replaces
                        __syncwarp(D == 128 ? ~0u : 0xFFFFu << (lane & 16));
                    }
                    if (starts && ends && !(flags & kMore)) {
                        const int32_t at_row = row0 + sum_row, tok = token_of(a, at_row);
                        const int64_t at = (int64_t)(tok0 + tok) * a.Hq + head * a.G + at_row - tok * a.G;
                        const float inv = 1.f / lt;
                        if (lt == 0.f) v = make_float4(0.f, 0.f, 0.f, 0.f);
                        else v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
                        store_row4(a.o, a.dtype, at * D + 4 * unit4, v);
                        if (a.lse && unit4 == 0) a.lse[at] = lse_of(top, lt);
                    } else {
                        float *dst = partial();
                        *reinterpret_cast<float4 *>(dst + 4 * unit4) = v;
                        if (unit4 == 0) dst[D] = top, dst[D + 1] = lt;
                    }
                }
                if (base + 4 < nrows) ok = meet();
            }
        }
        if (!ok) break;
        ml += ml_next;
        ml_next = -ml_next;
    }
    if (!ok) {
        if (lane == 0) flag_status(a.kv.status, KDA_DEV_TIMEOUT);
        __syncwarp();
        asm volatile("bar.arrive 1, %0;" ::"n"(kWarps * 32) : "memory");
    }
}

template <int FMT, int D, int NT, int NR>
cudaError_t run_rows(const AttnArgs &a, cudaStream_t st) {
    using M = Smem<FMT, D, NT, NR>;
    // (the split terms of float32 queries leave room for one stage less beside another CTA)
    static_assert(NT > 1 || 2 * (M::total(Shape<FMT, D>::stages) + 2048) <= 228 * 1024, "two CTAs an SM");
    const int smem = M::total(Shape<FMT, D>::stages - (NT > 1)) + 1024;
    auto kern = attn_decode_kernel<FMT, D, NT, NR>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<a.ctas, (kWarps + 1) * 32, smem, st>>>(a);
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

// Up to eight rows a sequence take one tile of rows; the split products of float32 queries, which are
// not bound by bytes, have one form for both.
template <int FMT, int D, int NT>
cudaError_t run(const AttnArgs &a, cudaStream_t st) {
    if constexpr (NT == 1)
        if ((int64_t)a.max_q * a.G <= 8) return run_rows<FMT, D, NT, 1>(a, st);
    return run_rows<FMT, D, NT, 2>(a, st);
}

}  // namespace

#ifdef KDA_ATTN_TREE
cudaError_t launch_attn_tree_decode(const AttnArgs &a, cudaStream_t s) {
#else
cudaError_t launch_attn_decode(const AttnArgs &a, cudaStream_t s) {
#endif
    const bool i8 = a.kv.fmt == KDA_KV_I8, f32 = a.dtype == KDA_F32;
    if (a.kv.d == 128) {
        if (i8) return f32 ? run<KDA_KV_I8, 128, 3>(a, s) : run<KDA_KV_I8, 128, 1>(a, s);
        return f32 ? run<KDA_KV_BF16, 128, 3>(a, s) : run<KDA_KV_BF16, 128, 1>(a, s);
    }
    if (i8) return f32 ? run<KDA_KV_I8, 64, 3>(a, s) : run<KDA_KV_I8, 64, 1>(a, s);
    return f32 ? run<KDA_KV_BF16, 64, 3>(a, s) : run<KDA_KV_BF16, 64, 1>(a, s);
}

}  // namespace kda
