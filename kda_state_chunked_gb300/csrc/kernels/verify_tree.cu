// Trees of drafts against recurrent states.
//
// verify_tree_kernel answers for every draft t of a tree with o_t = S_t^T q_t, S_t the state after the drafts of
// its branch, and keeps no draft's state.  With S_0 the request's state, A_t the product of alpha over t's branch
// (t and its ancestors) and r(t, i) the product over the part of it behind i:
//   S_t = Diag(A_t) S_0 + sum_{i in branch} (r(t, i) k_i) u_i^T
//   u_t = beta_t (v_t - S_0^T (A_t k_t) - sum_{i before t} c_ti u_i)      c_ti = <r(t, i) k_t, k_i>
//   o_t = S_0^T (A_t q_t) + sum_{i up to t} e_ti u_i                      e_ti = <r(t, i) q_t, k_i>
// (decay, delta-rule write, read, in that order).  The products r are formed along the branch and never by a
// division, so an alpha of 0 is like any other.  S_0 is read once, at the start, into registers; a draft costs its
// tokens' bytes and the arithmetic alone, where a state a draft would be written and read again: 2 x 64 KiB a head.
//
// A CTA takes one (request, head):
//   S_0 is asked into L2;  masks of the branches, convolutions along them;
//   sixteen lanes a draft walk its branch towards the root: c_ti, e_ti, A_t k_t, A_t q_t;
//   the products with S_0 (bf16 calls: warp-level matrix products, whose 16 rows fit 8 drafts' k and q; fp32 calls: FMA);
//   then a thread a column solves for u, eight drafts at a time, and all add up o.
//
// Bound: the states' bytes for small trees, the walk and the solve (n^2) for large ones.  Measured, 256 requests x 32
// heads of 128, bf16: trees of 16 drafts 302 us (floor 107: 36%), of 8 222 us, of 4 185 us; 64 requests x 64 drafts
// 547 us.  fp32: 16 drafts 605 us; 48 requests x 16 heads of 64, 1 to 64 drafts, 80 us.  A CTA's chain of dependent
// steps takes some 20 us and four a SM cover each other to 38% of the issue slots.  A thread a state element with
// FMA took 1,462 us for the 16 drafts; branches as bit lists in the solve 478; asking the state of the item one wave
// ahead into L2 cost 45 us and hid nothing.
#include "common.cuh"
#include "sm100_ptx.cuh"
#include "tc_common.cuh"

namespace kda {
namespace {

constexpr int kMost = kTreeMost;

template <class T>
constexpr int kVec = 16 / (int)sizeof(T);   // elements of a 16-byte load

__device__ __forceinline__ void load_vec(const float *p, float (&x)[4]) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void load_vec(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// A request of the call: its first packed row and its drafts; n = -1 where the metadata does not fit.
struct Request {
    int64_t first;
    int32_t n;
};
__device__ __forceinline__ Request request_of(const VerifyTreeArgs &a, int b) {
    const int64_t first = __ldg(a.cu_q + b), end = __ldg(a.cu_q + b + 1);
    if (first < 0 || end < first || end > a.T_tot || end - first > a.max_q) return {0, -1};
    return {first, (int32_t)(end - first)};
}

// Whether a page id of the object lies outside the pool; all threads call it.
__device__ __forceinline__ bool pages_lost(const PoolView &pv, const int32_t *pages) {
    bool lost = false;
    for (int i = threadIdx.x; i < pv.pages_per_object; i += blockDim.x) lost |= (uint32_t)__ldg(pages + i) >= (uint32_t)pv.num_pages;
    return __syncthreads_or(lost) != 0;
}

// Channel c of head h in a packed row of a token tensor, es bytes an element.
__device__ __forceinline__ const uint8_t *raw_at(const VerifyTreeArgs &a, const void *x, int64_t row, int h, int d, int c, int es) {
    return static_cast<const uint8_t *>(x) + ((row * a.H + h) * d + c) * es;
}

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kUnit = 256;   // bytes of a record that lie in one page: pages and records are multiples of it

// Shared memory for trees of up to N drafts (a multiple of 8), in bytes.
template <int D>
struct Lay {
    static constexpr int P = D * 4;   // of a draft's row

    int kb, al, xk, xq, v, ck, cq, part, unit, tab, mask, beta, total;
    // c_ti, e_ti at row_at(N, i) + t, 0 where i is not on t's branch.  64 drafts at d = 64: only t from i's eight on, which
    // makes room for a second CTA (48 fp32 trees of up to 64 drafts 101 -> 80 us); elsewhere it would cost 2 to 9%.
    static __host__ __device__ constexpr bool packed(int N) { return D == 64 && N == 64; }
    static __host__ __device__ constexpr int row_at(int N, int i) {
        return packed(N) ? 8 * (N * (i / 8) - 4 * (i / 8) * (i / 8 - 1)) + i % 8 * (N - i / 8 * 8) - i / 8 * 8 : i * N;
    }
    static __host__ __device__ constexpr int coefs(int N) { return packed(N) ? 4 * N * (N / 8 + 1) : N * N; }
    __host__ __device__ explicit Lay(int N) {
        int at = 0;
        auto take = [&](int bytes) {
            const int was = at;
            at += (bytes + 15) / 16 * 16;
            return was;
        };
        kb = take(N * P), al = take(N * P);       // k and alpha; when the branches are walked, the products with S_0
        xk = take(N * P), xq = take(N * P);       // A k and A q: two bf16 terms or fp32; xk then holds u, xq held q
        v = take(N * P);
        ck = take(coefs(N) * 4), cq = take(coefs(N) * 4);
        part = take(6144);                // the convolution's weights, then (fp32) sums of the products' parts
        unit = take(D * D * 4 / kUnit * 8);       // addresses of S_0
        tab = take(N * 16), mask = take(N * 8), beta = take(N * 4);
        total = at;
    }
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x, y as packed bf16: the nearest ones, and those of what is left.
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = tcx::f2_to_bf2(x, y);
    const float2 h = tcx::bf2_to_f2(hi);
    lo = tcx::f2_to_bf2(x - h.x, y - h.y);
}
// W elements as they lie in memory, and in pairs.
template <int BYTES>
struct Bits {
    using type = uint4;
};
template <>
struct Bits<8> {
    using type = uint2;
};
template <class T, int W>
__device__ __forceinline__ void pairs_of(const typename Bits<W * sizeof(T)>::type &u, float2 (&x)[W / 2]) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&u);
#pragma unroll
    for (int i = 0; i < W / 2; ++i)
        x[i] = sizeof(T) == 2 ? tcx::bf2_to_f2(w[i]) : make_float2(__uint_as_float(w[2 * i % (W * sizeof(T) / 4)]), __uint_as_float(w[(2 * i + 1) % (W * sizeof(T) / 4)]));
}

// CTAs an SM: a CTA's chain of loads and steps is long, and others' work covers it.
template <int D, class T, int MT>
constexpr int kPerSm = MT == 8 ? D == 64 ? 2 : 1 : MT == 4 || (D == 128 && sizeof(T) == 4) ? 2 : 4;

// MT: tiles of 16 rows of [A k | A q], of up to 8 MT drafts.
template <int D, class T, int MT>
__global__ void __launch_bounds__(kThreads, kPerSm<D, T, MT>) verify_tree_kernel(const __grid_constant__ VerifyTreeArgs a) {
    constexpr int N = 8 * MT, P = Lay<D>::P;
    constexpr bool kMma = sizeof(T) == 2;
    extern __shared__ __align__(16) uint8_t sm[];
    const Lay<D> L(N);
    float *kb = reinterpret_cast<float *>(sm + L.kb), *al = reinterpret_cast<float *>(sm + L.al);
    float *xk = reinterpret_cast<float *>(sm + L.xk), *xq = reinterpret_cast<float *>(sm + L.xq);
    float *vb = reinterpret_cast<float *>(sm + L.v), *part = reinterpret_cast<float *>(sm + L.part);
    float *ck = reinterpret_cast<float *>(sm + L.ck), *cq = reinterpret_cast<float *>(sm + L.cq);
    const uint8_t **unit = reinterpret_cast<const uint8_t **>(sm + L.unit);
    int4 *tab = reinterpret_cast<int4 *>(sm + L.tab);
    uint64_t *mask = reinterpret_cast<uint64_t *>(sm + L.mask);
    float *beta = reinterpret_cast<float *>(sm + L.beta);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int b = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const int32_t *pages = a.state_pages + (int64_t)b * a.pool.pages_per_object;
    const Request r = request_of(a, b);
    if (r.n <= 0) {
        if (r.n < 0 && h == 0 && tid == 0) flag_status(a.status, KDA_DEV_BAD_META);
        return;
    }
    const int n = r.n;
    const int64_t row0 = (r.first * a.H + h) * D;      // the first draft's row of a token tensor
    // ---- pages; S_0 is asked into L2, its addresses are kept
    const uint64_t rec = (uint64_t)h * (uint64_t)a.pool.rec_bytes, win_off = rec + (uint64_t)D * D * 4;
    int32_t wrong = 0;
    for (int i = tid; i < a.pool.pages_per_object; i += kThreads)
        if ((uint32_t)__ldg(pages + i) >= (uint32_t)a.pool.num_pages) wrong = KDA_DEV_BAD_PAGE;
    for (int i = tid; i < D * D * 4 / kUnit; i += kThreads) {
        const uint8_t *at = obj_addr(a.pool, pages, rec + (uint64_t)i * kUnit, nullptr);
        unit[i] = at;
    }
    if (warp == 0) {   // page by page
        const uint64_t pb = (uint64_t)a.pool.page_bytes, end = rec + (uint64_t)D * D * 4;
        for (uint64_t i = rec / pb + lane; i * pb < end; i += 32) {
            const int32_t id = __ldg(pages + i);
            const uint64_t from = i * pb > rec ? i * pb : rec, to = (i + 1) * pb < end ? (i + 1) * pb : end;
            if ((uint32_t)id < (uint32_t)a.pool.num_pages) ptx::prefetch_bulk(a.pool.base + (uint64_t)id * pb + (from - i * pb), (uint32_t)(to - from));
        }
    }
    for (int i = tid; i < 3 * D; i += kThreads)   // a channel's four taps; eight channels' places in other banks for each eight
        reinterpret_cast<float4 *>(part)[i ^ (i >> 3 & 7)] = __ldg(reinterpret_cast<const float4 *>(a.conv_w) + (int64_t)h * 3 * D + i);
    for (int i = tid; i < Lay<D>::coefs(N) / 2; i += kThreads) reinterpret_cast<float4 *>(ck)[i] = make_float4(0.f, 0.f, 0.f, 0.f);   // cq too
    // ---- by the last warp: branches, by pointer doubling as in the plan, and the rows that a convolution reads: the
    // draft's own and the three before it, in bytes from the first draft's; ~w for the window's row w
    if (warp == kWarps - 1) {
        uint64_t m[2];
        int32_t p[2], q[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int i = lane + 32 * x;
            p[x] = i < n ? __ldg(a.parent + r.first + i) : -1;
            if (p[x] < -1 || (i < n && p[x] >= i)) wrong |= KDA_DEV_BAD_META, p[x] = -1;
            q[x] = p[x], m[x] = 1ull << i;
            if (i < n) beta[i] = ld_elem(static_cast<const T *>(a.beta) + (r.first + i) * a.H + h);
        }
        int32_t *up = reinterpret_cast<int32_t *>(tab);   // [N] for now
#pragma unroll
        for (int x = 0; x < 2; ++x)
            if (lane + 32 * x < N) up[lane + 32 * x] = p[x];
        __syncwarp();
        int4 rows[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            int i = lane + 32 * x < N ? lane + 32 * x : 0, back = 3;
            int32_t o[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                o[y] = i >= 0 ? i * a.H * D * (int)sizeof(T) : ~--back;
                if (i >= 0) i = up[i];
            }
            rows[x] = make_int4(o[0], o[1], o[2], o[3]);
        }
        __syncwarp();
#pragma unroll 1
        for (int k = 1; k < N; k *= 2) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (lane + 32 * x < N) mask[lane + 32 * x] = m[x], up[lane + 32 * x] = q[x];
            __syncwarp();
            if (!__any_sync(0xFFFFFFFFu, q[0] >= 0 || q[1] >= 0)) break;
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (q[x] >= 0) m[x] |= mask[q[x]], q[x] = up[q[x]];
            __syncwarp();
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
            if (lane + 32 * x < N) mask[lane + 32 * x] = m[x], tab[lane + 32 * x] = rows[x];
    }
    if (__syncthreads_or(wrong)) {
        if (wrong && h == 0) flag_status(a.status, wrong);
        return;
    }
    // ---- convolutions along the branches; alpha
    {
        // W channels a thread: few where the registers are for other CTAs (16 drafts 338 us with 8, 308 with 4), many
        // where there are many drafts (64 x 64 drafts: 550 and 688)
        constexpr int W = MT >= 4 ? 16 / (int)sizeof(T) : 4;
        using Q = typename Bits<W * sizeof(T)>::type;
        constexpr int kGroups = 3 * D / W, kAt = kThreads / kGroups;   // drafts at a time
        const int g = tid % kGroups, c = g * W % D, which = g * W / D;
        const void *tensor = which == 0 ? a.q : which == 1 ? a.k : a.v;
        const uint8_t *src = static_cast<const uint8_t *>(tensor) + (row0 + c) * (int)sizeof(T);
        float *dst = (which == 0 ? xq : which == 1 ? kb : vb) + c;
        if (tid / kGroups < kAt) {
            Q win[3];
#pragma unroll
            for (int x = 0; x < 3; ++x)
                win[x] = *reinterpret_cast<const Q *>(obj_addr(a.pool, pages, win_off + ((uint64_t)x * 3 * D + W * g) * sizeof(T), nullptr));
            float2 w[4][W / 2];
#pragma unroll
            for (int x = 0; x < W / 2; ++x) {
                const int i = W * g + 2 * x;
                const float4 y = reinterpret_cast<const float4 *>(part)[i ^ (i >> 3 & 7)];
                const float4 z = reinterpret_cast<const float4 *>(part)[(i + 1) ^ (i >> 3 & 7)];
                w[0][x] = make_float2(y.x, z.x), w[1][x] = make_float2(y.y, z.y);
                w[2][x] = make_float2(y.z, z.z), w[3][x] = make_float2(y.w, z.w);
            }
            for (int t = tid / kGroups; t < n; t += kAt) {
                const int4 rows = tab[t];
                const int32_t o[4] = {rows.w, rows.z, rows.y, rows.x};
                Q z[4];
#pragma unroll
                for (int tap = 0; tap < 4; ++tap) {
                    if (o[tap] >= 0) z[tap] = __ldg(reinterpret_cast<const Q *>(src + o[tap]));
                    else z[tap] = o[tap] == ~2 ? win[2] : o[tap] == ~1 ? win[1] : win[0];
                }
                float2 y[W / 2];
#pragma unroll
                for (int x = 0; x < W / 2; ++x) y[x] = make_float2(0.f, 0.f);
#pragma unroll
                for (int tap = 3; tap >= 0; --tap) {
                    float2 f[W / 2];
                    pairs_of<T, W>(z[tap], f);
#pragma unroll
                    for (int x = 0; x < W / 2; ++x) y[x] = tcx::ffma2(w[tap][x], f[x], y[x]);
                }
#pragma unroll
                for (int x = 0; x < W; x += 4)
                    *reinterpret_cast<float4 *>(dst + t * D + x) = make_float4(y[x / 2].x, y[x / 2].y, y[x / 2 + 1].x, y[x / 2 + 1].y);
            }
        }
        const uint8_t *alpha = static_cast<const uint8_t *>(a.alpha) + row0 * (int)sizeof(T);
        for (int i = tid; i < n * (D / W); i += kThreads) {
            const int t = i / (D / W), ch = i % (D / W) * W;
            float2 f[W / 2];
            pairs_of<T, W>(__ldg(reinterpret_cast<const Q *>(alpha + (t * a.H * D + ch) * (int)sizeof(T))), f);
#pragma unroll
            for (int x = 0; x < W; x += 4)
                *reinterpret_cast<float4 *>(al + t * D + ch + x) = make_float4(f[x / 2].x, f[x / 2].y, f[x / 2 + 1].x, f[x / 2 + 1].y);
        }
    }
    __syncthreads();
    // ---- up the branches: sixteen lanes a draft, a lane 4 or 8 channels
    {
        constexpr int C = D / 16;
        const int l16 = lane % 16;
        auto get = [&](const float *row, float2 (&x)[C / 2]) {
#pragma unroll
            for (int i = 0; i < C; i += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(row + 16 * i + 4 * l16);
                x[i / 2] = make_float2(f.x, f.y), x[i / 2 + 1] = make_float2(f.z, f.w);
            }
        };
#pragma unroll 1
        for (int t0 = 2 * warp; t0 < n; t0 += 2 * kWarps) {
            const bool mine = t0 + lane / 16 < n;               // (where they are odd the last one goes along twice)
            const int t = mine ? t0 + lane / 16 : n - 1;
            float2 kr[C / 2], qr[C / 2];
            get(kb + t * D, kr);
            get(xq + t * D, qr);
            __syncwarp();
            uint64_t m = mask[t];
            int i = t;
            while (__any_sync(0xFFFFFFFFu, m != 0)) {
                float2 ki[C / 2], f[C / 2], dk = make_float2(0.f, 0.f), dq = dk;
                get(kb + i * D, ki);
                get(al + i * D, f);
#pragma unroll
                for (int x = 0; x < C / 2; ++x) dk = tcx::ffma2(kr[x], ki[x], dk), dq = tcx::ffma2(qr[x], ki[x], dq);
                // even lanes sum for k, odd ones for q
                const float sk = dk.x + dk.y, sq = dq.x + dq.y;
                float sum = (lane & 1 ? sq : sk) + __shfl_xor_sync(0xFFFFFFFFu, lane & 1 ? sk : sq, 1);
#pragma unroll
                for (int y = 2; y < 16; y <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, y);
                if (m) {
                    if (l16 < 2) (l16 ? cq : ck)[Lay<D>::row_at(N, i) + t] = sum;
#pragma unroll
                    for (int x = 0; x < C / 2; ++x) kr[x] = tcx::fmul2(kr[x], f[x]), qr[x] = tcx::fmul2(qr[x], f[x]);
                    m &= ~(1ull << i);
                    if (m) i = 63 - __clzll((long long)m);
                }
            }
            // A k, and A q in q's place (nobody else reads it).  Two bf16 terms: a row's 16-byte units are exchanged
            // by the row's number, so that eight rows' units of one column lie in different banks.
            if (mine)
#pragma unroll
                for (int row = 0; row < 2; ++row) {
                    uint8_t *at = reinterpret_cast<uint8_t *>(row ? xq : xk) + t * P;
#pragma unroll
                    for (int x = 0; x < C; x += 4) {
                        const float2 y = row ? qr[x / 2] : kr[x / 2], z = row ? qr[x / 2 + 1] : kr[x / 2 + 1];
                        if constexpr (kMma) {
                            uint2 hi, lo;
                            split2(y.x, y.y, hi.x, lo.x), split2(z.x, z.y, hi.y, lo.y);
                            const int to = (((2 * x + l16 / 2) ^ (t & 7)) << 4) + l16 % 2 * 8;   // channels 16 x + 4 l16 and up
                            *reinterpret_cast<uint2 *>(at + to) = hi;
                            *reinterpret_cast<uint2 *>(at + P / 2 + to) = lo;
                        } else {
                            *reinterpret_cast<float4 *>(at + (16 * x + 4 * l16) * 4) = make_float4(y.x, y.y, z.x, z.y);
                        }
                    }
                }
        }
    }
    // ---- their products with S_0: of A k over k, of A q over alpha
    if constexpr (kMma) {
        // A warp takes 16 columns (two tiles of 8, their columns in turn).  Both operands in two bf16 terms, three of
        // the four products: off by 3 x 2^-16 of the terms' absolute sum, below an output's own rounding of 2^-8 unless
        // the sum cancels to some hundredth of its terms (64 keys in the state, q at right angles to all: outputs 2.2e-3
        // off, 1.6e-3 by decode steps).  Three terms would be six products.
        constexpr int kCols = D / 16, kSplit = kWarps / kCols;    // d = 64: two warps a 16 columns, each half of the rows
        constexpr int kMine = MT >= kSplit ? MT / kSplit : 1;     // tiles of rows
        const int w = warp % kCols, g = lane / 4, t4 = lane % 4;
        const int mt0 = MT >= kSplit ? warp / kCols * kMine : 0;
        const bool works = MT >= kSplit || warp < kCols;
        // rows 16 s + 2 t4, + 1, + 8, + 9 of S_0, columns 16 w + 2 g and the next; two steps s are under way, the first
        // ones while the other warps still walk
        float2 f[2][4];
        auto fetch = [&](int s, float2 (&y)[4]) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int byte = (16 * s + 2 * t4 + (x & 1) + 8 * (x >> 1)) * D * 4 + (16 * w + 2 * g) * 4;
                y[x] = __ldcs(reinterpret_cast<const float2 *>(unit[byte / kUnit] + byte % kUnit));
            }
        };
        if (works) fetch(0, f[0]), fetch(1, f[1]);
        __syncthreads();
        if (works) {
            float acc[kMine][2][4] = {};
            const uint32_t at = ptx::smem_u32(sm + L.xk) + (mt0 * 16 + lane % 16) * P;   // (xq follows xk)
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                uint32_t hi[2][2], lo[2][2];                      // [tile][register]
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    split2(f[s & 1][2 * x].x, f[s & 1][2 * x + 1].x, hi[0][x], lo[0][x]);
                    split2(f[s & 1][2 * x].y, f[s & 1][2 * x + 1].y, hi[1][x], lo[1][x]);
                }
                if (s + 2 < D / 16) fetch(s + 2, f[s & 1]);
                const uint32_t to = at + (((2 * s + lane / 16) ^ (lane & 7)) << 4);
#pragma unroll
                for (int mt = 0; mt < kMine; ++mt) {
                    uint32_t ah[4], as[4];
                    ldsm4(ah, to + mt * 16 * P);
                    ldsm4(as, to + mt * 16 * P + P / 2);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        mma(acc[mt][y], as, hi[y][0], hi[y][1]);
                        mma(acc[mt][y], ah, lo[y][0], lo[y][1]);
                        mma(acc[mt][y], ah, hi[y][0], hi[y][1]);
                    }
                }
            }
#pragma unroll
            for (int mt = 0; mt < kMine; ++mt)
#pragma unroll
                for (int x = 0; x < 2; ++x)   // columns 16 w + 4 t4 and up: tiles 0, 1, 0, 1 (al follows kb)
                    *reinterpret_cast<float4 *>(kb + ((mt0 + mt) * 16 + g + 8 * x) * D + 16 * w + 4 * t4) =
                        make_float4(acc[mt][0][2 * x], acc[mt][1][2 * x], acc[mt][0][2 * x + 1], acc[mt][1][2 * x + 1]);
        }
        __syncthreads();
    } else {
        // a thread takes a column of S_0 and a part of its rows; eight rows of the products at a time
        constexpr int G = kThreads / D, R = D / G;
        const int j = tid % D, grp = tid / D;
        float s[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int byte = ((grp * R + i) * D + j) * 4;
            s[i] = __ldcs(reinterpret_cast<const float *>(unit[byte / kUnit] + byte % kUnit));
        }
        __syncthreads();
#pragma unroll 1
        for (int r0 = 0; r0 < 2 * N; r0 += 8) {
            if (r0 % N >= n) continue;                       // rows of no draft
            float y[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                y[x] = 0.f;
                const float4 *v = reinterpret_cast<const float4 *>(xk + (r0 + x) * D + grp * R);
#pragma unroll
                for (int i = 0; i < R / 4; ++i) {
                    const float4 f = v[i];
                    y[x] = fmaf(f.x, s[4 * i], y[x]), y[x] = fmaf(f.y, s[4 * i + 1], y[x]);
                    y[x] = fmaf(f.z, s[4 * i + 2], y[x]), y[x] = fmaf(f.w, s[4 * i + 3], y[x]);
                }
                if (grp) part[((grp - 1) * 8 + x) * D + j] = y[x];
            }
            __syncthreads();
            if (grp == 0)
#pragma unroll
                for (int x = 0; x < 8; ++x) {
#pragma unroll
                    for (int i = 0; i < G - 1; ++i) y[x] += part[(i * 8 + x) * D + j];
                    kb[(r0 + x) * D + j] = y[x];
                }
            __syncthreads();
        }
    }
    // ---- u, column by column, eight drafts at a time; every draft before counts, with 0 where it is not on the branch.
    // 0 times what is no number is none: a column with such a u is taken again, along the branches alone.
    float *u = xk;
    const int j = tid % D, grp = tid / D;
    auto add8 = [&](float2 (&acc)[4], const float *c, float x) {
        const float4 c0 = *reinterpret_cast<const float4 *>(c), c1 = *reinterpret_cast<const float4 *>(c + 4);
        const float2 xx = make_float2(x, x);
        acc[0] = tcx::ffma2(make_float2(c0.x, c0.y), xx, acc[0]), acc[1] = tcx::ffma2(make_float2(c0.z, c0.w), xx, acc[1]);
        acc[2] = tcx::ffma2(make_float2(c1.x, c1.y), xx, acc[2]), acc[3] = tcx::ffma2(make_float2(c1.z, c1.w), xx, acc[3]);
    };
    if (grp == 0) {
        bool strange = false;
#pragma unroll 1
        for (int t0 = 0; t0 < n; t0 += 8) {
            float2 acc[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[x] = make_float2(kb[(t0 + 2 * x) * D + j], kb[(t0 + 2 * x + 1) * D + j]);
#pragma unroll 4
            for (int i = 0; i < t0; ++i) add8(acc, ck + Lay<D>::row_at(N, i) + t0, u[i * D + j]);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                if (t0 + x >= n) break;
                const float y = beta[t0 + x] * (vb[(t0 + x) * D + j] - (x & 1 ? acc[x / 2].y : acc[x / 2].x));
                u[(t0 + x) * D + j] = y;
                strange |= !(fabsf(y) < INFINITY);
                if (x < 7) add8(acc, ck + Lay<D>::row_at(N, t0 + x) + t0, y);
            }
        }
        if (strange)
#pragma unroll 1
            for (int t = 0; t < n; ++t) {
                float acc = kb[t * D + j];
                for (uint64_t m = mask[t] & ~(1ull << t); m; m &= m - 1) {
                    const int i = __ffsll((long long)m) - 1;
                    acc = fmaf(ck[Lay<D>::row_at(N, i) + t], u[i * D + j], acc);
                }
                u[t * D + j] = beta[t] * (vb[t * D + j] - acc);
            }
    }
    __syncthreads();
    // ---- and o
    T *o = static_cast<T *>(a.o) + row0 + j;
    bool strange = false;
#pragma unroll 1
    for (int t0 = 8 * grp; t0 < n; t0 += 8 * (kThreads / D)) {
        float2 acc[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[x] = make_float2(al[(t0 + 2 * x) * D + j], al[(t0 + 2 * x + 1) * D + j]);
        const int end = min(t0 + 8, n);
#pragma unroll 4
        for (int i = 0; i < end; ++i) {
            const float y = u[i * D + j];
            strange |= !(fabsf(y) < INFINITY);
            add8(acc, cq + Lay<D>::row_at(N, i) + t0, y);
        }
#pragma unroll
        for (int x = 0; x < 8; ++x)
            if (t0 + x < n) st_elem(o + (t0 + x) * a.H * D, x & 1 ? acc[x / 2].y : acc[x / 2].x);
    }
    if (strange)
#pragma unroll 1
        for (int t = 0; t < n; ++t) {
            if (t / 8 % (kThreads / D) != grp) continue;
            float acc = al[t * D + j];
            for (uint64_t m = mask[t]; m; m &= m - 1) {
                const int i = __ffsll((long long)m) - 1;
                acc = fmaf(cq[Lay<D>::row_at(N, i) + t], u[i * D + j], acc);
            }
            st_elem(o + t * a.H * D, acc);
        }
}

// The state after the accepted branch: decode steps of its drafts one after another with the state in registers,
// read and written once.  Warp w of 16 has D / 16 rows of S, a lane D / 32 columns.  (The form for fp32, d = 64 and
// pages below 64 KiB: 256 x 32 heads of 128, 2.5 tokens a branch, fp32: 269 us.)
constexpr int kAccThreads = 512, kAccWarps = 16;

template <int D, class T>
__global__ void __launch_bounds__(kAccThreads, 2) verify_tree_accept_kernel(const __grid_constant__ VerifyTreeArgs a, int N) {
    constexpr int V = kVec<T>, C3 = 3 * D, R = D / kAccWarps, C = D / 32;
    extern __shared__ __align__(16) uint8_t sm[];
    float *kb = reinterpret_cast<float *>(sm), *vb = kb + N * D, *al = vb + N * D, *red = al + N * D, *w = red + kAccWarps * D;
    float *beta = w + D;
    int32_t *path = reinterpret_cast<int32_t *>(beta + kMost);
    T *win = reinterpret_cast<T *>(path + kMost);   // the window before, [3][3D]
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int b = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const Request r = request_of(a, b);
    const int m = r.n < 0 ? 0 : __ldg(a.accepted + b);
    if (r.n < 0 || m < 0 || m > r.n) {
        if (h == 0 && tid == 0) flag_status(a.status, KDA_DEV_BAD_META);
        return;
    }
    if (m == 0) return;
    int32_t at = -1;
    if (tid < m) path[tid] = at = __ldg(a.path + r.first + tid);
    const int32_t *pages = a.state_pages + (int64_t)b * a.pool.pages_per_object;
    if (pages_lost(a.pool, pages)) {
        if (h == 0 && tid == 0) flag_status(a.status, KDA_DEV_BAD_PAGE);
        return;
    }
    if (__syncthreads_or(tid < m && (at < (tid ? path[tid - 1] + 1 : 0) || at >= r.n))) {
        if (h == 0 && tid == 0) flag_status(a.status, KDA_DEV_BAD_META);
        return;
    }
    const uint64_t rec = (uint64_t)h * (uint64_t)a.pool.rec_bytes, win_off = rec + (uint64_t)D * D * 4;
    float s[R][C];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const uint8_t *p = obj_addr(a.pool, pages, rec + ((uint64_t)(warp * R + i) * D + lane * C) * 4, a.status);
#pragma unroll
        for (int x = 0; x < C; x += 2) {
            const float2 f = __ldcs(reinterpret_cast<const float2 *>(p) + x / 2);
            s[i][x] = f.x, s[i][x + 1] = f.y;
        }
    }
    for (int i = tid; i < 3 * C3 / V; i += kAccThreads)
        *reinterpret_cast<uint4 *>(win + i * V) =
            *reinterpret_cast<const uint4 *>(obj_addr(a.pool, pages, win_off + (uint64_t)i * V * sizeof(T), a.status));
    if (tid < m) beta[tid] = ld_elem(static_cast<const T *>(a.beta) + (r.first + at) * a.H + h);
    __syncthreads();
    // raw token x of the branch (x < 0: of the window, -1 the newest), channel c of q | k | v
    auto raw = [&](int x, int c) {
        if (x < 0) return static_cast<const T *>(win + (3 + x) * C3 + c);
        const void *src = c < D ? a.q : c < 2 * D ? a.k : a.v;
        return reinterpret_cast<const T *>(raw_at(a, src, r.first + path[x], h, D, c % D, sizeof(T)));
    };
    constexpr int kGroups = 2 * D / V;   // k and v alone: no answers here
    for (int i = tid; i < m * kGroups; i += kAccThreads) {
        const int t = i / kGroups, c = D + i % kGroups * V;
        float y[V];
#pragma unroll
        for (int x = 0; x < V; ++x) y[x] = 0.f;
#pragma unroll
        for (int tap = 0; tap < 4; ++tap) {
            float z[V];
            load_vec(raw(t - 3 + tap, c), z);
#pragma unroll
            for (int x = 0; x < V; ++x) y[x] = fmaf(__ldg(a.conv_w + ((int64_t)h * C3 + c + x) * 4 + tap), z[x], y[x]);
        }
        float *dst = c < 2 * D ? kb + t * D + c - D : vb + t * D + c - 2 * D;
#pragma unroll
        for (int x = 0; x < V; ++x) dst[x] = y[x];
    }
    for (int i = tid; i < m * (D / V); i += kAccThreads) {
        const int t = i / (D / V), c = i % (D / V) * V;
        float x[V];
        load_vec(reinterpret_cast<const T *>(raw_at(a, a.alpha, r.first + path[t], h, D, c, sizeof(T))), x);
#pragma unroll
        for (int y = 0; y < V; ++y) al[t * D + c + y] = x[y];
    }
    __syncthreads();
#pragma unroll 1
    for (int t = 0; t < m; ++t) {
        float y[C];
#pragma unroll
        for (int x = 0; x < C; ++x) y[x] = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float f = al[t * D + warp * R + i], k = kb[t * D + warp * R + i];
#pragma unroll
            for (int x = 0; x < C; ++x) s[i][x] *= f, y[x] = fmaf(k, s[i][x], y[x]);
        }
#pragma unroll
        for (int x = 0; x < C; ++x) red[warp * D + lane * C + x] = y[x];
        __syncthreads();
        if (tid < D) {
            float acc = 0.f;
#pragma unroll
            for (int i = 0; i < kAccWarps; ++i) acc += red[i * D + tid];
            w[tid] = beta[t] * (vb[t * D + tid] - acc);
        }
        __syncthreads();
        float z[C];
#pragma unroll
        for (int x = 0; x < C; ++x) z[x] = w[lane * C + x];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float k = kb[t * D + warp * R + i];
#pragma unroll
            for (int x = 0; x < C; ++x) s[i][x] = fmaf(k, z[x], s[i][x]);
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        uint8_t *p = obj_addr(a.pool, pages, rec + ((uint64_t)(warp * R + i) * D + lane * C) * 4, a.status);
#pragma unroll
        for (int x = 0; x < C; x += 2) __stcs(reinterpret_cast<float2 *>(p) + x / 2, make_float2(s[i][x], s[i][x + 1]));
    }
    // the window: the branch's last three raw tokens
    for (int i = tid; i < 3 * C3 / V; i += kAccThreads) {
        const int row = i / (C3 / V), c = i % (C3 / V) * V;
        *reinterpret_cast<uint4 *>(obj_addr(a.pool, pages, win_off + (uint64_t)i * V * sizeof(T), a.status)) =
            *reinterpret_cast<const uint4 *>(raw(m - 3 + row, c));
    }
}

// The same for bf16 records of d = 128 in pages of at least 64 KiB, as a pipeline of bulk copies: one CTA an SM, three
// slots of a record and its tokens; a warp looks branches up and copies records in and out, sixteen warps advance the
// state of the one between, a thread 32 rows of a column in registers over the whole branch.  Measured: 256 requests x 32
// heads, branches of 2.5 tokens (214 requests accept some): 211 us, 0.95 GB moved, 66% of the copy rate (339 us by the
// kernel above); a job's meetings of sixteen warps, two a token, bound it.  8192 branches of 1, 4, 8, 16 and 64 tokens each:
// 229, 270, 428, 860 and 3504 us (kernel above: 300, 461, 655, 1038 and 3619).
// Taken for any number of (request, head) pairs up to kPipeMost.  With few pairs it is the faster one too, a token's step
// being shorter (16 pairs with 1, 4, 16, 64 tokens: 7.2, 9.6, 19.3, 57.1 us, and 9.5, 12.9, 25.0, 76.7 by the kernel above;
// 256 pairs: 9.8, 13.7, 33.1, 109 and 11.9, 17.7, 40.8, 136).  But a CTA goes over its requests one by one, and the warps
// that wait for one that accepts something give up after some seconds; near 2^31 the count itself would wrap.  More records
// than 2^24 no memory holds.
constexpr int kPipeMost = 1 << 24;
constexpr int kPipe = 512, kPipeThreads = kPipe + 32, kSlots = 3;
constexpr int kSlotTokens = 4;                        // a branch's tokens that come with the record; others are fetched
constexpr uint32_t kRecBytes = 67840, kSlotBytes = kRecBytes + kSlotTokens * 1024;
struct PipeJob {
    int32_t item, m;                                  // m < 0: the end
    int64_t first;
    int32_t path[kMost];
    float beta[kMost];
};
constexpr uint32_t kPipeRed = kSlots * kSlotBytes, kPipeX = kPipeRed + 2 * 4 * 128 * 4, kPipeA = kPipeX + 2 * 256 * 4,
                   kPipeJobs = kPipeA + 2 * 128 * 4, kPipeMisc = kPipeJobs + kSlots * sizeof(PipeJob), kPipeSmem = kPipeMisc + 128;
static_assert(kSlotBytes % 128 == 0 && kPipeSmem <= 227 * 1024, "shared memory");

__global__ void __launch_bounds__(kPipeThreads, 1) verify_tree_accept_pipe_kernel(const __grid_constant__ VerifyTreeArgs a) {
    using bf16 = __nv_bfloat16;
    constexpr int D = 128, C3 = 3 * D;
    extern __shared__ __align__(128) uint8_t sm[];
    float *red = reinterpret_cast<float *>(sm + kPipeRed), *xb = reinterpret_cast<float *>(sm + kPipeX);
    float *al = reinterpret_cast<float *>(sm + kPipeA);
    PipeJob *jobs = reinterpret_cast<PipeJob *>(sm + kPipeJobs);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + kPipeMisc), *done = full + kSlots;
    volatile int *err = reinterpret_cast<volatile int *>(sm + kPipeMisc + 64), *go = err + 1;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, total = a.B * a.H;
    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            ptx::mbar_init(&full[i], 1);
            ptx::mbar_init(&done[i], 1);
        }
        *err = 0;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    if (warp == kPipe / 32) {
        // ------------------------------------------------------------------ branches and copies
        auto pieces = [&](int item, auto &&fn) {      // of an item's record, at most one a page
            const int32_t *pages = a.state_pages + (int64_t)(item / a.H) * a.pool.pages_per_object;
            int64_t off = (int64_t)(item % a.H) * a.pool.rec_bytes;
            for (uint32_t at = 0; at < kRecBytes;) {
                const int64_t pi = off / a.pool.page_bytes, in = off - pi * a.pool.page_bytes;
                const uint32_t len = (uint32_t)min((int64_t)(kRecBytes - at), a.pool.page_bytes - in);
                fn(a.pool.base + (int64_t)__ldg(pages + pi) * a.pool.page_bytes + in, at, len);
                off += len, at += len;
            }
        };
        auto store = [&](int n) {                     // job n's record back to its pages, by lane 0
            const int s = n % kSlots;
            pieces(jobs[s].item, [&](uint8_t *p, uint32_t at, uint32_t len) { ptx::bulk_store(p, sm + s * kSlotBytes + at, len); });
            ptx::bulk_commit();
        };
        int n = 0;                                    // jobs
        bool ok = true;
        // a slot for job n: the record that used it goes back first
        auto slot = [&]() {
            int stop = 0;
            if (lane == 0 && n >= kSlots) {
                if (!ptx::mbar_wait(&done[n % kSlots], (uint32_t)((n / kSlots - 1) & 1), err)) stop = 1;
                else {
                    store(n - kSlots);
                    ptx::bulk_wait_read0();
                }
            }
            return __shfl_sync(0xFFFFFFFFu, stop, 0) == 0;
        };
        for (int item = blockIdx.x; item < total; item += gridDim.x) {
            const int b = item / a.H, h = item % a.H;
            const Request r = request_of(a, b);
            const int32_t m = __ldg(a.accepted + b);
            bool lost = false;
            for (int i = lane; i < a.pool.pages_per_object; i += 32)
                lost |= (uint32_t)__ldg(a.state_pages + (int64_t)b * a.pool.pages_per_object + i) >= (uint32_t)a.pool.num_pages;
            lost = __any_sync(0xFFFFFFFFu, lost);
            int32_t p[2] = {-1, -1};
            bool wrong = r.n < 0 || m < 0 || m > r.n;
            if (!wrong) {
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (lane + 32 * x < m) p[x] = __ldg(a.path + r.first + lane + 32 * x);
                const int32_t before = __shfl_up_sync(0xFFFFFFFFu, p[0], 1), half = __shfl_sync(0xFFFFFFFFu, p[0], 31);
                const int32_t behind = __shfl_up_sync(0xFFFFFFFFu, p[1], 1);
                bool off = lane < m && (p[0] < 0 || p[0] >= r.n || (lane && p[0] <= before));
                off |= lane + 32 < m && (p[1] < 0 || p[1] >= r.n || p[1] <= (lane ? behind : half));
                wrong = __any_sync(0xFFFFFFFFu, off);
            }
            if (wrong || (lost && m)) {
                if (lane == 0 && h == 0) flag_status(a.status, wrong ? KDA_DEV_BAD_META : KDA_DEV_BAD_PAGE);
                continue;
            }
            if (m == 0) continue;
            float be[2];
#pragma unroll
            for (int x = 0; x < 2; ++x)
                be[x] = lane + 32 * x < m ? ld_elem(static_cast<const bf16 *>(a.beta) + (r.first + p[x]) * a.H + h) : 0.f;
            ok = slot();
            if (!ok) break;
            PipeJob &jb = jobs[n % kSlots];
#pragma unroll
            for (int x = 0; x < 2; ++x) jb.path[lane + 32 * x] = p[x], jb.beta[lane + 32 * x] = be[x];
            if (lane == 0) jb.item = item, jb.m = m, jb.first = r.first;
            __syncwarp();
            if (lane == 0) {
                uint64_t *bar = &full[n % kSlots];
                uint8_t *dst = sm + n % kSlots * kSlotBytes;
                const int toks = min(m, kSlotTokens);
                ptx::mbar_arrive_expect_tx(bar, kRecBytes + toks * 1024);
                pieces(item, [&](uint8_t *q, uint32_t at, uint32_t len) { ptx::bulk_load(dst + at, q, len, bar); });
                for (int t = 0; t < toks; ++t) {
                    const int64_t row = ((r.first + jb.path[t]) * a.H + h) * D;
                    const void *src[4] = {a.q, a.k, a.v, a.alpha};
                    for (int x = 0; x < 4; ++x)
                        ptx::bulk_load(dst + kRecBytes + t * 1024 + x * 256, static_cast<const bf16 *>(src[x]) + row, 256, bar);
                }
            }
            for (int i = 4 * kSlotTokens + lane; i < 4 * m; i += 32) {   // the other tokens are asked into L2
                const void *src = i % 4 == 0 ? a.q : i % 4 == 1 ? a.k : i % 4 == 2 ? a.v : a.alpha;
                ptx::prefetch_bulk(static_cast<const bf16 *>(src) + ((r.first + jb.path[i / 4]) * a.H + h) * D, 256);
            }
            __syncwarp();
            ++n;
        }
        if (ok && slot()) {                           // the end, and the last records back
            if (lane == 0) {
                jobs[n % kSlots].m = -1;
                ptx::mbar_arrive(&full[n % kSlots]);
                for (int i = max(0, n + 1 - kSlots); i < n; ++i) {
                    if (!ptx::mbar_wait(&done[i % kSlots], (uint32_t)(i / kSlots & 1), err)) break;
                    store(i);
                }
            }
        }
        if (lane == 0) {
            ptx::bulk_wait0();
            if (*err)                                 // leave no copy in flight
                for (int i = max(0, n - kSlots); i < n; ++i)
                    for (uint32_t k = 0; k < ptx::kSpinLimit && !ptx::mbar_try_wait(&full[i % kSlots], (uint32_t)(i / kSlots & 1)); ++k) {
                    }
        }
    } else {
        // ------------------------------------------------------------------ the states
        const int j = tid % D, rq = tid / D;
        auto meet = [&]() { tcx::named_bar(1, kPipe); };
        for (int n = 0;; ++n) {
            const int s = n % kSlots;
            if (tid == 0) *go = ptx::mbar_wait(&full[s], (uint32_t)(n / kSlots & 1), err) && !*err;
            meet();
            if (!*go) break;
            const PipeJob &jb = jobs[s];
            const int m = jb.m;
            if (m < 0) break;
            uint8_t *slot = sm + s * kSlotBytes;
            float *S = reinterpret_cast<float *>(slot);
            bf16 *win = reinterpret_cast<bf16 *>(slot + D * D * 4);
            const bf16 *tok = reinterpret_cast<const bf16 *>(slot + kRecBytes);
            const int h = jb.item % a.H;
            float sv[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) sv[i] = S[(rq * 32 + i) * D + j];
            // a thread a channel of q | k | v: the last three raw values; the others have alpha
            const int c = tid;
            bf16 p0{}, p1{}, p2{};
            float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < C3) {
                p0 = win[c], p1 = win[C3 + c], p2 = win[2 * C3 + c];
                if (c >= D) w = __ldg(reinterpret_cast<const float4 *>(a.conv_w) + (int64_t)h * C3 + c);
            }
            const bf16 *mine = static_cast<const bf16 *>(rq == 0 ? a.q : rq == 1 ? a.k : rq == 2 ? a.v : a.alpha);
            // tokens two steps ahead: those that did not come with the record come from L2, which takes longer than a step
            // (read where they are used, 8192 branches of 16 and 64 tokens take 995 and 3964 us, not 860 and 3504)
            auto token = [&](int t) { return t < kSlotTokens ? tok[t * 512 + c] : __ldg(mine + ((jb.first + jb.path[t]) * a.H + h) * D + j); };
            bf16 x1 = token(0), x2 = m > 1 ? token(1) : x1;
#pragma unroll 1
            for (int t = 0; t < m; ++t) {
                const int par = t & 1;
                const bf16 x = x1;
                x1 = x2;
                if (t + 2 < m) x2 = token(t + 2);
                if (c >= C3) {
                    al[par * D + j] = __bfloat162float(x);
                } else {
                    if (c >= D)
                        xb[par * 256 + c - D] = w.x * __bfloat162float(p0) + w.y * __bfloat162float(p1) + w.z * __bfloat162float(p2) +
                                                w.w * __bfloat162float(x);
                    p0 = p1, p1 = p2, p2 = x;
                }
                meet();
                const float4 *k4 = reinterpret_cast<const float4 *>(xb + par * 256 + rq * 32), *a4 = reinterpret_cast<const float4 *>(al + par * D + rq * 32);
                float acc = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 k = k4[i], f = a4[i];
                    sv[4 * i] *= f.x, sv[4 * i + 1] *= f.y, sv[4 * i + 2] *= f.z, sv[4 * i + 3] *= f.w;
                    acc = fmaf(k.x, sv[4 * i], acc), acc = fmaf(k.y, sv[4 * i + 1], acc);
                    acc = fmaf(k.z, sv[4 * i + 2], acc), acc = fmaf(k.w, sv[4 * i + 3], acc);
                }
                float *sum = red + par * 4 * D;
                sum[rq * D + j] = acc;
                meet();
                const float u = (sum[j] + sum[D + j]) + (sum[2 * D + j] + sum[3 * D + j]);
                const float wj = jb.beta[t] * (xb[par * 256 + D + j] - u);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 k = k4[i];
                    sv[4 * i] = fmaf(k.x, wj, sv[4 * i]), sv[4 * i + 1] = fmaf(k.y, wj, sv[4 * i + 1]);
                    sv[4 * i + 2] = fmaf(k.z, wj, sv[4 * i + 2]), sv[4 * i + 3] = fmaf(k.w, wj, sv[4 * i + 3]);
                }
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) S[(rq * 32 + i) * D + j] = sv[i];
            if (c < C3) win[c] = p0, win[C3 + c] = p1, win[2 * C3 + c] = p2;
            ptx::fence_proxy_async_smem();
            meet();
            if (tid == 0) ptx::mbar_arrive(&done[s]);
        }
    }
    __syncthreads();
    if (*err && tid == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
}

template <int D, class T, int MT>
cudaError_t verify_of(const VerifyTreeArgs &a, cudaStream_t st) {
    auto kern = verify_tree_kernel<D, T, MT>;
    const int smem = Lay<D>(8 * MT).total;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)(a.B * a.H), kThreads, smem, st>>>(a);
    return cudaGetLastError();
}
template <int D, class T>
cudaError_t verify(const VerifyTreeArgs &a, cudaStream_t st) {
    if (a.max_q <= 8) return verify_of<D, T, 1>(a, st);
    if (a.max_q <= 16) return verify_of<D, T, 2>(a, st);
    if (a.max_q <= 32) return verify_of<D, T, 4>(a, st);
    return verify_of<D, T, 8>(a, st);
}

template <int D, class T>
cudaError_t accept(const VerifyTreeArgs &a, cudaStream_t st) {
    if constexpr (D == 128 && sizeof(T) == 2)
        if (a.pool.page_bytes >= 65536 && a.B * a.H <= kPipeMost) {
            const cudaError_t e = cudaFuncSetAttribute(verify_tree_accept_pipe_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPipeSmem);
            if (e != cudaSuccess) return e;
            verify_tree_accept_pipe_kernel<<<(unsigned)min(a.B * a.H, kAttnSms), kPipeThreads, kPipeSmem, st>>>(a);
            return cudaGetLastError();
        }
    const int N = (a.max_q + 7) / 8 * 8;
    const int64_t smem = ((int64_t)3 * N * D + kAccWarps * D + D + 2 * kMost) * 4 + 9 * D * (int64_t)sizeof(T);
    auto kern = verify_tree_accept_kernel<D, T>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)(a.B * a.H), kAccThreads, (size_t)smem, st>>>(a, N);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_verify_tree(const VerifyTreeArgs &a, cudaStream_t s) {
    if (a.d == 128) return a.dtype == KDA_F32 ? verify<128, float>(a, s) : verify<128, __nv_bfloat16>(a, s);
    return a.dtype == KDA_F32 ? verify<64, float>(a, s) : verify<64, __nv_bfloat16>(a, s);
}

cudaError_t launch_verify_tree_accept(const VerifyTreeArgs &a, cudaStream_t s) {
    if (a.d == 128) return a.dtype == KDA_F32 ? accept<128, float>(a, s) : accept<128, __nv_bfloat16>(a, s);
    return a.dtype == KDA_F32 ? accept<64, float>(a, s) : accept<64, __nv_bfloat16>(a, s);
}

}  // namespace kda
