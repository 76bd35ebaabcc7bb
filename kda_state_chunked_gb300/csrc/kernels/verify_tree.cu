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
//   loads of S_0 are started;  masks of the branches, convolutions along them;
//   a warp a draft walks its branch towards the root: c_ti, e_ti, A_t k_t, A_t q_t;
//   the products with S_0;  then a thread a column solves for u, and all add up o.
#include "common.cuh"

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

// The convolution's inputs for one draft: packed rows of the three drafts before it on its branch, nearest first, or
// (negative) window rows: -1 the newest.
__device__ __forceinline__ const uint8_t *raw_at(const VerifyTreeArgs &a, const void *x, int64_t row, int h, int d, int c, int es) {
    return static_cast<const uint8_t *>(x) + ((row * a.H + h) * d + c) * es;
}

template <int D>
struct Lay {
    // floats, n: drafts rounded up to a multiple of 8
    static __host__ __device__ int64_t bytes(int n) {
        return ((int64_t)5 * n * D + 2 * (int64_t)n * n + 8 * D) * 4 + kMost * (8 + 4 + 4);
    }
};

// Threads: two groups of D.
template <int D, class T>
__global__ void __launch_bounds__(2 * D) verify_tree_kernel(const __grid_constant__ VerifyTreeArgs a, int N) {
    constexpr int NT = 2 * D, kWarps = NT / 32, V = kVec<T>;
    extern __shared__ __align__(16) float sm[];
    float *kb = sm, *xk = kb + N * D, *xq = xk + N * D, *al = xq + N * D, *u = al + N * D;   // u: v until solved
    float *ck = u + N * D, *cq = ck + N * N, *part = cq + N * N;                            // part: [8][D]
    uint64_t *mask = reinterpret_cast<uint64_t *>(part + 8 * D);
    float *beta = reinterpret_cast<float *>(mask + kMost);
    int32_t *up = reinterpret_cast<int32_t *>(beta + kMost);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int b = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const Request r = request_of(a, b);
    if (r.n <= 0) {
        if (r.n < 0 && h == 0 && tid == 0) flag_status(a.status, KDA_DEV_BAD_META);
        return;
    }
    const int n = r.n;
    const int32_t *pages = a.state_pages + (int64_t)b * a.pool.pages_per_object;
    if (pages_lost(a.pool, pages)) {
        if (h == 0 && tid == 0) flag_status(a.status, KDA_DEV_BAD_PAGE);
        return;
    }
    // ---- S_0: a thread takes a column and D / 2 rows
    const uint64_t rec = (uint64_t)h * (uint64_t)a.pool.rec_bytes, win_off = rec + (uint64_t)D * D * 4;
    const int j = tid % D, half = tid / D;
    float s[D / 2];
    {
        const uint64_t off = rec + ((uint64_t)(half * (D / 2)) * D + j) * 4, span = (uint64_t)(D / 2 - 1) * D * 4;
        const uint8_t *run = run_addr(a.pool, pages, off, span, a.status);
#pragma unroll
        for (int i = 0; i < D / 2; ++i)
            s[i] = __ldcs(reinterpret_cast<const float *>(run ? run + i * D * 4 : obj_addr(a.pool, pages, off + (uint64_t)i * D * 4, a.status)));
    }
    // ---- parents, branches
    int32_t p = -1;
    if (tid < n) p = __ldg(a.parent + r.first + tid);
    if (__syncthreads_or(p < -1 || (tid < n && p >= tid))) {
        if (h == 0 && tid == 0) flag_status(a.status, KDA_DEV_BAD_META);
        return;
    }
    {
        uint64_t m = tid < kMost ? 1ull << tid : 0;
        int32_t q = p;
#pragma unroll 1
        for (int k = 1; k < kMost; k *= 2) {
            if (tid < kMost) mask[tid] = m, up[tid] = q;
            if (!__syncthreads_or(q >= 0)) break;
            if (q >= 0) m |= mask[q], q = up[q];
            __syncthreads();
        }
        __syncthreads();
        if (tid < kMost) mask[tid] = m, up[tid] = p;
        if (tid < n) beta[tid] = ld_elem(static_cast<const T *>(a.beta) + (r.first + tid) * a.H + h);
    }
    __syncthreads();
    // ---- convolutions along the branches; alpha
    {
        constexpr int kGroups = 3 * D / V, kAt = NT / kGroups;   // drafts at a time
        const int g = tid % kGroups, c = g * V % D, part3 = g * V / D;
        const void *src = part3 == 0 ? a.q : part3 == 1 ? a.k : a.v;
        float *dst = part3 == 0 ? xq : part3 == 1 ? kb : u;
        if (tid / kGroups < kAt) {
            float w[V][4];
#pragma unroll
            for (int x = 0; x < V; ++x) {
                const float4 f = *reinterpret_cast<const float4 *>(a.conv_w + ((int64_t)h * 3 * D + part3 * D + c + x) * 4);
                w[x][0] = f.x, w[x][1] = f.y, w[x][2] = f.z, w[x][3] = f.w;
            }
            for (int t = tid / kGroups; t < n; t += kAt) {
                float y[V];
#pragma unroll
                for (int x = 0; x < V; ++x) y[x] = 0.f;
                int i = t, back = 0;                             // draft, or rows into the window
#pragma unroll
                for (int tap = 3; tap >= 0; --tap) {
                    const T *at = i >= 0 ? reinterpret_cast<const T *>(raw_at(a, src, r.first + i, h, D, c, sizeof(T)))
                                         : reinterpret_cast<const T *>(obj_addr(a.pool, pages, win_off + ((uint64_t)(2 - back) * 3 * D + part3 * D + c) * sizeof(T), a.status));
                    float x4[V];
                    load_vec(at, x4);
#pragma unroll
                    for (int x = 0; x < V; ++x) y[x] = fmaf(w[x][tap], x4[x], y[x]);
                    if (i >= 0) i = up[i];
                    else ++back;
                }
#pragma unroll
                for (int x = 0; x < V; ++x) dst[t * D + c + x] = y[x];
            }
        }
        for (int i = tid; i < n * (D / V); i += NT) {
            const int t = i / (D / V), ch = i % (D / V) * V;
            float x[V];
            load_vec(reinterpret_cast<const T *>(raw_at(a, a.alpha, r.first + t, h, D, ch, sizeof(T))), x);
#pragma unroll
            for (int y = 0; y < V; ++y) al[t * D + ch + y] = x[y];
        }
    }
    __syncthreads();
    // ---- a warp a draft: up its branch, a lane D / 32 channels
    constexpr int C = D / 32;
#pragma unroll 1
    for (int t = warp; t < n; t += kWarps) {
        float kr[C], qr[C];
#pragma unroll
        for (int x = 0; x < C; ++x) kr[x] = kb[t * D + lane + 32 * x], qr[x] = xq[t * D + lane + 32 * x];
        uint64_t m = mask[t];
        int i = t;
        for (;;) {
            float dk = 0.f, dq = 0.f;
#pragma unroll
            for (int x = 0; x < C; ++x) {
                const float ki = kb[i * D + lane + 32 * x];
                dk = fmaf(kr[x], ki, dk), dq = fmaf(qr[x], ki, dq);
            }
#pragma unroll
            for (int y = 16; y; y >>= 1) dk += __shfl_xor_sync(0xFFFFFFFFu, dk, y), dq += __shfl_xor_sync(0xFFFFFFFFu, dq, y);
            if (lane == 0) ck[t * N + i] = dk, cq[t * N + i] = dq;
#pragma unroll
            for (int x = 0; x < C; ++x) {
                const float f = al[i * D + lane + 32 * x];
                kr[x] *= f, qr[x] *= f;
            }
            m &= ~(1ull << i);
            if (!m) break;
            i = 63 - __clzll((long long)m);
        }
#pragma unroll
        for (int x = 0; x < C; ++x) xk[t * D + lane + 32 * x] = kr[x], xq[t * D + lane + 32 * x] = qr[x];
    }
    __syncthreads();
    // ---- rows of [A k | A q] times S_0, in their places, eight at a time: each group sums its half of the channels
    for (int r0 = 0; r0 < 2 * n; r0 += 8) {
        float y[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            y[x] = 0.f;
            const int row = r0 + x;
            if (row < 2 * n) {
                const float4 *v = reinterpret_cast<const float4 *>((row < n ? xk + row * D : xq + (row - n) * D) + half * (D / 2));
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const float4 f = v[i];
                    y[x] = fmaf(f.x, s[4 * i], y[x]), y[x] = fmaf(f.y, s[4 * i + 1], y[x]);
                    y[x] = fmaf(f.z, s[4 * i + 2], y[x]), y[x] = fmaf(f.w, s[4 * i + 3], y[x]);
                }
            }
        }
        if (half)
#pragma unroll
            for (int x = 0; x < 8; ++x) part[x * D + j] = y[x];
        __syncthreads();
        if (!half)
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const int row = r0 + x;
                if (row < 2 * n) (row < n ? xk + row * D : xq + (row - n) * D)[j] = y[x] + part[x * D + j];
            }
        __syncthreads();
    }
    // ---- u, column by column
    if (!half) {
#pragma unroll 1
        for (int t = 0; t < n; ++t) {
            float acc = xk[t * D + j];
            for (uint64_t m = mask[t] & ~(1ull << t); m; m &= m - 1) {
                const int i = __ffsll((long long)m) - 1;
                acc = fmaf(ck[t * N + i], u[i * D + j], acc);
            }
            u[t * D + j] = beta[t] * (u[t * D + j] - acc);
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int t = half; t < n; t += 2) {
        float acc = xq[t * D + j];
        for (uint64_t m = mask[t]; m; m &= m - 1) {
            const int i = __ffsll((long long)m) - 1;
            acc = fmaf(cq[t * N + i], u[i * D + j], acc);
        }
        st_elem(static_cast<T *>(a.o) + ((r.first + t) * a.H + h) * D + j, acc);
    }
}

// The state after the accepted branch: decode steps of its drafts one after another with the state in registers,
// read and written once.  Warp w of 16 has D / 16 rows of S, a lane D / 32 columns.
constexpr int kAccThreads = 512, kAccWarps = 16;

template <int D, class T>
__global__ void __launch_bounds__(kAccThreads) verify_tree_accept_kernel(const __grid_constant__ VerifyTreeArgs a, int N) {
    constexpr int V = kVec<T>, C3 = 3 * D, R = D / kAccWarps, C = D / 32;
    extern __shared__ __align__(16) float sm[];
    float *kb = sm, *vb = kb + N * D, *al = vb + N * D, *red = al + N * D, *w = red + kAccWarps * D;
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

template <class K>
cudaError_t launch(K kern, const VerifyTreeArgs &a, int threads, int64_t smem, int N, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)(a.B * a.H), threads, (size_t)smem, st>>>(a, N);
    return cudaGetLastError();
}

template <int D, class T>
cudaError_t verify(const VerifyTreeArgs &a, cudaStream_t st) {
    const int N = (a.max_q + 7) / 8 * 8;
    return launch(verify_tree_kernel<D, T>, a, 2 * D, Lay<D>::bytes(N), N, st);
}

template <int D, class T>
cudaError_t accept(const VerifyTreeArgs &a, cudaStream_t st) {
    const int N = (a.max_q + 7) / 8 * 8;
    const int64_t smem = ((int64_t)3 * N * D + kAccWarps * D + D + 2 * kMost) * 4 + 9 * D * (int64_t)sizeof(T);
    return launch(verify_tree_accept_kernel<D, T>, a, kAccThreads, smem, N, st);
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
