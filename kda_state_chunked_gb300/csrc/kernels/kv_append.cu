// Filling and reading the paged key/value cache.
//
// kv_append_kernel writes the call's new keys and values into their blocks and rotates queries and
// keys by position on the way:
//   halves  y_i = x_i c_i - x_{i+R/2} s_i,  y_{i+R/2} = x_{i+R/2} c_i + x_i s_i   (i < R/2)
//   pairs   the same for (x_{2i}, x_{2i+1})
// Products and sums are rounded one by one in fp32, never contracted, so a code does not depend on
// how the compiler orders them.  In the 8-bit form a block's scale for a head is
//   s = max(max |x| over its new tokens / 127, s_old if it holds older tokens)
// and a code is rne(x / s), both divisions IEEE fp32 (the rule of the 8-bit checkpoints).  When s
// grows, the older codes c become rne(c s_old / s): the values they stood for, rounded again.
//
// Bound: bytes.  A CTA takes one (block, head, K or V): the block's new rows stay in registers
// between the maximum and the codes, so every input is read once and every code written once.  A
// thread holds 8 + 8 elements of a row, the two places that rotate together, and so needs no
// exchange with another thread.  Query rows are handled by CTAs of their own in the same launch.
//
// Measured: 4 x 8192 tokens, 16 + 16 heads of 128, 16-bit cache: 162 us, 5.0 TB/s, 74% of the copy
// rate; 256 single tokens, 32 + 8 heads, 8-bit: 8.3 us, where a block of codes is opened or its scale
// looked at for each (latency).  kv_gather_kernel: those 32768 rows back in 83 us, 6.5 TB/s; the 256
// blocks in 12.0 us.
#include <cuda_bf16.h>

#include "kv_common.cuh"

namespace kda {
namespace {

__device__ __forceinline__ void unpack8(const uint4 &u, float *x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float *x) { unpack8(*reinterpret_cast<const uint4 *>(p), x); }
__device__ __forceinline__ void load8(const float *p, float *x) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ uint4 pack8(const float *x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float *x) { *reinterpret_cast<uint4 *>(p) = pack8(x); }
__device__ __forceinline__ void store8(float *p, const float *x) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// Places of the two groups of eight that thread c of a row holds: the halves that rotate
// together, or sixteen neighbours (pairs, and what is not rotated).
struct Place {
    int a, b;
    bool turned;
};
__device__ __forceinline__ Place place(int c, int rot, bool interleaved) {
    const bool turned = 16 * c < rot;
    if (turned && !interleaved) return {8 * c, rot / 2 + 8 * c, true};
    return {16 * c, 16 * c + 8, turned};
}

__device__ __forceinline__ void turn(float &u, float &w, float co, float si) {
    const float a = __fsub_rn(__fmul_rn(u, co), __fmul_rn(w, si));
    w = __fadd_rn(__fmul_rn(w, co), __fmul_rn(u, si));
    u = a;
}

// Rotate x (8 + 8 elements of thread c) by the table row cs of the token's position.
__device__ __forceinline__ void rotate(float (&x)[16], const float *cs, int c, int rot, bool interleaved) {
    float co[8], si[8];
    load8(cs + 8 * c, co);
    load8(cs + rot / 2 + 8 * c, si);
    if (interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) turn(x[2 * j], x[2 * j + 1], co[j], si[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) turn(x[j], x[j + 8], co[j], si[j]);
    }
}

__device__ __forceinline__ int8_t code_of(float x, float s) {
    const int c = __float2int_rn(__fdiv_rn(x, s));
    return (int8_t)max(-127, min(127, c));
}
// Eight codes of values x at scale s; all zero where the scale is (nothing but zeros, or so small
// that a 127th of it is not a number of its own).
__device__ __forceinline__ uint2 codes8(const float *x, float s) {
    uint32_t w[2] = {0, 0};
    if (s != 0.f)
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i >> 2] |= (uint32_t)(uint8_t)code_of(x[i], s) << (8 * (i & 3));
    return make_uint2(w[0], w[1]);
}

constexpr int kMaxToks = 128;   // tokens of a CTA that rotates queries

// A sequence with no place, or no angle, for some of its new tokens: all of it is skipped, queries too.
__device__ __forceinline__ bool no_place(const KvAppendArgs &a, const KvSeq &q) {
    return q.len < q.n || (a.rot_dim > 0 && q.len > a.max_pos);
}

// NT threads; ROWS: new rows of a block that one thread may hold.
template <int FMT, int D, class TIN, int NT, int ROWS>
__global__ void __launch_bounds__(NT) kv_append_kernel(KvAppendArgs a, int32_t q_ctas, int32_t q_toks, int64_t items) {
    constexpr int kTpr = D / 16;          // threads a row
    constexpr int kRpp = NT / kTpr;       // rows a pass
    constexpr int kRow = kKvRow<FMT, D>;
    const int tid = threadIdx.x;
    const bool il = a.interleaved != 0;
    const int rot = a.rot_dim;

    if ((int)blockIdx.x < q_ctas) {
        // a token's place in its sequence, by one warp a token; none where the sequence is skipped
        __shared__ int64_t place_of[kMaxToks];
        const int64_t t_lo = (int64_t)blockIdx.x * q_toks;
        const int per_tok = a.Hq * kTpr;
        for (int i = tid / 32; i < q_toks; i += NT / 32) {
            const int64_t tok = t_lo + i;
            if (tok >= a.T_tot) break;
            const int s = kv_find(a.nseq, tok, [&](int m) { return (int64_t)__ldg(a.cu_q + m); });
            const KvSeq q = kv_seq(a.cu_q, a.kv_len, s, a.T_tot, a.max_q, a.kv);
            int64_t pos = (int64_t)q.len - q.n + (tok - q.tok0);
            if (tok < q.tok0 || tok >= (int64_t)q.tok0 + q.n) pos = -1;
            else if (no_place(a, q)) {
                flag_status(a.kv.status, KDA_DEV_BAD_META);
                pos = -1;
            }
            if (tid % 32 == 0) place_of[i] = pos;
        }
        __syncthreads();
        for (int i = tid; i < q_toks * per_tok; i += NT) {
            const int64_t tok = t_lo + i / per_tok;
            if (tok >= a.T_tot) break;
            const int64_t pos = place_of[i / per_tok];
            if (pos < 0) continue;
            const int h = (i % per_tok) / kTpr, c = i % kTpr;
            const Place p = place(c, rot, il);
            const TIN *src = static_cast<const TIN *>(a.q) + tok * a.q_stride + h * D;
            float x[16];
            load8(src + p.a, x);
            load8(src + p.b, x + 8);
            if (p.turned) rotate(x, a.cos_sin + pos * rot, c, rot, il);
            TIN *dst = static_cast<TIN *>(a.q_out) + (tok * a.Hq + h) * D;
            store8(dst + p.a, x);
            store8(dst + p.b, x + 8);
        }
        return;
    }

    // (block slot, head, K or V); the heads of a block side by side
    const uint32_t w = blockIdx.x - q_ctas;
    const bool is_v = (w & 1u) != 0;
    const int head = (int)((w >> 1) % (uint32_t)a.kv.Hkv);
    const int64_t item = (w >> 1) / (uint32_t)a.kv.Hkv;
    const int pt = a.kv.page_tokens;
    int s, block;
    KvSeq q;
    if (a.max_q == 1) {
        // a token is a block's only new one
        s = kv_find(a.nseq, item, [&](int m) { return (int64_t)__ldg(a.cu_q + m); });
        q = kv_seq(a.cu_q, a.kv_len, s, a.T_tot, a.max_q, a.kv);
        if (item < q.tok0 || item >= (int64_t)q.tok0 + q.n) return;
        block = (q.len - q.n) / pt;
    } else {
        // sequence m owns block slots cu[m] / pt + 2 m and up: as many as n tokens can touch
        auto start = [&](int m) { return (int64_t)(__ldg(a.cu_q + m) / pt) + 2 * (int64_t)m; };
        s = kv_find(a.nseq, item, start);
        q = kv_seq(a.cu_q, a.kv_len, s, a.T_tot, a.max_q, a.kv);
        if (q.n == 0 || item < start(s)) return;
        const int64_t b = (int64_t)((q.len - q.n) / pt) + (item - start(s));
        if (b * pt >= q.len && !no_place(a, q)) return;
        block = (int)b;
    }
    const int old = q.len - q.n;
    if (no_place(a, q)) {
        if (tid == 0) flag_status(a.kv.status, KDA_DEV_BAD_META);
        return;
    }
    const int32_t page = __ldg(a.kv.table + (int64_t)s * a.kv.max_pages + block);   // used when the rows are under way
    const int lo = max(old - block * pt, 0), hi = min(q.len - block * pt, pt);   // slots of the new rows
    const int64_t tok_of_slot0 = (int64_t)q.tok0 + (int64_t)block * pt - old;

    const int c = tid % kTpr, r0 = tid / kTpr;
    const Place p = is_v ? Place{16 * c, 16 * c + 8, false} : place(c, rot, il);
    const TIN *src = is_v ? static_cast<const TIN *>(a.v) : static_cast<const TIN *>(a.k);
    const int64_t stride = is_v ? a.v_stride : a.k_stride;
    float x[ROWS][16];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int slot = lo + i * kRpp + r0;
        if (slot < hi) {
            const TIN *row = src + (tok_of_slot0 + slot) * stride + head * D;
            load8(row + p.a, x[i]);
            load8(row + p.b, x[i] + 8);
        }
    }
    uint8_t *rec = kv_record(a.kv, page, head);
    if (!rec) return;
    uint8_t *tile = rec + (is_v ? pt * kRow : 0);
    float *scale_at = reinterpret_cast<float *>(rec + 2 * pt * kRow) + (is_v ? 1 : 0);
    uint32_t s_old = 0;
    if (FMT == KDA_KV_I8 && lo > 0) s_old = __float_as_uint(*scale_at) & 0x7FFFFFFFu;
    if (p.turned) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int slot = lo + i * kRpp + r0;
            if (slot < hi) rotate(x[i], a.cos_sin + ((int64_t)block * pt + slot) * rot, c, rot, il);
        }
    }
    if constexpr (FMT == KDA_KV_BF16) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int slot = lo + i * kRpp + r0;
            if (slot < hi) {
                *reinterpret_cast<uint4 *>(tile + kv_tile_off<kRow>(pt, slot, 2 * p.a)) = pack8(x[i]);
                *reinterpret_cast<uint4 *>(tile + kv_tile_off<kRow>(pt, slot, 2 * p.b)) = pack8(x[i] + 8);
            }
        }
    } else {
        // The maximum goes by the bits of |x|: an infinity or a NaN wins, so that a block that holds
        // one reads as NaN instead of losing it.
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (lo + i * kRpp + r0 < hi)
#pragma unroll
                for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(x[i][j]) & 0x7FFFFFFFu);
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        __shared__ uint32_t tops[NT / 32];
        if (tid % 32 == 0) tops[tid / 32] = top;
        __syncthreads();   // behind it every thread has read the old scale
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) top = max(top, tops[i]);
        const uint32_t s_bits = max(__float_as_uint(__fdiv_rn(__uint_as_float(top), 127.f)) & 0x7FFFFFFFu, s_old);
        const float sc = __uint_as_float(s_bits);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int slot = lo + i * kRpp + r0;
            if (slot < hi) {
                *reinterpret_cast<uint2 *>(tile + kv_tile_off<kRow>(pt, slot, p.a)) = codes8(x[i], sc);
                *reinterpret_cast<uint2 *>(tile + kv_tile_off<kRow>(pt, slot, p.b)) = codes8(x[i] + 8, sc);
            }
        }
        if (lo > 0 && s_bits != s_old) {
            const float so = __uint_as_float(s_old);
            for (int i = tid; i < lo * (kRow / 8); i += NT) {   // rows below lo: whole, in any order of units
                const int slot = i / (kRow / 8);
                uint2 *at = reinterpret_cast<uint2 *>(tile + kv_tile_off<kRow>(pt, slot, 8 * (i % (kRow / 8))));
                const uint2 u = *at;
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __fmul_rn((float)(int8_t)((j < 4 ? u.x : u.y) >> (8 * (j & 3))), so);
                *at = codes8(v, sc);
            }
        }
        if (tid == 0) *scale_at = sc;
    }
}

// Cached ranges as values.  A thread takes 16 elements of K and of V of one head, in kGatherRows rows
// whose loads are under way together; neighbours take the next elements and heads, so a warp writes
// whole lines of both outputs.
constexpr int kGatherRows = 2;
template <int FMT, int D, class TOUT>
__global__ void __launch_bounds__(256) kv_gather_kernel(KvGatherArgs a) {
    constexpr int kTpr = D / 16, kRow = kKvRow<FMT, D>;
    const uint32_t per_row = a.kv.Hkv * kTpr, i = blockIdx.x * 256u + threadIdx.x;   // below 2^31 threads a launch
    const int64_t row0 = a.row0 + (int64_t)(i / per_row) * kGatherRows;
    const int c = (int)(i % kTpr), head = (int)(i % per_row) / kTpr, pt = a.kv.page_tokens;
    // the warp's first row's sequence; a thread steps on from there
    int s = kv_find(a.nseq, __shfl_sync(0xFFFFFFFFu, row0, 0), [&](int m) { return (int64_t)__ldg(a.cu_out + m); });
    int32_t page[kGatherRows], slot[kGatherRows], wrong = 0;
    bool mine[kGatherRows];
#pragma unroll
    for (int r = 0; r < kGatherRows; ++r) {
        const int64_t row = row0 + r;
        mine[r] = row < a.T_out;
        page[r] = slot[r] = 0;
        if (!mine[r]) continue;
        while (s + 1 < a.nseq && __ldg(a.cu_out + s + 1) <= row) ++s;
        const int64_t at = __ldg(a.cu_out + s), end = __ldg(a.cu_out + s + 1), first = __ldg(a.begin + s);
        mine[r] = row >= at && row < end;               // rows that no sequence owns stay as they are
        const int64_t tok = first + (row - at);
        if (mine[r] && (first < 0 || tok >= (int64_t)a.kv.max_pages * pt)) {
            wrong |= KDA_DEV_BAD_META;
            mine[r] = false;
        }
        if (!mine[r]) continue;
        const int block = (int)tok / pt;
        slot[r] = (int)tok - block * pt;
        page[r] = __ldg(a.kv.table + (int64_t)s * a.kv.max_pages + block);
    }
    const uint8_t *rec[kGatherRows];
#pragma unroll
    for (int r = 0; r < kGatherRows; ++r) {
        const bool there = (uint32_t)page[r] < (uint32_t)a.kv.num_pages;
        if (mine[r] && !there) wrong |= KDA_DEV_BAD_PAGE;
        rec[r] = mine[r] && there ? a.kv.base + (int64_t)page[r] * a.kv.page_bytes + (int64_t)head * a.kv.rec_bytes : nullptr;
    }
    if (wrong) flag_status(a.kv.status, wrong);
    constexpr int kUnits = FMT == KDA_KV_I8 ? 1 : 2;    // 16-byte units of 16 elements
    uint4 u[kGatherRows][2][kUnits];
    float2 sc[kGatherRows];
#pragma unroll
    for (int r = 0; r < kGatherRows; ++r) {
        if (!rec[r]) continue;
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int y = 0; y < kUnits; ++y)
                u[r][v][y] = *reinterpret_cast<const uint4 *>(rec[r] + v * pt * kRow +
                                                              kv_tile_off<kRow>(pt, slot[r], 16 * (kUnits * c + y)));
        if (FMT == KDA_KV_I8) sc[r] = *reinterpret_cast<const float2 *>(rec[r] + 2 * pt * kRow);
    }
#pragma unroll
    for (int r = 0; r < kGatherRows; ++r) {
        if (!rec[r]) continue;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            TOUT *out = static_cast<TOUT *>(v ? a.v_out : a.k_out) + ((row0 + r) * a.kv.Hkv + head) * D + 16 * c;
            float x[16];
            if constexpr (FMT == KDA_KV_I8) {
                const uint4 z = u[r][v][0];
                const uint32_t w[4] = {z.x, z.y, z.z, z.w};
                const float f = v ? sc[r].y : sc[r].x;
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = __fmul_rn((float)(int8_t)(w[j >> 2] >> (8 * (j & 3))), f);
            } else {
#pragma unroll
                for (int y = 0; y < kUnits; ++y) unpack8(u[r][v][y], x + 8 * y);
            }
            store8(out, x);
            store8(out + 8, x + 8);
        }
    }
}

template <int FMT, int D, class TIN, int NT, int ROWS>
cudaError_t append(const KvAppendArgs &a, cudaStream_t st) {
    // about four pairs of eights a thread for the queries' CTAs
    const int32_t q_toks = a.q ? min(kMaxToks, max(1, 4 * NT / (a.Hq * (D / 16)))) : 1;
    const int64_t q_ctas = a.q ? (a.T_tot + q_toks - 1) / q_toks : 0;
    const int64_t items = a.max_q == 1 ? a.T_tot : a.T_tot / a.kv.page_tokens + 2 * (int64_t)a.nseq;
    const int64_t grid = q_ctas + 2 * items * a.kv.Hkv;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    kv_append_kernel<FMT, D, TIN, NT, ROWS><<<(unsigned)grid, NT, 0, st>>>(a, (int32_t)q_ctas, q_toks, items);
    return cudaGetLastError();
}

// Few new tokens a sequence leave all but one row of a block's threads idle, so small CTAs take
// them; a CTA of 256 holds a whole block of new rows, and one made for blocks of up to 64 tokens
// needs half the registers of the largest, so that more of them have loads under way on an SM
// (4 x 8192 tokens in 64-token blocks: 162 us, and 263 us with the largest's registers).
template <int FMT, int D, class TIN>
cudaError_t append_sized(const KvAppendArgs &a, cudaStream_t st) {
    constexpr int kMost = kKvMaxPageTokens * (D / 16) / 256;
    if (a.max_q <= 8) return append<FMT, D, TIN, 64, 1>(a, st);
    if (a.kv.page_tokens <= kKvMaxPageTokens / 2) return append<FMT, D, TIN, 256, kMost / 2>(a, st);
    return append<FMT, D, TIN, 256, kMost>(a, st);
}

template <int FMT, int D>
cudaError_t gather(const KvGatherArgs &a, cudaStream_t st) {
    KvGatherArgs part = a;
    const int64_t per_row = (int64_t)a.kv.Hkv * (D / 16), most = ((int64_t)1 << 30) / per_row * kGatherRows;   // rows a launch
    for (part.row0 = 0; part.row0 < a.T_out; part.row0 += most) {
        const int64_t rows = min(most, a.T_out - part.row0);
        const unsigned grid = (unsigned)(((rows + kGatherRows - 1) / kGatherRows * per_row + 255) / 256);
        if (a.dtype == KDA_F32) kv_gather_kernel<FMT, D, float><<<grid, 256, 0, st>>>(part);
        else kv_gather_kernel<FMT, D, __nv_bfloat16><<<grid, 256, 0, st>>>(part);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs &a, cudaStream_t s) {
    const bool i8 = a.kv.fmt == KDA_KV_I8, f32 = a.dtype == KDA_F32;
    if (a.kv.d == 128) {
        if (i8) return f32 ? append_sized<KDA_KV_I8, 128, float>(a, s) : append_sized<KDA_KV_I8, 128, __nv_bfloat16>(a, s);
        return f32 ? append_sized<KDA_KV_BF16, 128, float>(a, s) : append_sized<KDA_KV_BF16, 128, __nv_bfloat16>(a, s);
    }
    if (i8) return f32 ? append_sized<KDA_KV_I8, 64, float>(a, s) : append_sized<KDA_KV_I8, 64, __nv_bfloat16>(a, s);
    return f32 ? append_sized<KDA_KV_BF16, 64, float>(a, s) : append_sized<KDA_KV_BF16, 64, __nv_bfloat16>(a, s);
}

cudaError_t launch_kv_gather(const KvGatherArgs &a, cudaStream_t s) {
    if (a.kv.d == 128) return a.kv.fmt == KDA_KV_I8 ? gather<KDA_KV_I8, 128>(a, s) : gather<KDA_KV_BF16, 128>(a, s);
    return a.kv.fmt == KDA_KV_I8 ? gather<KDA_KV_I8, 64>(a, s) : gather<KDA_KV_BF16, 64>(a, s);
}

}  // namespace kda
