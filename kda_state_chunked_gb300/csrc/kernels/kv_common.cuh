// Device helpers of the key/value-cache kernels: where a token lies in a page, and what a
// sequence's row of the call's metadata says.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace kda {

// Bytes of one token's row of a K or V tile.
template <int FMT, int D>
constexpr int kKvRow = D * (FMT == KDA_KV_I8 ? 1 : 2);

// Byte of (token slot t, byte b of its row) in a K or V tile: rows are cut into 128-byte lines,
// line block after line block, and the 16-byte units of a line are XOR-ed with the slot, so that
// eight slots' units of one column lie in eight different bank groups of shared memory.
template <int ROW>
__host__ __device__ __forceinline__ uint32_t kv_tile_off(uint32_t pt, uint32_t t, uint32_t b) {
    if (ROW == 64) return t * 64u + ((((b >> 4) ^ (t >> 1)) & 3u) << 4) + (b & 15u);
    return (b >> 7) * pt * 128u + t * 128u + (((((b >> 4) & 7u) ^ t) & 7u) << 4) + (b & 15u);
}

// Record of (page id, head); null, and the status bit set, for an id outside the pool.
__device__ __forceinline__ uint8_t *kv_record(const KvView &kv, int32_t id, int32_t head) {
    if ((uint32_t)id >= (uint32_t)kv.num_pages) {
        flag_status(kv.status, KDA_DEV_BAD_PAGE);
        return nullptr;
    }
    return kv.base + (int64_t)id * kv.page_bytes + (int64_t)head * kv.rec_bytes;
}

// One sequence of a call: its first packed token, its new tokens and its tokens in the cache.
// Metadata that does not fit sets KDA_DEV_BAD_META and reads as a sequence without new tokens.
struct KvSeq {
    int32_t tok0, n, len;
};
__device__ __forceinline__ KvSeq kv_seq(const int32_t *cu, const int32_t *kv_len, int32_t s, int64_t T_tot,
                                        int32_t max_q, const KvView &kv) {
    const int32_t a = __ldg(cu + s), b = __ldg(cu + s + 1), len = __ldg(kv_len + s);
    const int64_t n = (int64_t)b - a;
    if (a < 0 || n < 0 || b > T_tot || n > max_q || len < 0 || len > (int64_t)kv.max_pages * kv.page_tokens) {
        flag_status(kv.status, KDA_DEV_BAD_META);
        return {0, 0, 0};
    }
    return {a, (int32_t)n, len};
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

// The last s in [0, nseq) with start(s) <= x, for a start() that does not fall; 0 if there is none.
// The whole warp calls it with one x: 32 places are looked at a time, so that 1,024 sequences take
// two reads one behind the other and not ten.
template <class F>
__device__ __forceinline__ int32_t kv_find(int32_t nseq, int64_t x, F start) {
    int32_t lo = 0, n = nseq;   // start(lo) <= x, or lo = 0; the answer is in [lo, lo + n)
    const int lane = threadIdx.x % 32;
    while (n > 1) {
        const int32_t step = (n + 31) / 32, at = lo + lane * step;
        const bool below = at < lo + n && (at == lo || start(at) <= x);
        const int32_t k = 31 - __clz(__ballot_sync(0xFFFFFFFFu, below));
        const int32_t end = lo + n;
        lo += k * step;
        n = min(step, end - lo);
    }
    return lo;
}

}  // namespace kda
