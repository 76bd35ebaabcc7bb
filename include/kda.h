/*
 * kda.h — C ABI of the KDA state library (libkda.so) for one GB300 GPU (sm_103a).
 *
 * The library computes the Kimi Delta Attention (KDA) state path:
 *   - a chunked varlen prefill that reads q, k, v, alpha, beta, applies the width-4 causal
 *     depthwise conv to q | k | v, runs the recurrence
 *         S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T,  o_t = S_t^T q_t
 *     (decay first, then the delta-rule write, then the read: "Lesson 01 · Architecture
 *     map", §两种 Attention，两种状态), writes o, streams checkpoints of (S, conv window) at
 *     a sparse subset of 512-token hash-block ends into a paged pool ("Cache de préfixe
 *     hybride KDA–MLA", §La solution and §Le fonctionnement du prefill) and writes the
 *     final state to the sequence's private (active) object;
 *   - resume from any checkpoint: copy it into the private object, then prefill with
 *     has_init = 1 (same page, §Les checkpoints sont en lecture seule);
 *   - a batched single-token decode step that gathers each request's state through a page
 *     table and updates it in place ("KIMI K3 경량 복제에서 본 KDA의 AI 인프라 과제",
 *     §0x08 8.2.2: conv state and recurrent state handed to a fused decode kernel).
 *
 * Conventions
 * -----------
 * - Every function returns a kda_status (int); functions that return a count return it as
 *   a non-negative value and errors as negative kda_status values.
 * - dtype: KDA_F32 or KDA_BF16; it is the type of q, k, v, alpha, beta, o and of the conv
 *   window stored in records.  The recurrent state is always fp32.  conv_w is always fp32.
 * - "device" pointers are CUDA device addresses on the current device; "host" pointers are
 *   ordinary host memory that is read (or written) before the call returns.
 * - The caller owns every device buffer (inputs, outputs, the pool base, page tables, the
 *   workspace and the int32 device status word).  The library owns only the host-side pool
 *   metadata behind the opaque kda_pool (free set, reference counts) and a few pinned host
 *   staging buffers that carry call metadata to the workspace.
 * - GPU work is enqueued asynchronously on `stream` (a cudaStream_t; NULL = legacy default
 *   stream).  Buffers handed to a call must stay alive until that work completes.
 * - Nothing aborts or traps.  Host-side argument errors return KDA_EINVAL / KDA_ENOPAGES /
 *   KDA_EREF before anything is enqueued.  Kernels check page ids and metadata and, on a bad
 *   value, skip the access and set a bit in *status_dev; kda_sync_status reports it as
 *   KDA_EDEVICE.  CUDA launch errors return KDA_ECUDA.
 * - A kda_pool may be used from one host thread at a time.
 *
 * Paged state layout (bit-exact)
 * ------------------------------
 * One page byte size for the whole pool.  A head record is S as fp32 row-major [d][d]
 * (row i = key channel i, column j = value channel j), then the conv window [3][3d] in
 * dtype (oldest raw token first, channels q | k | v), zero-padded to a multiple of 256
 * bytes.  An object is the H head records of one sequence, one after another in head order
 * (heads stored contiguously: "Cache de préfixe hybride KDA–MLA", §La mise en page
 * unifiée).  Logical byte x of an object lives in page list[x / page_bytes] at byte
 * x % page_bytes of that page; the page lists are int32 [P] with P = kda_object_pages().
 */
#ifndef KDA_H
#define KDA_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum kda_status_code {
    KDA_OK = 0,
    KDA_EINVAL = -1,    /* bad argument, shape, dtype, position or size */
    KDA_ENOPAGES = -2,  /* pool exhausted: nothing was allocated */
    KDA_EREF = -3,      /* reference-count misuse (freeing a free page, claiming a used one) */
    KDA_ECUDA = -4,     /* CUDA launch / runtime error */
    KDA_EDEVICE = -5    /* a kernel found a bad page id, bad metadata or an out-of-range decay
                           (see kda_sync_status) */
} kda_status_code;

typedef enum kda_dtype { KDA_F32 = 0, KDA_BF16 = 1 } kda_dtype;

/* Device status bits set by kernels (reported through kda_sync_status). */
#define KDA_DEV_BAD_PAGE 1   /* a page id outside [0, num_pages) was met; access skipped */
#define KDA_DEV_BAD_META 2   /* inconsistent metadata in the workspace; work skipped */
#define KDA_DEV_TIMEOUT 4    /* an internal pipeline wait gave up; that sequence is incomplete */
#define KDA_DEV_RANGE 8      /* prefill: a chunk's decay product fell below the supported range
                                (see alpha in kda_prefill_varlen); that sequence's results are undefined */

typedef struct kda_pool kda_pool;

/* ---------------------------------------------------------------- sizes --------------- */

/* Bytes of one head record for head dimension d (64 or 128) and dtype; KDA_EINVAL if bad. */
int64_t kda_record_bytes(int32_t d, int32_t dtype);

/* Bytes of one object (H records).  KDA_EINVAL if bad. */
int64_t kda_object_bytes(int32_t H, int32_t d, int32_t dtype);

/* Pages per object in this pool: ceil(kda_object_bytes / page_bytes).  KDA_EINVAL if bad. */
int32_t kda_object_pages(const kda_pool *pool, int32_t H, int32_t d, int32_t dtype);

/* ---------------------------------------------------------------- pool ---------------- */
/* One refcounted page allocator for every state object ("Cache de préfixe hybride
 * KDA–MLA", §La mise en page unifiée: one allocation / reference-count / eviction path for
 * all page kinds).  Device memory for the pages is the caller's: num_pages * page_bytes
 * bytes at `pool_base`, passed to each GPU call. */

/* page_bytes must be a positive multiple of 256; num_pages > 0.  *out receives the pool. */
int kda_pool_create(int64_t page_bytes, int32_t num_pages, kda_pool **out);
/* Frees the pool's host metadata and its pinned staging buffers, first waiting for any
 * upload still reading them; the caller's device pages are untouched.  KDA_EINVAL for NULL. */
int kda_pool_destroy(kda_pool *pool);
/* The page size in bytes, the number of pages, and the number of free pages (reference count
 * 0).  KDA_EINVAL for NULL. */
int64_t kda_pool_page_bytes(const kda_pool *pool);
int32_t kda_pool_num_pages(const kda_pool *pool);
int32_t kda_pool_free_count(const kda_pool *pool);

/* Allocate n pages, lowest free id first, each with refcount 1; ids written to out_ids[n].
 * KDA_ENOPAGES (nothing allocated) if fewer than n pages are free. */
int kda_page_alloc(kda_pool *pool, int32_t n, int32_t *out_ids);

/* Take the n given free pages (refcount 0 -> 1), e.g. to follow a caller's page table.
 * KDA_EREF if any is in use or repeated, KDA_EINVAL if out of range; all or nothing. */
int kda_page_claim(kda_pool *pool, int32_t n, const int32_t *ids);

/* Pin (refcount + 1) n pages that are in use; KDA_EREF if one is free.  All or nothing.
 * Pinning every hit page before any allocation is the first concurrency rule of "Cache de
 * préfixe hybride KDA–MLA", §La cohérence sous ordonnancement concurrent. */
int kda_page_incref(kda_pool *pool, int32_t n, const int32_t *ids);

/* Unpin n pages; a page is free again at refcount 0.  KDA_EREF if a count would go below
 * zero (repeated ids count once per occurrence).  All or nothing. */
int kda_page_decref(kda_pool *pool, int32_t n, const int32_t *ids);

/* Refcount of page id, or KDA_EINVAL if out of range. */
int32_t kda_page_refcount(const kda_pool *pool, int32_t id);

/* ---------------------------------------------------------------- policy -------------- */

/* Checkpoint positions of one forward over absolute positions [start, end): every p with
 * p % (hash_block * stride) == 0 and start < p <= end, plus floor(end / hash_block) *
 * hash_block when include_last != 0 and it is > start ("Cache de préfixe hybride KDA–MLA",
 * §La solution: a sparse subset of hash-block ends; §Le fonctionnement du prefill: persist
 * the last hash-aligned position processed).  Writes up to cap ascending positions to out
 * and returns the total count (which may exceed cap), or KDA_EINVAL. */
int32_t kda_ckpt_positions(int64_t start, int64_t end, int32_t hash_block, int32_t stride,
                           int32_t include_last, int64_t *out, int32_t cap);

/* Plan the checkpoints of one prefill call and allocate their objects.  Sequence s covers
 * absolute positions [start_pos[s], start_pos[s] + cu_seqlens[s+1] - cu_seqlens[s]).
 * Checkpoints are listed in (sequence ascending, position ascending) order and each gets P
 * fresh pages, lowest free first, refcount 1 (new checkpoints go to fresh slots: "Cache de
 * préfixe hybride KDA–MLA", §Les checkpoints sont en lecture seule).  Outputs (host):
 * *out_n, out_seq[cap], out_pos[cap], out_pages[cap * P].  KDA_EINVAL if more than cap
 * checkpoints would result; KDA_ENOPAGES if the pool cannot hold them (nothing allocated).
 * hash_block must be a positive multiple of 64. */
int kda_ckpt_plan(kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t nseq,
                  const int32_t *cu_seqlens, const int64_t *start_pos, int32_t hash_block,
                  int32_t stride, int32_t include_last, int32_t cap, int32_t *out_n,
                  int32_t *out_seq, int64_t *out_pos, int32_t *out_pages);

/* ---------------------------------------------------------------- prefill ------------- */

/* Workspace bytes kda_prefill_varlen needs for this batch (the same arguments as that call):
 *   H, d, dtype            heads, head dimension, token dtype
 *   nseq, cu_seqlens, start_pos   host arrays as in kda_prefill_varlen (they may be NULL when
 *                          the path for this shape needs metadata only: fp32 or d = 64)
 *   n_ckpt, pages_per_object      the checkpoint count of the call and kda_object_pages()
 * For bf16 with d = 128 the workspace also holds the chunk-operand images of the split
 * tensor-core prefill: two slots of at most ~512 MiB of images each (one image of 82,432 B per
 * (chunk, head) of a wave of chunks), plus the state handed between waves (64 KiB per
 * (sequence, head), when there is more than one wave) and the final conv windows.  Returns
 * the byte count, or KDA_EINVAL for a bad shape or inconsistent arrays. */
int64_t kda_prefill_workspace_bytes(int32_t H, int32_t d, int32_t dtype, int32_t nseq,
                                    const int32_t *cu_seqlens, const int64_t *start_pos,
                                    int32_t n_ckpt, int32_t pages_per_object);

/* Number of kernel launches kda_prefill_varlen makes for this batch (same arguments as
 * kda_prefill_workspace_bytes; cu_seqlens / start_pos host arrays): one for fp32 or d = 64;
 * for bf16 with d = 128, two per wave of chunks (chunk preparation and chains, the
 * preparation of a wave overlapping the chains of the one before), or one when every
 * sequence is empty.
 * KDA_EINVAL for a bad shape. */
int32_t kda_prefill_kernel_launches(int32_t H, int32_t d, int32_t dtype, int32_t nseq,
                                    const int32_t *cu_seqlens, const int64_t *start_pos);

/* The wave split of the bf16 d = 128 prefill for this batch (same arguments as
 * kda_prefill_kernel_launches): wave w covers local chunks [wave_c0[w], wave_c0[w + 1]) of
 * every sequence (local chunk 0 = the chunk holding start_pos).  Writes min(cap, W + 1) bounds
 * to the host array wave_c0 (may be NULL when cap = 0) and returns the wave count W (0 when
 * every sequence is empty, or for shapes that do not take the split path).  The split is
 * chosen by a cost model among splits whose operand images fit one workspace slot; it changes
 * speed only, never results.  KDA_EINVAL for a bad shape or inconsistent arrays. */
int32_t kda_prefill_waves(int32_t H, int32_t d, int32_t dtype, int32_t nseq, const int32_t *cu_seqlens,
                          const int64_t *start_pos, int32_t *wave_c0, int32_t cap);

/* Chunked varlen prefill (chunk = 64 tokens, chunks aligned to absolute positions).
 *   H, d, dtype      heads, head dimension (64 or 128), dtype of the token tensors
 *   nseq             number of sequences (>= 1)
 *   cu_seqlens       host int32 [nseq + 1], token offsets into the packed arrays
 *   start_pos        host int64 [nseq], absolute position of each sequence's first token
 *   has_init         host uint8 [nseq]; 1 = read the initial (S, window) from the active
 *                    object, 0 = start from zeros
 *   q, k, v, alpha   device [T_tot][H][d] dtype (q, k as given: any normalisation is the
 *                    caller's; the conv runs here)
 *                    alpha is the forget gate, in [0, 1] per key channel.  The chunked
 *                    kernels factor a chunk's decay through its running product per channel,
 *                    so the product of alpha over each 64-token chunk must stay at or above
 *                    2^-100 in every channel (a geometric-mean gate above 0.34 over a full
 *                    chunk; a gate of exactly 0 is below it).  A chunk below that sets
 *                    KDA_DEV_RANGE, and the outputs, states and checkpoints of its
 *                    (sequence, head) from that chunk on are undefined.  kda_decode_step
 *                    steps token by token and has no such limit.
 *   beta             device [T_tot][H] dtype
 *   conv_w           device fp32 [H][3d][4]; tap j multiplies raw token t-3+j
 *   o                device [T_tot][H][d] dtype, written
 *   pool_base        device base of the page pool
 *   active_pages     host int32 [nseq * P]: each sequence's private object (read when
 *                    has_init, always written with the final state and window)
 *   n_ckpt, ckpt_seq, ckpt_pos, ckpt_pages   host: the checkpoints to stream (as produced
 *                    by kda_ckpt_plan): sequence ids ascending, positions ascending within
 *                    a sequence, each position p with start < p <= end and p % 64 == 0 or
 *                    p == end; ckpt_pages [n_ckpt * P] must be allocated pages
 *   workspace        device scratch (16-byte aligned) of at least
 *                    kda_prefill_workspace_bytes() for the same batch; the call
 *                    writes metadata there (one async host-to-device copy)
 *   status_dev       device int32 status word (bits KDA_DEV_*), OR-ed by the kernel
 * The state checkpoint at p is S after tokens [0, p) with the raw tokens p-3, p-2, p-1 as
 * window, in the record layout above. */
int kda_prefill_varlen(kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t nseq,
                       const int32_t *cu_seqlens, const int64_t *start_pos,
                       const uint8_t *has_init, const void *q, const void *k, const void *v,
                       const void *alpha, const void *beta, const float *conv_w, void *o,
                       void *pool_base, const int32_t *active_pages, int32_t n_ckpt,
                       const int32_t *ckpt_seq, const int64_t *ckpt_pos,
                       const int32_t *ckpt_pages, void *workspace, int64_t ws_bytes,
                       int32_t *status_dev, void *stream);

/* Bytes of the fixed device scratch used by kda_prefill_varlen_noalloc. */
#define KDA_NOALLOC_SCRATCH_BYTES (1 << 20)

/* Allocation-free variant of kda_prefill_varlen.  The source pages have no counterpart:
 * this is an interface convenience of this library.  It serves callers that cannot
 * allocate device memory when they call the prefill: a serving runtime that reserved all
 * of HBM for its own pool at start-up (a cudaMalloc there fails or fragments that pool),
 * or a latency-critical path where cudaMalloc / cudaFree and the device synchronisation
 * they can cause are not allowed.  Arguments and results are those of kda_prefill_varlen
 * without the workspace: the per-call metadata goes to a fixed array of
 * KDA_NOALLOC_SCRATCH_BYTES bytes inside the library's device image, which every GPU that
 * loads the library holds until the process exits.
 *   - Metadata that does not fit (32 bytes per sequence and 16 per checkpoint, each part
 *     rounded up to 256 bytes, plus 4 * (nseq + n_ckpt) * pages_per_object bytes of page
 *     lists) returns KDA_EINVAL and enqueues nothing.
 *   - The first call on each device looks up the array's device address, with that device
 *     current; make that first call before any stream capture.
 *   - Every call reuses the one array and overwrites all of the metadata it reads, so no
 *     state carries over between calls; calls whose GPU work may overlap (different streams
 *     without ordering between them) race on it.  Calls on one stream are ordered.
 *   - It calls no cudaMalloc, cudaFree or other allocating routine: the metadata is built
 *     in a static host buffer and sent with one cudaMemcpyAsync from that pageable buffer.
 *     A copy from pageable memory is staged by the runtime before the call returns, and it
 *     can make the host wait for work already queued on the stream. */
int kda_prefill_varlen_noalloc(kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t nseq,
                               const int32_t *cu_seqlens, const int64_t *start_pos,
                               const uint8_t *has_init, const void *q, const void *k,
                               const void *v, const void *alpha, const void *beta,
                               const float *conv_w, void *o, void *pool_base,
                               const int32_t *active_pages, int32_t n_ckpt,
                               const int32_t *ckpt_seq, const int64_t *ckpt_pos,
                               const int32_t *ckpt_pages, int32_t *status_dev, void *stream);

/* ---------------------------------------------------------------- decode -------------- */

/* One decode step for B requests, one token each.  q, k, v, alpha device [B][H][d] dtype,
 * beta device [B][H] dtype, conv_w device fp32 [H][3d][4], o device [B][H][d] dtype.
 * state_pages device int32 [B * P]: the page table of each request's active object, read
 * and updated in place (S and the conv window: the window is shifted by one token).
 * Page ids outside the pool set KDA_DEV_BAD_PAGE and that (request, head) is skipped. */
int kda_decode_step(const kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t B,
                    const void *q, const void *k, const void *v, const void *alpha,
                    const void *beta, const float *conv_w, void *o, void *pool_base,
                    const int32_t *state_pages, int32_t *status_dev, void *stream);

/* Ping-pong decode step: as kda_decode_step, but each request's state is read from its
 * source object (src_pages, device int32 [B * P]) and written, with the shifted window, to its
 * destination object (dst_pages, device int32 [B * P]).  A request whose two page lists are
 * equal is updated in place; for one whose lists differ (and do not overlap), the source
 * object is left untouched and holds the state at the request's position: a decode-interval
 * checkpoint taken without a copy, which the caller donates to the cache while the request
 * continues on the destination object ("KIMI K3 경량 복제에서 본 KDA의 AI 인프라 과제", §0x05
 * 5.2: decode checkpoints at a fixed interval; §0x06 6.7 and 6.8: a second slot requested at a
 * checkpoint boundary, the new state written to it, the old slot donated).  Page ids outside
 * the pool in either list set KDA_DEV_BAD_PAGE and the request is skipped. */
int kda_decode_step_pp(const kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t B,
                       const void *q, const void *k, const void *v, const void *alpha,
                       const void *beta, const float *conv_w, void *o, void *pool_base,
                       const int32_t *src_pages, const int32_t *dst_pages, int32_t *status_dev,
                       void *stream);

/* Host plan of a ping-pong step at decode-checkpoint interval `interval`:
 *   pos           host int64 [B]: tokens each request has consumed (its state's position)
 *   active_pages  host int32 [B * P]: the requests' active objects (private: refcount 1)
 * Requests with pos > 0 and pos % interval == 0 are due: for each of them, in request order,
 * P fresh pages are allocated (lowest free first, refcount 1) as the destination object, and
 * the request index is appended to donated_out (host int32 [B]; count in *n_donated_out).
 * dst_pages_out (host int32 [B * P]) receives the destination lists: the fresh pages for due
 * requests, the active pages for the others.  After the step, each due request's old active
 * pages hold its checkpoint at position pos[r] and its new active object is the destination.
 * All or nothing: KDA_ENOPAGES allocates nothing. */
int kda_decode_pingpong_plan(kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t B,
                             const int64_t *pos, int32_t interval, const int32_t *active_pages,
                             int32_t *dst_pages_out, int32_t *donated_out, int32_t *n_donated_out);

/* Speculative verify ("KIMI K3 경량 복제에서 본 KDA의 AI 인프라 과제", §0x06 6.4: a verify pass
 * carries intermediate-state indices next to the recurrent and conv states): K draft tokens per
 * request are applied one after another and the state after each of them is kept in its own
 * object, so that the state at any accepted length is available without recomputation.
 *
 * kda_verify_plan: allocate the K * B intermediate objects (lowest free first, refcount 1;
 * all or nothing) into inter_pages_out, host int32 [K][B][P] (object of token j of request b
 * at (j * B + b) * P). */
int kda_verify_plan(kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t B, int32_t K,
                    int32_t *inter_pages_out);

/* kda_verify_step: q, k, v, alpha [K][B][H][d] and beta [K][B][H] (device, dtype; draft token
 * major), o [K][B][H][d] written.  src_pages (device int32 [B * P]) holds each request's state
 * before the drafts and is not modified; inter_pages (device int32 [K][B][P]) receives the
 * state after draft token j.  1 <= K <= 64.  For bf16, d = 128, pages of at least 64 KiB and
 * K <= 8 it is one kernel that reads each source record once and keeps the state on chip
 * across the K tokens (traffic: one record read and K record writes per request-head);
 * otherwise it runs as K stream-ordered ping-pong decode steps (kda_decode_step_pp), token j
 * reading the object token j - 1 wrote. */
int kda_verify_step(const kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t B, int32_t K,
                    const void *q, const void *k, const void *v, const void *alpha,
                    const void *beta, const float *conv_w, void *o, void *pool_base,
                    const int32_t *src_pages, const int32_t *inter_pages, int32_t *status_dev,
                    void *stream);

/* kda_verify_accept (host only): accepted[b] in [0, K] draft tokens kept for request b.  The
 * request's new active object is written to active_out (host int32 [B * P]): the source
 * object when accepted[b] == 0, else the object of token accepted[b] - 1.  Every other object
 * among the request's source and intermediates is released (decref).  Call it once the
 * stream has passed the verify step. */
int kda_verify_accept(kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t B, int32_t K,
                      const int32_t *accepted, const int32_t *src_pages, const int32_t *inter_pages,
                      int32_t *active_out);

/* ---------------------------------------------------------------- checkpoints --------- */

/* Workspace bytes for a checkpoint copy of n objects. */
int64_t kda_copy_workspace_bytes(int32_t n, int32_t pages_per_object);

/* Snapshot: allocate n fresh objects (lowest free first, refcount 1), copy each source
 * object (host page lists src_pages [n * P]) into them and return their pages in
 * dst_pages_out [n * P] (host).  KDA_ENOPAGES if the pool cannot hold them. */
int kda_ckpt_write(kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t n,
                   const int32_t *src_pages, int32_t *dst_pages_out, void *pool_base,
                   void *workspace, int64_t ws_bytes, int32_t *status_dev, void *stream);

/* Restore (copy-on-write): pin (incref) the checkpoint pages, then copy each checkpoint
 * object ckpt_pages [n * P] into the private object active_pages [n * P] (both host
 * lists).  The checkpoint is only read.  Release the pin with kda_ckpt_release once the
 * copy has completed on the stream. */
int kda_ckpt_restore(kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t n,
                     const int32_t *ckpt_pages, const int32_t *active_pages, void *pool_base,
                     void *workspace, int64_t ws_bytes, int32_t *status_dev, void *stream);

/* Drop the pin kda_ckpt_restore took: decref the same n * P checkpoint page ids. */
int kda_ckpt_release(kda_pool *pool, int32_t n, int32_t pages_per_object,
                     const int32_t *ckpt_pages);

/* ---------------------------------------------------------------- host offload ------ */

/* Write-back offload and prefetch of checkpoints ("Infrastructure pour le RL à un million de
 * jetons", §La solution : découpler la rétention de la résidence GPU: an idle reusable prefix
 * is written to CPU DRAM only when it leaves the GPU, and prefetched before its next reuse).
 * The host buffer must be pinned and mapped into the device address space (cudaHostAlloc /
 * cudaHostRegister; pinned torch tensors qualify) and 16-byte aligned; object i occupies
 * bytes [i * B, (i + 1) * B) with B = kda_object_bytes(H, d, dtype), in the object's logical
 * byte order (the same bytes as in the pool).
 *
 * Offload: copy the n objects (pages: host int32 [n * P], allocated) to host_dst; the pages
 * stay allocated: the caller decrefs them once the stream has passed the copy (the eviction).
 * workspace: device, at least kda_copy_workspace_bytes(n, P).  A host buffer that is not
 * device-accessible returns KDA_EINVAL. */
int kda_ckpt_offload(kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t n,
                     const int32_t *pages, void *host_dst, int64_t host_bytes, void *pool_base,
                     void *workspace, int64_t ws_bytes, int32_t *status_dev, void *stream);

/* Prefetch: allocate n * P fresh pages (lowest free first, refcount 1; returned in pages_out,
 * host int32 [n * P]) and copy the n host objects into them.  All or nothing. */
int kda_ckpt_prefetch(kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t n,
                      const void *host_src, int64_t host_bytes, int32_t *pages_out, void *pool_base,
                      void *workspace, int64_t ws_bytes, int32_t *status_dev, void *stream);

/* ---------------------------------------------------------------- INT8 checkpoints -- */

/* INT8 compressed checkpoints ("KIMI K3 경량 복제에서 본 KDA의 AI 인프라 과제", §0x05 5.3 and
 * §0x06 6.6: checkpoints waiting in the cache may hold the recurrent state in INT8 while the
 * small conv window keeps its native precision; a hit is dequantised once into a fresh active
 * slot, so the recurrence itself never runs on quantised state).
 * INT8 head record: scale fp32 [d] | codes int8 [d][d] (row i = key channel i, column j =
 * value channel j) | window [3][3d] in dtype, zero-padded to a multiple of 256 bytes
 * (19,200 bytes at d = 128 bf16 against 67,840 for the full record); an INT8 object is the H
 * records in head order, paged like a full object.  scale_i = max_j |S[i][j]| / 127 and
 * code = round-to-nearest-even(S[i][j] / scale_i) clamped to [-127, 127], both divisions IEEE
 * fp32; a zero row has scale 0 and codes 0; dequantisation writes code * scale_i. */
int64_t kda_record_bytes_q8(int32_t d, int32_t dtype);
/* H INT8 records, and the pages of this pool they span; KDA_EINVAL for a bad shape or pool. */
int64_t kda_object_bytes_q8(int32_t H, int32_t d, int32_t dtype);
int32_t kda_object_pages_q8(const kda_pool *pool, int32_t H, int32_t d, int32_t dtype);

/* Snapshot n full objects (src_pages, host int32 [n * P], allocated) into n new INT8
 * checkpoint objects: allocates n * Pq fresh pages (lowest free first, refcount 1; Pq =
 * kda_object_pages_q8), returns them in dst_pages_out (host int32 [n * Pq]) and enqueues the
 * quantisation.  workspace: device, at least kda_copy_workspace_bytes(n, P).  On an error
 * nothing is allocated.  The pool's pages and every object must be below 4 GiB. */
int kda_ckpt_write_q8(kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t n,
                      const int32_t *src_pages, int32_t *dst_pages_out, void *pool_base,
                      void *workspace, int64_t ws_bytes, int32_t *status_dev, void *stream);

/* Restore n INT8 checkpoints (ckpt_pages, host int32 [n * Pq], allocated) into n private full
 * objects (active_pages, host int32 [n * P], refcount 1, disjoint from the checkpoints): the
 * checkpoint pages are pinned (incref) for the conversion and released by
 * kda_ckpt_release(pool, n, Pq, ckpt_pages) once the stream has passed it. */
int kda_ckpt_restore_q8(kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t n,
                        const int32_t *ckpt_pages, const int32_t *active_pages, void *pool_base,
                        void *workspace, int64_t ws_bytes, int32_t *status_dev, void *stream);

/* ---------------------------------------------------------------- key/value cache ----- */

/* The other layers of a hybrid model attend over cached keys and values.  Their cache lives in
 * the same pool of pages as the recurrent states ("Cache de préfixe hybride KDA–MLA", §La mise en
 * page unifiée: one page size, one allocator for every kind), one page table row a sequence:
 * table[s][b] is the page of the sequence's tokens [b * page_tokens, (b + 1) * page_tokens).
 *
 * A page is one block of page_tokens tokens (a multiple of 16, 16 to 128) of all Hkv heads of one
 * layer: Hkv records in head order, each
 *     K tile | V tile | KDA_KV_I8 only: float K scale, float V scale, 8 bytes that no call writes
 * A tile is page_tokens rows of d elements (bf16, or int8 codes), cut into lines of 128 bytes (64
 * where a row has only 64): line block c holds bytes [128 c, 128 c + 128) of every row, row after
 * row, and the 16-byte unit u of token slot t's line lies at place u ^ (t % 8) (64-byte lines:
 * u ^ ((t / 2) % 4)).  A record is thus shared-memory ready: copied as it is, eight tokens' units
 * of one column fall into different banks.
 *
 * Formats: KDA_KV_BF16, values rounded to bf16; KDA_KV_I8, value = code * scale with one scale
 * for the keys and one for the values of each (block, head).  Appending to a block sets
 * scale = max(max |x| over the new tokens / 127, the block's scale if it holds older tokens) and
 * code = round-to-nearest-even(x / scale), both divisions IEEE fp32; when the scale grows, older
 * codes c become rne(c * old scale / scale).  A block with an infinity or a NaN in it reads as NaN
 * (that head's K or V); a scale of 0 reads as zeros.  Scales are not negative.
 *
 * Batches: cu_q (device int32 [nseq + 1], ascending) cuts the call's T_tot packed token rows into
 * sequences; kv_len (device int32 [nseq]) is each sequence's length in the cache with the call's
 * own tokens in it, so that its n new tokens stand at positions kv_len - n .. kv_len - 1.  The
 * same arrays serve kda_kv_append and kda_attn_paged.  max_q bounds the new tokens of any one
 * sequence (host).  Nothing is read back to the host, so the calls can be captured in a graph and
 * replayed on new lengths.  Metadata out of range (n > max_q, kv_len beyond the table, cu_q beyond
 * T_tot) sets KDA_DEV_BAD_META and that sequence is skipped; a page id outside the pool sets
 * KDA_DEV_BAD_PAGE and that block is skipped.  Output rows of a skipped sequence, and those that no
 * sequence owns, stay as they were.
 *
 * Token tensors q, k, v are [T_tot][H][d] in dtype with token rows `stride` elements apart (at
 * least H * d: the parts of one fused projection will do); pointers are 16-byte aligned and
 * strides multiples of 16 bytes.  d is 64 or 128.  max_pages * page_tokens is at most 2^30. */
#define KDA_KV_BF16 0
#define KDA_KV_I8 1

/* Bytes of one page of such a cache, rounded up to a valid pool page size (a multiple of 256); a
 * pool with larger pages holds it too.  KDA_EINVAL for a bad shape. */
int64_t kda_kv_page_bytes(int32_t Hkv, int32_t d, int32_t fmt, int32_t page_tokens);

/* Append the call's keys and values to their blocks, keys rotated by position on the way, and
 * write the rotated queries.
 *   q, q_out      queries [T_tot][Hq][d] and their rotated copy (contiguous, dtype; may be q
 *                 itself when q is contiguous).  Both NULL: keys and values only
 *   k, v          new keys and values [T_tot][Hkv][d]
 *   cos_sin       device fp32 [max_pos][rot_dim]: row p holds the rot_dim / 2 cosines, then the
 *                 sines, of position p.  NULL (rot_dim 0): no rotation.  A sequence that
 *                 reaches past max_pos sets KDA_DEV_BAD_META and is skipped, its queries too
 *   rot_dim       leading elements of a head that rotate: a multiple of 16, at most d
 *   interleaved   0: element i turns with i + rot_dim / 2; else 2 i with 2 i + 1
 * The pages written must be private to their sequence (a shared prefix ends on a block's end, or
 * its last block is copied first).  A call whose kv_len < n for a sequence skips it
 * (KDA_DEV_BAD_META).  One launch. */
int kda_kv_append(const kda_pool *pool, int32_t Hq, int32_t Hkv, int32_t d, int32_t dtype, int32_t fmt,
                  int32_t page_tokens, int32_t nseq, int64_t T_tot, int32_t max_q, const int32_t *cu_q,
                  const int32_t *kv_len, const int32_t *page_table, int32_t max_pages, const void *q,
                  int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                  const float *cos_sin, int32_t max_pos, int32_t rot_dim, int32_t interleaved, void *q_out,
                  void *pool_base, int32_t *status_dev, void *stream);

/* Read cached ranges back as values: row cu_out[s] + i of k_out and v_out ([T_out][Hkv][d], dtype)
 * is sequence s's token begin[s] + i (cu_out device int32 [nseq + 1], begin device int32 [nseq]).
 * For handing a prefix on, or checking what a cache stands for. */
int kda_kv_gather(const kda_pool *pool, int32_t Hkv, int32_t d, int32_t dtype, int32_t fmt, int32_t page_tokens,
                  int32_t nseq, int64_t T_out, const int32_t *cu_out, const int32_t *begin,
                  const int32_t *page_table, int32_t max_pages, void *k_out, void *v_out, const void *pool_base,
                  int32_t *status_dev, void *stream);

/* Workspace bytes of kda_attn_paged for such a batch (partial results of sequences that several
 * CTAs share; nothing in it outlives a call).  KDA_EINVAL for a bad shape. */
int64_t kda_attn_workspace_bytes(int32_t Hq, int32_t Hkv, int32_t d, int32_t dtype, int32_t nseq, int64_t T_tot,
                                 int32_t max_q);

/* Attention of the call's queries over the cache: query head h reads key/value head
 * h / (Hq / Hkv), and a query at position p sees the cached tokens j <= p with
 *     window == 0  or  j > p - window  or  j < sinks
 * (causal; with a window, the last `window` tokens and the first `sinks` ones).
 *   q             [T_tot][Hq][d] as rotated by kda_kv_append, its tokens already in the cache
 *   scale         factor of q . k, commonly 1 / sqrt(d); finite
 *   o             [T_tot][Hq][d] contiguous, dtype: softmax(scale q k) v
 *   lse           device fp32 [T_tot][Hq] or NULL: the log of the sum of the exponentials
 *   workspace     device, 16-byte aligned, kda_attn_workspace_bytes(); one call at a time uses it
 * A query that sees nothing (kv_len < n puts it before the first token) gets o = 0 and
 * lse = -infinity.  What a query does not see never changes its result, a NaN or an infinity
 * included; pages that no query of the call sees are not read, and their table entries may hold
 * anything.  Sums, maxima and accumulators are fp32; KDA_F32 calls keep fp32 accuracy throughout.
 * KDA_BF16 calls round each probability before its product with the value: over KDA_KV_BF16 to bf16,
 * or to 16 bits where max_q * Hq / Hkv is at most 16 (a caller who wants more passes KDA_F32 tokens);
 * over KDA_KV_I8, times the block's value scale, to fp16 with a range that follows the query's own
 * tokens: a product of probability and value scale 2^19 times below the largest that the query sees
 * loses bits, one 2^30 below may add nothing to o.  Results do not depend on timing: the same call
 * gives the same bits. */
int kda_attn_paged(const kda_pool *pool, int32_t Hq, int32_t Hkv, int32_t d, int32_t dtype, int32_t fmt,
                   int32_t page_tokens, int32_t nseq, int64_t T_tot, int32_t max_q, const int32_t *cu_q,
                   const int32_t *kv_len, const int32_t *page_table, int32_t max_pages, const void *q,
                   int64_t q_stride, float scale, int32_t window, int32_t sinks, void *o, float *lse,
                   const void *pool_base, void *workspace, int64_t ws_bytes, int32_t *status_dev, void *stream);

/* ---------------------------------------------------------------- trees of drafts ----- */

/* Speculation with a tree of drafts: a draft model offers several continuations that share their
 * beginnings, one pass answers for all of them, and one branch is kept.  A sequence's n <= KDA_TREE_MAX
 * drafts are its n new tokens of the call, in the calls' packed rows (cu_q, kv_len and max_q as for the
 * key/value cache); draft i's parent is an earlier draft, parent[cu_q[s] + i] in [0, i), or -1: it then
 * follows the sequence's last accepted token.  One round of a hybrid model:
 *     kda_tree_plan            masks and positions, once for all layers
 *     kda_kv_append_at, kda_attn_tree       each layer with a cache
 *     kda_verify_tree          each recurrent layer
 *     (the caller compares the model's answers with the drafts and finds the accepted branch)
 *     kda_kv_accept            each layer with a cache
 *     kda_verify_tree_accept   each recurrent layer
 * The accepted branch: path[cu_q[s] + i], i < accepted[s], the drafts kept, from the tree's root on and so
 * ascending; 0 <= accepted[s] <= n.  Trees, branches and lengths stay on the device: a round can be captured
 * in a graph and replayed on others of at most max_q drafts.  A sequence whose metadata is out of range (a
 * parent at or behind its draft or below -1, a path that does not ascend or leaves the tree, a length below n,
 * n > max_q) sets KDA_DEV_BAD_META and is skipped by every call that is given that metadata; what it owns stays
 * as it was.  Parents are given to kda_tree_plan and kda_verify_tree alone: the plan of a tree with such a parent
 * has no positions (below), so that kda_kv_append_at skips its tokens too, and kda_attn_tree's answers for it
 * count for nothing.  Neither kda_kv_accept nor kda_verify_tree_accept sees parents: 0 accepted drafts leave such
 * a sequence's cache and state as they were.  max_q is at most KDA_TREE_MAX (KDA_EINVAL). */
#define KDA_TREE_MAX 64

/* Masks and positions of the drafts: bit j of mask[t] (device uint64 [T_tot]) says that the draft of packed
 * row t is draft j or descends from it; pos[t] (device int32 [T_tot]) is kv_len - n + its depth, the tree's
 * roots having depth 0.  A tree with a parent that is none gets pos[t] = -1 and mask[t] = 0 in its rows, but for
 * those whose pos is negative already, which are left as they are.  pos is a token's coordinate where coordinates
 * are places in the cache.  Behind pictures, or on several axes, the caller forms kda_kv_append_at's [T_tot][axes]
 * from the depth, pos[t] - (kv_len - n), and leaves a negative pos negative.  One launch. */
int kda_tree_plan(int32_t nseq, int64_t T_tot, int32_t max_q, const int32_t *cu_q, const int32_t *kv_len,
                  const int32_t *parent, uint64_t *mask, int32_t *pos, int32_t *status_dev, void *stream);

/* kda_kv_append for tokens whose position is not their place in the cache: the drafts of a tree, or tokens
 * of pictures and video with coordinates on several axes (time, height, width).  Also for more than
 * KDA_TREE_MAX new tokens.
 *   pos           device int32 [T_tot][axes]: each token's coordinates, in [0, max_pos)
 *   axes          1 to KDA_MAX_AXES
 *   sections      host int32 [axes]: of a head's rot_dim / 2 angles the first sections[0] go by a token's
 *                 first coordinate, the next sections[1] by its second, and so on; positive multiples of 8
 *                 whose sum is rot_dim / 2
 *   cos_sin       as there, not NULL; row p serves coordinate p of any axis
 * A coordinate outside [0, max_pos) sets KDA_DEV_BAD_META; the block that would hold the token is then
 * skipped, keys and values, and that token's query.  Everything else is as kda_kv_append has it. */
#define KDA_MAX_AXES 4
int kda_kv_append_at(const kda_pool *pool, int32_t Hq, int32_t Hkv, int32_t d, int32_t dtype, int32_t fmt,
                     int32_t page_tokens, int32_t nseq, int64_t T_tot, int32_t max_q, const int32_t *cu_q,
                     const int32_t *kv_len, const int32_t *page_table, int32_t max_pages, const void *q,
                     int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                     const float *cos_sin, int32_t max_pos, int32_t rot_dim, int32_t interleaved, const int32_t *pos,
                     int32_t axes, const int32_t *sections, void *q_out, void *pool_base, int32_t *status_dev,
                     void *stream);

/* Attention of a tree's drafts over the cache, their own keys and values in it: kda_attn_paged with another
 * rule of who sees what.  With base = kv_len - n, draft i sees
 *     the cached tokens j < base with window == 0 or j > pos[i] - window or j < sinks
 *     the drafts j whose bit of mask[i] is set, whatever the window
 *   mask          device uint64 [T_tot], as kda_tree_plan writes it; any other will do (bits from n on count
 *                 for nothing, a draft need not see itself)
 *   pos           device int32 [T_tot]; read with a window only (NULL without one).  A position before base
 *                 or behind the last draft's place counts as that
 * Sequences with kv_len < n are skipped (KDA_DEV_BAD_META); a draft that sees nothing gets o = 0 and
 * lse = -infinity; one that sees an infinite value gets an infinity or NaN in that column, and one that
 * sees an infinite key may get NaN.  KDA_BF16 calls over KDA_KV_BF16 keep 16 bits of each probability.
 * Workspace, types, other roundings, unseen infinities and NaN, and the same bits for the same call: as
 * kda_attn_paged has them. */
int64_t kda_attn_tree_workspace_bytes(int32_t Hq, int32_t Hkv, int32_t d, int32_t dtype, int32_t nseq, int64_t T_tot,
                                      int32_t max_q);
int kda_attn_tree(const kda_pool *pool, int32_t Hq, int32_t Hkv, int32_t d, int32_t dtype, int32_t fmt,
                  int32_t page_tokens, int32_t nseq, int64_t T_tot, int32_t max_q, const int32_t *cu_q,
                  const int32_t *kv_len, const int32_t *page_table, int32_t max_pages, const uint64_t *mask,
                  const int32_t *pos, const void *q, int64_t q_stride, float scale, int32_t window, int32_t sinks,
                  void *o, float *lse, const void *pool_base, void *workspace, int64_t ws_bytes, int32_t *status_dev,
                  void *stream);

/* Keep the accepted branch in the cache: the keys and values of token base + path[i] move to place base + i
 * (base = kv_len - n, i < accepted), and kv_len_out (device int32 [nseq], apart from kv_len and accepted) receives
 * base + accepted.  What stands behind it afterwards is left over and counts for nothing.  Rows of the 16-bit cache
 * move as they are.  KDA_KV_I8: a block that takes in tokens of another block sets scale = max(max |x| / 127 over
 * those, the block's scale if a token stays in it: an older one, or an accepted one that it held already) and
 * codes as kda_kv_append does, x = code * scale in fp32; without such tokens its scale and codes stay.  The pages
 * that hold the drafts must be private to their sequence.  A page id outside the pool among the blocks that rows
 * move from or to (and those between) sets KDA_DEV_BAD_PAGE, and the sequence is skipped.  One launch. */
int kda_kv_accept(const kda_pool *pool, int32_t Hkv, int32_t d, int32_t fmt, int32_t page_tokens, int32_t nseq,
                  int64_t T_tot, int32_t max_q, const int32_t *cu_q, const int32_t *kv_len, const int32_t *page_table,
                  int32_t max_pages, const int32_t *path, const int32_t *accepted, int32_t *kv_len_out,
                  void *pool_base, int32_t *status_dev, void *stream);

/* Verify a tree against recurrent states: o[t] is what kda_decode_step would answer for draft t after the
 * drafts of its branch, starting from the request's state; convolution windows follow the branches too.  The
 * state is read once and nothing but o is written: the state after draft t is
 *     S_t = Diag(A_t) S_0 + sum over the branch of (r(t, i) k_i) u_i^T,
 *     u_t = beta_t (v_t - S_0^T (A_t k_t) - sum over the branch before t of <k_t, r(t, i) k_i> u_i)
 * with A_t the product of alpha over the branch and r(t, i) over the part behind i, and o_t = S_t^T q_t needs the
 * products with S_0, the inner products and the u alone.  Any alpha in [0, 1] will do, 0 included.
 *   q, k, v, alpha   device [T_tot][H][d] dtype, contiguous, 16-byte aligned; beta [T_tot][H]
 *   cu_q             device int32 [B + 1]; a request may have no drafts
 *   parent           device int32 [T_tot]
 *   state_pages      device int32 [B * P], P = kda_object_pages(): read only
 * Sums and the products' operands are fp32 for KDA_F32.  KDA_BF16: the products with S_0 take either operand in
 * two bf16 terms, and are off by 3 x 2^-16 of the absolute sum of their terms: below o's own rounding unless o
 * cancels to a hundredth of those terms.  Nothing of that enters a state (kda_verify_tree_accept).  A page id
 * outside the pool sets KDA_DEV_BAD_PAGE and the request is skipped.  One launch. */
int kda_verify_tree(const kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t B, int64_t T_tot, int32_t max_q,
                    const int32_t *cu_q, const int32_t *parent, const void *q, const void *k, const void *v,
                    const void *alpha, const void *beta, const float *conv_w, void *o, const void *pool_base,
                    const int32_t *state_pages, int32_t *status_dev, void *stream);

/* Advance each request's state and convolution window over its accepted branch, in place (decode steps without the
 * answers, the state read and written once; fp32 throughout).  The arguments are those of kda_verify_tree, the same
 * tokens among them; the objects of state_pages are private, each in the call once.  A request that accepts nothing is
 * left as it is.  One launch. */
int kda_verify_tree_accept(const kda_pool *pool, int32_t H, int32_t d, int32_t dtype, int32_t B, int64_t T_tot,
                           int32_t max_q, const int32_t *cu_q, const int32_t *path, const int32_t *accepted,
                           const void *q, const void *k, const void *v, const void *alpha, const void *beta,
                           const float *conv_w, void *pool_base, const int32_t *state_pages, int32_t *status_dev,
                           void *stream);

/* ---------------------------------------------------------------- status -------------- */

/* Wait for `stream`, read and clear *status_dev.  Returns KDA_OK, KDA_EDEVICE (bits in
 * *bits_out if not NULL) or KDA_ECUDA. */
int kda_sync_status(int32_t *status_dev, void *stream, int32_t *bits_out);

/* Static description of a status code. */
const char *kda_status_string(int code);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
