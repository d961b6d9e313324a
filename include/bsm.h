/*
 * bsm.h -- block-sparse masked attention (Splash-style) on GB300: the
 * forward and its backward.
 *
 * C ABI of libbsm.so.  All compute runs in hand-written CUDA kernels for
 * sm_103a; there is no CPU path.  The library allocates no device memory:
 * the caller owns every buffer (inputs, outputs and the mask-info buffer).
 * Pointers marked "device" must be device (or managed) memory of the current
 * CUDA device; `stream` is a cudaStream_t passed as void* (NULL = the legacy
 * default stream).  Work is enqueued asynchronously; argument errors are
 * returned synchronously, before anything is enqueued, with a message in
 * bsm_last_error().  No function falls back to another algorithm silently.
 *
 * Sources (page title, section):
 *   [HSTU]   RecML "recml/core/ops/hstu_ops.py" -- pointwise splash attention:
 *            _next_nonzero (block classes), _apply_mask (element mask),
 *            _pointwise_splash_attention_fwd_kernel_impl (pointwise scores),
 *            pointwise_splash_attention (API, defaults, argument checks).
 *   [NOTES]  "JAX 到 VLIW, Pallas / Splash Attention 复习笔记" -- section 12
 *            (naive attention), 15 (online softmax m/l/o), 18-19 (grid
 *            h, i, j), 21 (sparse K/V indirection via data_next).
 *   [KERNELS] "Attention Kernels -- Splash, Flash, SDPA on TPU" -- section
 *            "Splash Attention via call_jax" (make_splash_mha(mask) then
 *            kernel(q, k, v)).
 */
#ifndef BSM_H_
#define BSM_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum bsm_status {
  BSM_OK = 0,
  BSM_ERR_INVALID_ARG = -1,    /* bad shape, pointer, stride or size */
  BSM_ERR_UNSUPPORTED = -2,    /* valid but not built (e.g. head_dim 96) */
  BSM_ERR_CUDA = -3,           /* a CUDA runtime/driver call failed */
  BSM_ERR_DEVICE_TIMEOUT = -4  /* a kernel gave up waiting (see below) */
} bsm_status;

/* Score path.  SOFTMAX: out = softmax(scale * q k^T restricted to the
 * visible keys) v, plus the per-row logsumexp ([NOTES] section 15).
 * POINTWISE: out = sum over visible keys of x*sigmoid(x)/Sq * v with
 * x = scale * q.k, no normalisation ([HSTU] fwd kernel impl). */
typedef enum bsm_score {
  BSM_SCORE_SOFTMAX = 0,
  BSM_SCORE_POINTWISE = 1
} bsm_score;

/* Mask predicates, AND-ed; flags == 0 is the full mask ([HSTU]
 * pointwise_splash_attention: MaskType.CAUSAL / FULL, segment ids).
 *   CAUSAL : key k visible from query q iff k <= q
 *   LOCAL  : iff q - k < window            (window >= 1)
 *   BAND   : with LOCAL only, the window also bounds the keys after q:
 *            iff k - q < window, so LOCAL|BAND is the symmetric sliding
 *            window |q - k| < window (hstu_ops LocalMask((w, w)) with
 *            MaskType.FULL)
 *   SEGMENT: iff q_segment_ids[b][q] == kv_segment_ids[b][k]
 *   DENSE  : iff bit k % 32 of word dense_bits[q * dense_row_words + k / 32]
 *            is set: an arbitrary mask ([HSTU]'s NumpyMask), bit-packed,
 *            one row of dense_row_words >= ceil(Skv / 32) uint32 words per
 *            query row, shared by every batch row and head; device memory
 *            owned by the caller, read by bsm_build_mask_info and again by
 *            bsm_splash_fwd (keep it alive while the mask info is used)
 * Elements past Sq or Skv (a ragged last block) are never visible. */
#define BSM_MASK_CAUSAL 1u
#define BSM_MASK_LOCAL 2u
#define BSM_MASK_SEGMENT 4u
#define BSM_MASK_BAND 8u
#define BSM_MASK_DENSE 16u

typedef struct bsm_mask_spec {
  uint32_t flags;
  int32_t window;  /* used with BSM_MASK_LOCAL only */
  const uint32_t* dense_bits; /* BSM_MASK_DENSE only, else NULL */
  int64_t dense_row_words;    /* BSM_MASK_DENSE only */
} bsm_mask_spec;

/* Mask-info tables ([HSTU] _next_nonzero; [NOTES] section 21), filled by
 * bsm_build_mask_info.  All arrays are device memory inside the caller's
 * buffer.  num_tables is B when SEGMENT is set (one table per batch row),
 * else 1 (shared by all batch rows and heads).  Row r = t*nq + i.
 *   block_mask[t][i][j] int8: 0 empty (never loaded), 1 partial (element
 *                       mask applied), 2 full (no mask)
 *   data_next[t][i][j]  int32: smallest nonzero j' >= j of row i; if none,
 *                       the largest nonzero j' < j; 0 for an empty row
 *   row_ptr[r]          int32, num_tables*nq + 1 entries, CSR offsets
 *   kv_idx[row_ptr[r]..row_ptr[r+1])  nonzero j of row r, ascending
 *   kv_cls[...]         their classes (1 or 2)
 *   seg_range[b][q][2]  int32 (SEGMENT only): first and last key index whose
 *                       segment id equals q's, valid when every kv segment-id
 *                       row is non-decreasing (packed sequences); first > last
 *                       when no key has q's id
 *   seg_flags[0]        int32 (SEGMENT only): bit 0 set if some kv segment-id
 *                       row is not non-decreasing (then seg_range is unused and
 *                       segments are compared element by element); entries
 *                       1..num_tables are the builder's per-table scratch
 *   super_order[k]      int32, num_tables*num_super entries: the pairs
 *                       (table t, super-tile s) as t*num_super + s, ordered by
 *                       decreasing work (query rows times nonzero blocks
 *                       they see, quantised to 19 bits of the largest),
 *                       ties by decreasing index.  A super-tile is 256 query
 *                       rows, the forward's work unit; bsm_splash_fwd hands
 *                       its units out in this order (longest first).  NULL
 *                       when num_tables*num_super > 8192 (the forward then
 *                       takes the last super-tiles first).  Scheduling only:
 *                       no result depends on it.  No counterpart on the
 *                       pages, whose grid walks the query blocks in order.
 * kv_idx/kv_cls have capacity num_tables*nq*nk. */
typedef struct bsm_mask_info {
  uint32_t flags;
  int32_t window;
  int32_t num_tables;
  int32_t Sq, Skv;
  int32_t block_q, block_kv;
  int32_t nq, nk; /* ceil(Sq / block_q), ceil(Skv / block_kv) */
  int8_t* block_mask;
  int32_t* data_next;
  int32_t* row_ptr;
  int32_t* kv_idx;
  int8_t* kv_cls;
  int32_t* seg_range;
  int32_t* seg_flags;
  int32_t num_super; /* ceil(Sq / 256) */
  int32_t* super_order;
  const uint32_t* dense_bits; /* the spec's, for the forward (DENSE only) */
  int64_t dense_row_words;
} bsm_mask_info;

/* Bytes the caller must allocate for bsm_build_mask_info (0 on bad
 * arguments).  B is the batch size (only used with BSM_MASK_SEGMENT). */
size_t bsm_mask_info_bytes(const bsm_mask_spec* spec, int32_t B, int32_t Sq,
                           int32_t Skv, int32_t block_q, int32_t block_kv);

/* Build the mask-info tables on the device ([HSTU] process_mask call in
 * pointwise_splash_attention; class encoding of _next_nonzero; next-block
 * table of [NOTES] section 21).  Exact: block classes come from the same
 * per-element predicate the forward kernel applies.
 *   q_segment_ids  device int32 [B][Sq], contiguous; required iff SEGMENT
 *   kv_segment_ids device int32 [B][Skv]; required iff SEGMENT
 *   block_q, block_kv in {16, 32, 64, 128, 256, 512}
 *   buffer         device, >= bsm_mask_info_bytes(...) bytes, 256-aligned
 *   info           host struct, filled with the shape and pointers into
 *                  `buffer` (valid once the enqueued work has run)
 * Returns BSM_ERR_INVALID_ARG for non-positive/inconsistent sizes, a
 * missing or superfluous segment-id array ([HSTU]: both or neither),
 * window < 1 with LOCAL, or a buffer that is too small or misaligned. */
bsm_status bsm_build_mask_info(const bsm_mask_spec* spec,
                               const int32_t* q_segment_ids,
                               const int32_t* kv_segment_ids, int32_t B,
                               int32_t Sq, int32_t Skv, int32_t block_q,
                               int32_t block_kv, void* buffer,
                               size_t buffer_bytes, bsm_mask_info* info,
                               void* stream);

/* Bit-pack a boolean mask into the BSM_MASK_DENSE layout (the role of
 * [HSTU]'s dense mask array, stored as bits): bit k % 32 of word
 * words[q * row_words + k / 32] is (mask[q * mask_row_stride + k] != 0) for
 * k < Skv; the rest of each row's words are zero.
 *   mask             device uint8 [Sq][mask_row_stride] (torch.bool bytes)
 *   words            device uint32 [Sq][row_words], row_words >=
 *                    ceil(Skv / 32); pass it as bsm_mask_spec.dense_bits
 * One kernel launch on `stream`.  Returns BSM_ERR_INVALID_ARG for negative
 * sizes, row_words or mask_row_stride too small, or a NULL pointer with a
 * nonempty mask. */
bsm_status bsm_pack_dense_mask(const uint8_t* mask, int64_t mask_row_stride,
                               int32_t Sq, int32_t Skv, uint32_t* words,
                               int32_t row_words, void* stream);

/* Block-sparse masked attention forward ([NOTES] sections 15, 18, 21;
 * [HSTU] _pointwise_splash_attention_fwd_kernel_impl).  For each (batch,
 * head, 128-row query tile) the kernel walks only the KV tiles the mask-info
 * marks nonzero; full tiles skip the element mask.
 *   q           device bf16, logical [B][H][Sq][D], head_dim contiguous
 *   k, v        device bf16, logical [B][H_kv][Skv][D], head_dim contiguous
 *   *_strides   element strides of the batch, head and sequence dims
 *               (so [B,H,S,D] and [B,S,H,D] storage both work); every
 *               stride and pointer must be a multiple of 16 bytes
 *   H % H_kv == 0: query head h reads K/V head h / (H / H_kv)
 *   D           64 or 128 (else BSM_ERR_UNSUPPORTED)
 *   info        from bsm_build_mask_info with the same Sq, Skv, mask and
 *               (with SEGMENT) the same B; block_q and block_kv must divide
 *               or be multiples of 128
 *   q/kv_segment_ids  as for bsm_build_mask_info (required iff SEGMENT)
 *   scale       logits are scale * q.k ([HSTU] default 1/sqrt(D))
 *   score       bsm_score
 *   out         device bf16 [B][H][Sq][D] at o_strides, rounded to nearest
 *   lse         SOFTMAX: device f32 [B][H][Sq] contiguous, natural-log
 *               logsumexp of the visible scaled logits (-inf for a row that
 *               sees no key), or NULL; POINTWISE: must be NULL
 *   workspace   device, >= bsm_splash_fwd_workspace_bytes(), 16-aligned:
 *               the persistent CTAs take work units (batch, head, 256 query
 *               rows; heaviest rows first) from a counter kept there and
 *               write the units' KV-tile lists there
 * Rows that see no key get out = 0.  Returns BSM_ERR_UNSUPPORTED for
 * Sq > 262144 or Skv > 262144. */
bsm_status bsm_splash_fwd(const void* q, const void* k, const void* v,
                          const int64_t q_strides[3],
                          const int64_t k_strides[3],
                          const int64_t v_strides[3],
                          const int64_t o_strides[3], int32_t B, int32_t H,
                          int32_t H_kv, int32_t Sq, int32_t Skv, int32_t D,
                          const bsm_mask_info* info,
                          const int32_t* q_segment_ids,
                          const int32_t* kv_segment_ids, float scale,
                          int32_t score, void* out, float* lse,
                          void* workspace, size_t workspace_bytes,
                          void* stream);

/* Modified softmax scores: with x = scale * q.k, the logit of a visible key is
 *     z = softcap * tanh(x / softcap)   (softcap > 0; else z = x)
 *     z -= alibi_slopes[h] * |q - k|    (alibi_slopes != NULL)
 * with q, k the row's and the key's positions and h the query head.  The mask
 * is applied after both.  These scores have no counterpart on the pages.
 *   softcap       0 (no cap) or positive, with scale / softcap finite in f32
 *   alibi_slopes  device f32 [H], contiguous, at most 2^64 in magnitude, of
 *                 any sign, or NULL; read by the kernels (not checked).
 *                 Constants: the backward gives them no gradient
 * Scores and bias are f32: a logit is off by at most about 6e-7 of its value
 * (|x| <= softcap / 2, where tanh is a polynomial) or 2^-22 of softcap (beyond,
 * and everywhere for softcap above 2^18 scale, where it is 1 - 2 / (1 + e^(2 x
 * / softcap))), and by 2^-22 of slope times the distance, or times 64 if that
 * is more.  As without a modification, a key that a row does not see weighs 0,
 * and 0 times an infinity or NaN in V (in the backward: in any operand) of a
 * key tile that the row's query tile visits is NaN.  A row that sees a NaN
 * score gets NaN for its output and logsumexp.  With a cap a row's weights are
 * f32 numbers up to 2^90 until they are normalised, and their products with V
 * are summed in f32: |V| up to 2^20 (about 10^6) is safe at every length. */
typedef struct bsm_score_mod {
  float softcap;
  const float* alibi_slopes;
} bsm_score_mod;

/* bsm_splash_fwd with modified softmax scores: the same arguments, checks and
 * kernels, plus `mod` (NULL, or with softcap 0 and no slopes: exactly
 * bsm_splash_fwd).  A NaN or negative softcap, an overflowing scale / softcap,
 * or a modification on the pointwise score path returns
 * BSM_ERR_INVALID_ARG. */
bsm_status bsm_splash_fwd_mod(const void* q, const void* k, const void* v,
                              const int64_t q_strides[3],
                              const int64_t k_strides[3],
                              const int64_t v_strides[3],
                              const int64_t o_strides[3], int32_t B, int32_t H,
                              int32_t H_kv, int32_t Sq, int32_t Skv, int32_t D,
                              const bsm_mask_info* info,
                              const int32_t* q_segment_ids,
                              const int32_t* kv_segment_ids, float scale,
                              int32_t score, const bsm_score_mod* mod,
                              void* out, float* lse, void* workspace,
                              size_t workspace_bytes, void* stream);

/* Bytes of the forward's device workspace (about 6 MiB): the work-unit
 * counter and each CTA's lists of the KV tiles of its next units.  The
 * counter is zeroed on `stream` before each launch; the launch overwrites
 * the rest.  Two forward calls that may run at the same time need separate
 * workspaces. */
size_t bsm_splash_fwd_workspace_bytes(void);

/* Bytes of the device buffer bsm_splash_fwd_host needs (0 on bad
 * arguments): device copies of q, k, v, out, lse (SOFTMAX) and the segment
 * ids (SEGMENT), the mask info and the forward's workspace. */
size_t bsm_splash_fwd_host_bytes(const bsm_mask_spec* spec, int32_t B,
                                 int32_t H, int32_t H_kv, int32_t Sq,
                                 int32_t Skv, int32_t D, int32_t block_q,
                                 int32_t block_kv, int32_t score);

/* The forward on host buffers, end to end (this entry point has no
 * counterpart in the pages; it is a property of this library): copies the
 * inputs to the device, builds the mask info, runs bsm_splash_fwd and
 * copies out (and lse) back, pipelined over n_chunks ranges of K/V heads
 * (their query heads follow): the host-to-device copies of one range, the
 * forward of the previous one and the device-to-host copies of the one
 * before that run at the same time, on two copy streams the library keeps
 * per device (made on the first call in a CUDA context) and the caller's
 * stream.  Each range moves as one strided copy per tensor.
 *   spec, block_q, block_kv, scale, score  as for bsm_build_mask_info and
 *               bsm_splash_fwd (spec->dense_bits, if any, is device memory)
 *   q           host bf16 [B][H][Sq][D], contiguous
 *   k, v        host bf16 [B][H_kv][Skv][D], contiguous
 *   q/kv_segment_ids  host int32 [B][Sq] / [B][Skv]; both iff SEGMENT
 *   out         host bf16 [B][H][Sq][D]; lse host f32 [B][H][Sq] or NULL
 *               (NULL for POINTWISE)
 *   device_buffer  device, >= bsm_splash_fwd_host_bytes(...) bytes,
 *               256-byte aligned, owned by the caller; two calls that may
 *               run at the same time need separate buffers
 *   n_chunks    1..16 head ranges, capped at H_kv; <= 0 picks 4
 * Host memory should be page-locked (cudaHostAlloc / cudaHostRegister):
 * copies from or to pageable memory are correct but do not overlap.
 * Everything is enqueued: the call returns once the work is issued and
 * `stream` waits for the last copy, so out and lse are ready after the
 * stream is synchronised.  Argument errors as for bsm_splash_fwd, found
 * before anything is enqueued; a failure part-way returns its status with
 * the work enqueued until then left to run, `stream` still waiting for it
 * (so the device buffer is free once `stream` is synchronised). */
bsm_status bsm_splash_fwd_host(const bsm_mask_spec* spec, const void* q,
                               const void* k, const void* v,
                               const int32_t* q_segment_ids,
                               const int32_t* kv_segment_ids, int32_t B,
                               int32_t H, int32_t H_kv, int32_t Sq,
                               int32_t Skv, int32_t D, int32_t block_q,
                               int32_t block_kv, float scale, int32_t score,
                               void* out, float* lse, void* device_buffer,
                               size_t device_bytes, int32_t n_chunks,
                               void* stream);

/* bsm_splash_fwd for callers that cannot allocate device memory (this entry
 * point has no counterpart in the pages; it is a property of this library).
 * Plugins handed finished buffers by a host framework, serving engines that
 * reserve all free HBM up front, and loops that cannot afford cudaMalloc's
 * implicit synchronisation can call it: it takes the same arguments as
 * bsm_splash_fwd minus the workspace and allocates nothing (no cudaMalloc,
 * no cudaFree, no allocating library routine).  Its workspace is a 6 MiB
 * (bsm_splash_fwd_workspace_bytes()) array in the library's own device
 * code, held on a device from the moment that code is loaded there until
 * the process exits.
 * Limits: Sq, Skv <= 262144 (else BSM_ERR_UNSUPPORTED), at most 256 CTAs
 * (every supported GPU).
 * Set-up: the first call on a device (per CUDA context) looks up the
 * array's device address (cudaGetSymbolAddress, with that device current)
 * and keeps it for later calls in that context.  Under CUDA's default lazy
 * module loading that first call is also where the library's device code,
 * with the array, is loaded into the context, which takes device memory
 * and may synchronise: make it once, before reserving the device's free
 * memory and before any stream capture.  Later calls take no device memory.
 * Sharing: every call on a device uses the same array.  The work-unit
 * counter in it is zeroed on `stream` before each launch (the rest is
 * overwritten), so a call never depends on what an earlier call left there;
 * calls that overlap on the GPU (e.g. on two streams) race on it and must
 * not be issued. */
bsm_status bsm_splash_fwd_noalloc(const void* q, const void* k, const void* v,
                                  const int64_t q_strides[3],
                                  const int64_t k_strides[3],
                                  const int64_t v_strides[3],
                                  const int64_t o_strides[3], int32_t B,
                                  int32_t H, int32_t H_kv, int32_t Sq,
                                  int32_t Skv, int32_t D,
                                  const bsm_mask_info* info,
                                  const int32_t* q_segment_ids,
                                  const int32_t* kv_segment_ids, float scale,
                                  int32_t score, void* out, float* lse,
                                  void* stream);

/* A bf16 tensor in device memory, logical [B][heads][S][D] with head_dim
 * contiguous; strides are in elements for the batch, head and sequence
 * dims (multiples of 8, positive), data 16-byte aligned.  `data` is read
 * for inputs and written for outputs. */
typedef struct bsm_tensor {
  void* data;
  int64_t strides[3];
} bsm_tensor;

/* Bytes of bsm_splash_bwd's device workspace: B*H*Sq floats (the softmax
 * path's per-row D_q = sum_d dO * out), 0 for the pointwise path. */
size_t bsm_splash_bwd_workspace_bytes(int32_t B, int32_t H, int32_t Sq,
                                      int32_t score);

/* Backward of bsm_splash_fwd: dQ, dK, dV of sum(dout * out) over the same
 * mask ([HSTU] _pointwise_splash_attention_bwd_kernel_impl and its
 * launcher, which accumulate dK/dV over query blocks and dQ over key
 * blocks; for the softmax path the forward of [NOTES] section 15,
 * differentiated: with P = exp(scale q.k - lse) over the visible keys and
 * D_q = sum_d dout[q, d] out[q, d],
 *     dV = P^T dout,  dS = P * (dout V^T - D_q),
 *     dQ = scale dS K,  dK = scale dS^T Q;
 * pointwise: with x = scale q.k and sig = logistic(x),
 *     dV = (x sig / Sq)^T dout,  dS = (dout V^T) sig (1 + x (1 - sig)) / Sq,
 *     dQ = scale dS K,  dK = scale dS^T Q).
 * P and dS are rounded to bf16 for the products (as [HSTU]'s backward
 * casts p to the input type); accumulation is f32.
 *   q, k, v, info, segment ids, scale, score: as given to bsm_splash_fwd
 *   out, lse     the forward's output and logsumexp (SOFTMAX; NULL allowed
 *                for POINTWISE)
 *   dout         device bf16 [B][H][Sq][D]: gradient of the output
 *   dq           device bf16 [B][H][Sq][D], written
 *   dk, dv       device bf16 [B][H_kv][Skv][D], written; with H_kv < H the
 *                gradient of a K/V head sums over its group of query heads
 *   workspace    device, >= bsm_splash_bwd_workspace_bytes(B, H, Sq, score)
 *                bytes, 16-byte aligned (may be NULL when that is 0)
 * Rows and keys that see nothing get zero gradients.  Returns the same
 * argument errors as bsm_splash_fwd. */
bsm_status bsm_splash_bwd(const bsm_tensor* q, const bsm_tensor* k,
                          const bsm_tensor* v, const bsm_tensor* out,
                          const float* lse, const bsm_tensor* dout, int32_t B,
                          int32_t H, int32_t H_kv, int32_t Sq, int32_t Skv,
                          int32_t D, const bsm_mask_info* info,
                          const int32_t* q_segment_ids,
                          const int32_t* kv_segment_ids, float scale,
                          int32_t score, const bsm_tensor* dq,
                          const bsm_tensor* dk, const bsm_tensor* dv,
                          void* workspace, size_t workspace_bytes,
                          void* stream);

/* bsm_splash_bwd with modified softmax scores (see bsm_score_mod): the same
 * arguments and checks plus the `mod` given to the forward.  With
 * t = tanh(x / softcap), P = exp(z - lse) over the visible keys and D_q as
 * above: dV = P^T dout, dS = P * (dout V^T - D_q) * (1 - t^2) (no factor
 * without a cap), dQ = scale dS K, dK = scale dS^T Q.  The slopes get no
 * gradient.
 *   workspace    as for bsm_splash_bwd; with at least
 *                bsm_splash_bwd_mod_workspace_bytes(...) bytes, short inputs
 *                run faster: their dK/dV sums are spread over more CTAs and
 *                added up in f32 (which rounds in another order) */
bsm_status bsm_splash_bwd_mod(const bsm_tensor* q, const bsm_tensor* k,
                              const bsm_tensor* v, const bsm_tensor* out,
                              const float* lse, const bsm_tensor* dout,
                              int32_t B, int32_t H, int32_t H_kv, int32_t Sq,
                              int32_t Skv, int32_t D,
                              const bsm_mask_info* info,
                              const int32_t* q_segment_ids,
                              const int32_t* kv_segment_ids, float scale,
                              int32_t score, const bsm_score_mod* mod,
                              const bsm_tensor* dq, const bsm_tensor* dk,
                              const bsm_tensor* dv, void* workspace,
                              size_t workspace_bytes, void* stream);

/* Bytes with which bsm_splash_bwd_mod spreads the dK/dV sums of short inputs:
 * bsm_splash_bwd_workspace_bytes plus f32 partial sums (none for inputs whose
 * key tiles fill the GPU). */
size_t bsm_splash_bwd_mod_workspace_bytes(int32_t B, int32_t H, int32_t H_kv,
                                          int32_t Sq, int32_t Skv, int32_t D);

/* A paged cache of keys and values in 8-bit floating point (no counterpart on
 * the pages; it serves tokens one by one after the prompt's forward).  A page
 * holds `page_size` consecutive tokens of one sequence for every K/V head:
 *   k, v              device e4m3 [num_pages][H_kv][page_size][D], contiguous,
 *                     16-byte aligned
 *   k_scale, v_scale  device f32 [num_pages][H_kv], contiguous: an element is
 *                     its code times its page's and head's scale; between
 *                     2^-40 and 2^40 wherever a page holds tokens, as
 *                     bsm_kv_append leaves them (not checked; the attention
 *                     joins values whose scales differ by up to 2^80)
 *   page_size         16, 32, 64 or 128; D 64 or 128
 * The memory is the caller's.  A sequence's tokens are found through a page
 * table: entry j of its row is the page of tokens [j page_size, (j + 1)
 * page_size); entries past its last token are never read. */
typedef struct bsm_kv_cache {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int32_t num_pages, H_kv, page_size, D;
} bsm_kv_cache;

/* Append tokens to the cache: sequence b, which holds lens[b] tokens, gets
 * n_new[b] more, k_new[b][:][0 .. n_new[b]) and v_new likewise.  Per page and
 * head, with amax the largest finite magnitude among the new tokens there and
 * e the smallest integer in [-40, 40] with amax <= 448 * 2^e: a page without
 * tokens takes the scale 2^e; one that holds some keeps the larger of its
 * scale and 2^e, and where its scale grows its old codes are rounded again.
 * Codes are element / scale rounded to the nearest e4m3 value (ties to even;
 * a kept scale that is no power of two first makes the quotient an f32);
 * magnitudes above 448 scales (infinities among them) become 448 scales, NaN
 * stays NaN.  Nothing else of the cache is written: not the page's tokens
 * behind the new ones, nor pages that get none.  `lens` is not changed.
 *   page_table  device int32, row b at page_table + b * table_stride, with
 *               max_pages entries; the rows must hold the new tokens' pages
 *   lens, n_new device int32 [B]; n_new NULL = T new tokens each
 *   k_new, v_new  device bf16 [B][H_kv][T][D] (head_dim contiguous, strides
 *               multiples of 8, 16-byte aligned)
 * A page that gets tokens must belong to one sequence only, and stand in its
 * row once (copy a shared last page first).  On the device, lens[b] < 0, n_new[b] outside [0, T],
 * more tokens than max_pages pages hold, or a page outside [0, num_pages)
 * leave that sequence (or page) unwritten and are reported by
 * bsm_device_status as BSM_ERR_INVALID_ARG.  One launch on `stream`. */
bsm_status bsm_kv_append(const bsm_kv_cache* cache, const int32_t* page_table,
                         int64_t table_stride, int32_t max_pages,
                         const int32_t* lens, const int32_t* n_new,
                         const bsm_tensor* k_new, const bsm_tensor* v_new,
                         int32_t B, int32_t T, void* stream);

/* Attention over the cache.  The T queries of sequence b are its last tokens:
 * query t is at position p = lens[b] - T + t and sees the keys j <= p of its
 * sequence, with window > 0 only those with p - j < window.  Scores as in
 * bsm_splash_fwd_mod (softmax; `mod` may be NULL, its bias is slope (p - j)).
 *   q, out      device bf16 [B][H][T][D], strides as above; H a multiple of
 *               the cache's H_kv (query head h reads head h / (H / H_kv))
 *   lens        device int32 [B]: tokens in the cache, the queries' own
 *               among them (append first); 0 is allowed
 *   lse         device f32 [B][H][T], contiguous, or NULL: natural-log
 *               logsumexp of the visible logits
 *   workspace   device, >= bsm_paged_attention_workspace_bytes() bytes,
 *               16-byte aligned; its contents do not matter.  Two calls that
 *               may run at once need separate ones
 * A row that sees no key (lens[b] = 0, or T > lens[b]) gets out = 0 and lse =
 * -inf.  On the device, a length outside [0, max_pages * page_size] is cut to
 * it, tokens of a page outside [0, num_pages) count as masked, and both are
 * reported by bsm_device_status as BSM_ERR_INVALID_ARG. */
bsm_status bsm_paged_attention(const bsm_tensor* q, const bsm_kv_cache* cache,
                               const int32_t* page_table, int64_t table_stride,
                               int32_t max_pages, const int32_t* lens,
                               int32_t B, int32_t H, int32_t T, float scale,
                               int32_t window, const bsm_score_mod* mod,
                               const bsm_tensor* out, float* lse,
                               void* workspace, size_t workspace_bytes,
                               void* stream);

/* Bytes of bsm_paged_attention's device workspace (16 MiB and a little): the
 * parts of rows whose keys are split over several CTAs. */
size_t bsm_paged_attention_workspace_bytes(void);

/* Synchronise `stream` and report whether a kernel of this library gave up
 * on a bounded wait since the last call (then BSM_ERR_DEVICE_TIMEOUT; the
 * affected outputs are undefined, the CUDA context stays usable), or a cache
 * kernel met a length or page out of range (BSM_ERR_INVALID_ARG; with a
 * timeout pending too, the next call reports it).  If
 * `detail` is non-NULL it receives 4 ints: code, block, role, phase; for the
 * cache kernels 2, the sequence, the page slot (-1: a length) and the value. */
bsm_status bsm_device_status(void* stream, int32_t* detail);

/* Failure-detection self test: enqueue one tiny kernel that waits on an
 * mbarrier nothing ever arrives on, with the given limit in nanoseconds
 * (1e3..1e10), so that the bounded wait must run out.  A later
 * bsm_device_status() then returns BSM_ERR_DEVICE_TIMEOUT. */
bsm_status bsm_selftest_wait_timeout(int64_t timeout_ns, void* stream);

/* Tracing (diagnostics).  With a non-NULL device buffer, every following
 * bsm_splash_fwd launch records timestamped events into it: the buffer is
 * split evenly over the launch's CTAs (see bsm_debug_fwd_grid) into
 * 16-byte records; a CTA's records 0-1 hold the event counts of its six
 * recording threads as uint32 {load, mma tile 0, score tile 0, score tile 1,
 * list, mma tile 1, 0, 0}, then come six equal regions, one per thread, of
 * records {uint64 %globaltimer ns, uint32 role<<28 | event<<24 | tile<<20 |
 * entry, uint32 unit}.  NULL (or bytes too small) switches tracing off.  The
 * buffer stays owned by the caller; it must outlive the launches. */
bsm_status bsm_debug_set_trace(void* buffer, size_t bytes);

/* Number of CTAs bsm_splash_fwd launches for these sizes (-1 on error). */
int32_t bsm_debug_fwd_grid(int32_t B, int32_t H, int32_t Sq);

/* Thread-local text of the last error of this thread ("" if none). */
const char* bsm_last_error(void);

/* ABI version (major*10000 + minor*100 + patch): 302 = 0.3.2, adding
 * bsm_splash_fwd_host and bsm_splash_fwd_host_bytes to 0.3.1 (which added
 * bsm_pack_dense_mask to 0.3.0: the backward entry points and bsm_tensor
 * added to 0.2.0's forward, mask spec and mask info).  Entry points added
 * since, with structs of their own, leave the number as it is: callers of
 * 302 are served unchanged. */
int32_t bsm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* BSM_H_ */
