// Internal declarations shared by the host C ABI (bsm_api.cu) and the kernel
// translation units.  Not part of the public interface.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/bsm.h"

namespace bsm {

// Query tile (rows of one tcgen05 accumulator) and KV tile of the forward
// kernel; one work unit is two query tiles (256 rows) of one (batch, head).
constexpr int kTileM = 128;
constexpr int kTileN = 128;
constexpr int kUnitRows = 2 * kTileM;
constexpr int kMaxSeq = 262144;
constexpr int kMaxKvTiles = kMaxSeq / kTileN;  // list capacity per unit
// Forward workspace: 256 bytes of counters, then per CTA two sets (one per
// query-tile pipeline of the packed-sequence kernel; the other kernel uses
// the first) of three unit lists of kMaxKvTiles uint16 entries (up to
// kMaxCtas CTAs).
constexpr int kMaxCtas = 256;
constexpr int kMaxSuperOrder = 8192;  // longest-first table size limit
constexpr int kListBufs = 3;
constexpr size_t kListBytes = static_cast<size_t>(kMaxKvTiles) * 2;
constexpr size_t kFwdWorkspaceBytes =
    256 + static_cast<size_t>(kMaxCtas) * 2 * kListBufs * kListBytes;

struct MaskInfoParams {
  uint32_t flags;
  int32_t window;
  int32_t Sq, Skv, bq, bkv, nq, nk, tables;
  const int32_t* q_seg;   // [tables][Sq] (SEGMENT only)
  const int32_t* kv_seg;  // [tables][Skv]
  int8_t* block_mask;
  int32_t* data_next;
  int32_t* row_ptr;
  int32_t* kv_idx;
  int8_t* kv_cls;
  int32_t* seg_range;  // [tables][Sq][2] (SEGMENT only)
  int32_t* seg_flags;  // [1]: bit 0 = some kv id row is not sorted
  int32_t n_super;        // ceil(Sq / kUnitRows)
  int32_t* super_order;   // [tables * n_super] or null
  const uint32_t* dense;  // DENSE: [Sq][dense_words] bit-packed, else null
  int64_t dense_words;
  // one-launch build: staged row lists [tables * nq][nk] and the ticket word
  int32_t fused;
  uint16_t* staged;
  unsigned long long* ticket;
  unsigned long long epoch;  // 1 .. 2^40 - 1, new for every build
};

// Modified softmax scores: with x = scale * q.k, z = cap * tanh(x / cap) (or
// x), minus slope_h * |q - k|.  All in log2 units, as the kernels use them.
constexpr int kModCap = 1, kModBias = 2;
struct ScoreMod {
  int32_t kind;         // kModCap | kModBias; 0 = unmodified scores
  float cap_e;          // 2 log2(e) scale / cap: tanh from exp2(cap_e * q.k)
  float cap_log2;       // cap * log2(e)
  // cap_log2 * tanh(scale S / cap) = S * (poly[0] + poly[1] S^2 + ...) for
  // |S| <= poly_max (negative: nowhere), and with wide[] for |S| <= wide_max
  float poly[4], poly_max;
  float wide[7], wide_max;
  float inv_cap2;       // 1 / cap_log2^2
  const float* slopes;  // [H], or null
};

struct FwdParams {
  int32_t B, H, Hkv, Sq, Skv, D;
  int32_t n_super;    // ceil(Sq / 256)
  const int32_t* super_order;  // longest-first (table, super-tile) or null
  const uint32_t* dense;       // DENSE: [Sq][dense_words] bit-packed, else null
  int64_t dense_words;
  int32_t n_kvtiles;  // ceil(Skv / 128)
  int32_t num_units;  // B * H * n_super
  // mask
  uint32_t flags;
  int32_t window;
  const int8_t* block_mask;  // [tables][mi_nq][mi_nk]
  int32_t mi_nq, mi_nk, bq, bkv, tables;
  const int32_t* q_seg;      // [B][Sq]
  const int32_t* kv_seg;     // [B][Skv]
  const int32_t* seg_range;  // [B][Sq][2] from the mask-info
  const int32_t* seg_flags;  // bit 0: kv ids not sorted
  // scores
  int32_t score;     // bsm_score
  float scale_log2;  // softmax: scale * log2(e)
  float scale;       // pointwise
  float inv_sq;      // pointwise: 1 / Sq
  float pw_half;     // pointwise: scale / 2
  float pw_g;        // pointwise: scale / (2 Sq)
  ScoreMod mod;      // softmax: cap and distance bias
  // outputs
  uint16_t* out;  // bf16 bits
  int64_t o_sb, o_sh, o_ss;
  int32_t o_vec8;  // out and its strides allow 32-byte row stores
  float* lse;
  int32_t* unit_counter;  // workspace: next work unit (zeroed per launch)
  uint16_t* lists;        // workspace: [grid][kListBufs][kMaxKvTiles]
  uint64_t timeout_ns;
  // optional event trace (records of 16 bytes, cap per CTA), else null
  void* trace;
  uint32_t trace_cap;
};

// Whether a forward with modified scores takes the kernel with decoupled query
// tiles: not with an arbitrary mask, nor, as it adds a bias alone as slope /
// scale inside the product, with a scale that is negative or next to nothing.
inline bool fwd_mod_dt(const FwdParams& p) {
  return p.dense == nullptr && (p.mod.kind != kModBias || p.scale >= 0x1p-20f);
}

struct BwdParams {
  int32_t B, H, Hkv, Sq, Skv, D;
  // mask
  uint32_t flags;
  int32_t window;
  const int8_t* block_mask;  // [tables][mi_nq][mi_nk]
  int32_t mi_nq, mi_nk, bq, bkv;
  const int32_t* q_seg;   // [B][Sq] (SEGMENT only)
  const int32_t* kv_seg;  // [B][Skv]
  const uint32_t* dense;  // DENSE: [Sq][dense_words] bit-packed, else null
  int64_t dense_words;
  // scores
  int32_t score;
  float scale, scale_log2, inv_sq;
  ScoreMod mod;      // softmax: cap and distance bias
  const float* lse;  // forward logsumexp [B][H][Sq] (softmax)
  float* delta;      // workspace: D_q = sum_d dO * out, [B][H][Sq] (softmax)
  const uint16_t* out;   // forward output (softmax), bf16
  int64_t o_sb, o_sh, o_ss;
  const uint16_t* dout;  // gradient of the output, bf16
  int64_t do_sb, do_sh, do_ss;
  // gradients, bf16
  uint16_t* dq;
  int64_t dq_sb, dq_sh, dq_ss;
  uint16_t* dk;
  int64_t dk_sb, dk_sh, dk_ss;
  uint16_t* dv;
  int64_t dv_sb, dv_sh, dv_ss;
  // modified scores: the dK/dV walks cut into this many parts, and where they
  // leave f32 sums: [part][dV, dK][B][Hkv][Skv][D]
  int32_t parts;
  float* part_sums;
  uint64_t timeout_ns;
};
// Parts of a dK/dV walk (a function of the sizes alone).
int bwd_parts(int64_t B, int64_t H, int64_t Hkv, int64_t Sq, int64_t Skv);

struct AppendParams {
  uint8_t *k, *v;  // pages [num_pages][H_kv][page_size][D], e4m3
  float *k_scale, *v_scale;  // [num_pages][H_kv]
  int32_t num_pages, H_kv, page_size, D;
  const int32_t* table;  // [B][table_stride], max_pages entries per sequence
  int64_t table_stride;
  int32_t max_pages;
  const int32_t* lens;   // [B] tokens before the call
  const int32_t* n_new;  // [B] or null (T each)
  int32_t B, T;
  const uint16_t *k_new, *v_new;  // bf16 [B][H_kv][T][D]
  int64_t k_sb, k_sh, k_ss, v_sb, v_sh, v_ss;
};

// Norm and rotation of rows, as bsm_norm_rope and bsm_kv_append_rope take them.
struct TurnParams {
  const void *q_weight, *k_weight;  // [D] or null
  int32_t weights_bf16;
  int32_t norm;                     // 0: none
  float eps;
  bsm_rope rope;                    // dim 0: none
  const int32_t* pos;               // or null: token indices
  int64_t pos_sa, pos_sb, pos_ss;
};

struct RowView {
  uint16_t* data;
  int64_t sb, sh, ss;
};

struct NormRopeParams {
  RowView x[2], g[2], out[2];  // queries, keys; g: the backward's gradients
  int32_t B, S, D;
  int32_t heads[2];
  int32_t per[2];     // heads of one token that a group of lanes takes
  int32_t chunks[2];  // ceil(heads / per)
  // backward: blocks of the queries and of the keys, weight gradients (or
  // null) and the blocks' sums [block][D]
  int32_t blocks[2];
  float* dw[2];
  float* partial;
  TurnParams turn;
};
constexpr int kNormRopeMaxBlocks = 1024;  // of the backward

struct PagedParams {
  const uint8_t *k, *v;
  const float *k_scale, *v_scale;
  int32_t num_pages, H_kv, page_size, D;
  const int32_t* table;
  int64_t table_stride;
  int32_t max_pages;
  const int32_t* lens;  // [B] tokens, the queries' own among them
  int32_t B, H, T;
  int32_t window;  // 0 = none
  int32_t page_shift;  // log2(page_size)
  ScoreMod mod;
  float scale_x;  // scale * log2(e), or with a cap 2 scale log2(e) / cap
  const uint16_t* q;  // bf16 [B][H][T][D]
  int64_t q_sb, q_sh, q_ss;
  uint16_t* out;
  int64_t o_sb, o_sh, o_ss;
  float* lse;  // [B][H][T] or null
  float* parts;  // workspace: parts of the items cut across CTAs
  // drafted tokens (bsm_paged_attention_tree): how many of a sequence's last
  // tokens are drafts, or null (T), and the bits of the drafts that each sees,
  // tree[b * tree_sb + t * tree_st + word], or null (those up to itself)
  const int32_t* n_new;
  const uint32_t* tree;
  int64_t tree_sb, tree_st;
};
// The workspace: for up to kPaMaxSms SMs with kPaMaxPerSm CTAs each, two parts
// per CTA: o, m and l of up to 16 query rows.
constexpr int kPaMaxSms = 256, kPaMaxPerSm = 4;
constexpr size_t kPaWorkspaceBytes = static_cast<size_t>(kPaMaxSms) *
                                     kPaMaxPerSm * 2 * 16 * (128 + 2) * 4;

// Launchers (return a cudaError_t from the launch).
cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t stream);
cudaError_t launch_kv_append_rope(const AppendParams& p, const TurnParams& t,
                                  cudaStream_t stream);
cudaError_t launch_norm_rope(NormRopeParams& p, int num_sms,
                             cudaStream_t stream);
cudaError_t launch_norm_rope_bwd(NormRopeParams& p, int num_sms,
                                 cudaStream_t stream);
cudaError_t launch_paged_attention(const PagedParams& p, int num_sms,
                                   cudaStream_t stream);
cudaError_t launch_paged_tree(const PagedParams& p, int num_sms,
                              cudaStream_t stream);
// The same for many query rows, on the tensor core: tiles of 128 query rows
// that a CTA takes at once (0: too few rows, launch_paged_tree serves them),
// its workspace (for up to kTreeMaxSms SMs) and launch.
constexpr int kTreeMaxSms = 160;
int tree_tiles(int64_t rows);
size_t tree_workspace_bytes(int64_t rows, int D);
cudaError_t launch_tree_tc(const PagedParams& p, int num_sms,
                           uint64_t timeout_ns, cudaStream_t stream);
// One block whose roles wait for steps that never come.
cudaError_t launch_tree_selftest(uint64_t timeout_ns, cudaStream_t stream);
// Reads and clears its device error record.
cudaError_t read_tree_error(int code, int32_t out[4]);
// Reads and clears the device error record of the cache kernels.
cudaError_t read_cache_error(int32_t out[4]);
cudaError_t launch_mask_info(const MaskInfoParams& p, cudaStream_t stream);
cudaError_t launch_pack_dense(const uint8_t* mask, int64_t stride, int32_t Sq,
                              int32_t Skv, uint32_t* words, int32_t row_words,
                              int num_sms, cudaStream_t stream);
// Whether a mask of these sizes is built in one launch.
bool mask_info_fused(int64_t tables, int64_t nq, int64_t nk);
int fwd_grid_size(const FwdParams& p, int num_sms);
cudaError_t launch_splash_fwd(const FwdParams& p, const CUtensorMap& tq,
                              const CUtensorMap& tk, const CUtensorMap& tv,
                              int num_sms, cudaStream_t stream);
cudaError_t launch_wait_selftest(uint64_t timeout_ns, cudaStream_t stream);
// D_q (softmax), then the dK/dV and dQ kernels.
cudaError_t launch_splash_bwd(const BwdParams& p, const CUtensorMap& tq,
                              const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& tdo, cudaStream_t stream);
// Reads and clears the device error record of the backward kernels.
cudaError_t read_bwd_error(int32_t out[4]);
// Sets the thread-local text returned by bsm_last_error().
void set_last_error(const char* msg);
// Reads and clears the device error record of the forward kernel TU.
cudaError_t read_device_error(int32_t out[4], cudaStream_t stream);

}  // namespace bsm
