// Host side of the C ABI declared in include/bsm.h: argument validation,
// layout of the caller's mask-info buffer, TMA tensor-map encoding and the
// kernel launches.  Allocates no device memory.
#include <cudaTypedefs.h>

#include <atomic>
#include <chrono>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <string>

#include "bsm_internal.h"

namespace {

thread_local std::string g_last_error;

bsm_status fail(bsm_status s, const std::string& msg) {
  g_last_error = msg;
  return s;
}

bsm_status cuda_fail(cudaError_t e, const char* what) {
  return fail(BSM_ERR_CUDA,
              std::string(what) + ": " + cudaGetErrorName(e) + " (" +
                  cudaGetErrorString(e) + ")");
}

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool is_block_size(int32_t b) {
  return b >= 16 && b <= 512 && (b & (b - 1)) == 0;
}

struct MiLayout {
  size_t off_bm, off_dn, off_rp, off_idx, off_cls, off_sr, off_sf, off_so,
      off_stage, off_ticket, total;
};

// seg_rows = B * Sq with segment ids, else 0.
int64_t super_pairs(int64_t tables, int64_t Sq) {
  return tables * ((Sq + bsm::kUnitRows - 1) / bsm::kUnitRows);
}

MiLayout mi_layout(int64_t tables, int64_t nq, int64_t nk, int64_t seg_rows,
                   int64_t pairs) {
  const size_t cells = static_cast<size_t>(tables * nq * nk);
  const size_t rows = static_cast<size_t>(tables * nq);
  MiLayout L;
  size_t o = 0;
  L.off_bm = o;
  o = align_up(o + cells, 256);
  L.off_dn = o;
  o = align_up(o + cells * 4, 256);
  L.off_rp = o;
  o = align_up(o + (rows + 1) * 4, 256);
  L.off_idx = o;
  o = align_up(o + cells * 4, 256);
  L.off_cls = o;
  o = align_up(o + cells, 256);
  L.off_sr = o;
  o = align_up(o + static_cast<size_t>(seg_rows) * 8, 256);
  L.off_sf = o;  // [0]: any table unsorted; [1 + t]: table t (builder scratch)
  o = align_up(o + 4 * (1 + (seg_rows > 0 ? tables : 0)), 256);
  L.off_so = o;
  if (pairs <= bsm::kMaxSuperOrder)
    o = align_up(o + static_cast<size_t>(pairs) * 4, 256);
  // one-launch build: the rows' staged lists and the (epoch, count) ticket
  L.off_stage = o;
  L.off_ticket = o;
  if (bsm::mask_info_fused(tables, nq, nk)) {
    o = align_up(o + cells * 2, 256);
    L.off_ticket = o;
    o = align_up(o + 8, 256);
  }
  L.total = o;
  return L;
}

bsm_status check_spec(const bsm_mask_spec* spec) {
  if (spec == nullptr) return fail(BSM_ERR_INVALID_ARG, "mask spec is NULL");
  const uint32_t known = BSM_MASK_CAUSAL | BSM_MASK_LOCAL | BSM_MASK_SEGMENT |
                         BSM_MASK_BAND | BSM_MASK_DENSE;
  if (spec->flags & ~known)
    return fail(BSM_ERR_INVALID_ARG, "unknown mask flag bits");
  if ((spec->flags & BSM_MASK_BAND) && !(spec->flags & BSM_MASK_LOCAL))
    return fail(BSM_ERR_INVALID_ARG, "BSM_MASK_BAND needs BSM_MASK_LOCAL");
  if ((spec->flags & BSM_MASK_LOCAL) && spec->window < 1)
    return fail(BSM_ERR_INVALID_ARG, "local window must be >= 1");
  return BSM_OK;
}

bsm_status check_mi_shape(const bsm_mask_spec* spec, int32_t B, int32_t Sq,
                          int32_t Skv, int32_t bq, int32_t bkv) {
  bsm_status s = check_spec(spec);
  if (s != BSM_OK) return s;
  if (B < 0 || Sq < 0 || Skv < 0)
    return fail(BSM_ERR_INVALID_ARG, "negative size");
  if (Sq > bsm::kMaxSeq || Skv > bsm::kMaxSeq)
    return fail(BSM_ERR_UNSUPPORTED, "sequence length above 262144");
  if (!is_block_size(bq) || !is_block_size(bkv))
    return fail(BSM_ERR_INVALID_ARG,
                "block_q and block_kv must be powers of two in [16, 512]");
  return BSM_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                         cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// 4-D bf16 map over [B][H][S][D] storage with element strides (sb, sh, ss);
// box = 64 head-dim elements (128 bytes, 128-byte swizzle) x 128 rows.
bsm_status make_map(CUtensorMap* map, const void* ptr, int32_t B, int32_t H,
                    int32_t S, int32_t D, const int64_t strides[3],
                    const char* name) {
  auto enc = tensor_map_encoder();
  if (enc == nullptr)
    return fail(BSM_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  // Strides of size-1 dimensions are never used; give them a valid value.
  const int64_t ss = S > 1 ? strides[2] : D;
  const int64_t sh = H > 1 ? strides[1] : ss * S;
  const int64_t sb = B > 1 ? strides[0] : sh * H;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(S),
                        static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(B)};
  cuuint64_t gstr[3] = {static_cast<cuuint64_t>(ss * 2),
                        static_cast<cuuint64_t>(sh * 2),
                        static_cast<cuuint64_t>(sb * 2)};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(bsm::kTileM), 1, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                   const_cast<void*>(ptr), dims, gstr, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(BSM_ERR_INVALID_ARG,
                std::string("tensor map for ") + name +
                    " rejected (strides must be multiples of 8 elements)");
  return BSM_OK;
}

bsm_status check_device(int* num_sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  int major = 0, minor = 0, sms = 0;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (major != 10 || minor != 3)
    return fail(BSM_ERR_UNSUPPORTED,
                "libbsm is built for sm_103a (GB300) only; device is sm_" +
                    std::to_string(major) + std::to_string(minor));
  if (num_sms) *num_sms = sms;
  return BSM_OK;
}

uint64_t wait_timeout_ns() {
  static uint64_t v = [] {
    const char* s = std::getenv("BSM_WAIT_TIMEOUT_NS");
    if (s != nullptr) {
      const unsigned long long x = std::strtoull(s, nullptr, 10);
      if (x >= 1000ull && x <= 100000000000ull) return static_cast<uint64_t>(x);
    }
    return static_cast<uint64_t>(2000000000ull);  // 2 s
  }();
  return v;
}

std::mutex g_trace_mu;
void* g_trace_buf = nullptr;
size_t g_trace_bytes = 0;

bool aligned16(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// The kernels' form of a caller's score modification (mod may be NULL).
bsm_status check_mod(const bsm_score_mod* mod, float scale, int32_t score,
                     bsm::ScoreMod* out) {
  *out = bsm::ScoreMod{};
  out->poly_max = out->wide_max = -1.f;
  if (mod == nullptr) return BSM_OK;
  if (!(mod->softcap >= 0.f) || !std::isfinite(mod->softcap))
    return fail(BSM_ERR_INVALID_ARG, "softcap must be finite and >= 0");
  const double log2e = 1.4426950408889634;
  if (mod->softcap > 0.f) {
    out->kind |= bsm::kModCap;
    const double cap = mod->softcap, c1 = static_cast<double>(scale) / cap;
    out->cap_e = static_cast<float>(2.0 * log2e * c1);
    out->cap_log2 = static_cast<float>(cap * log2e);
    if (!std::isfinite(out->cap_e) || !std::isfinite(out->cap_log2 * 2.f))
      return fail(BSM_ERR_INVALID_ARG, "softcap out of range for this scale");
    // tanh(y) / y in powers of y^2, interpolated at the Chebyshev nodes of y^2:
    // four terms for |y| <= 0.5, off by at most 5.5e-7 of the value there (a
    // logit by 2.8e-7 of the cap), seven for |y| <= 1.2, off by 4.2e-7.  The
    // kernels take them in powers of S = y / c1; c1 is kept to a range where
    // no coefficient leaves f32's.
    static const double kNear[4] = {0.999999451, -0.3332628423, 0.1318993943,
                                    -0.04439273843};
    static const double kWide[7] = {0.9999995837,    -0.3333048319,
                                    0.1330069738,    -0.05252428411,
                                    0.01868168763,   -0.004920490605,
                                    0.0006554170517};
    if (std::fabs(c1) >= 0x1p-18 && std::fabs(c1) <= 0x1p6 && cap <= 0x1p20) {
      double f = cap * log2e * c1;
      for (int i = 0; i < 7; ++i, f *= c1 * c1) {
        if (i < 4) out->poly[i] = static_cast<float>(kNear[i] * f);
        out->wide[i] = static_cast<float>(kWide[i] * f);
      }
      out->poly_max = static_cast<float>(0.5 / std::fabs(c1));
      if (std::fabs(c1) >= 0x1p-10)
        out->wide_max = static_cast<float>(1.2 / std::fabs(c1));
    }
    out->inv_cap2 = 1.f / (out->cap_log2 * out->cap_log2);
  }
  if (mod->alibi_slopes != nullptr) {
    out->kind |= bsm::kModBias;
    out->slopes = mod->alibi_slopes;
  }
  if (out->kind != 0 && score != BSM_SCORE_SOFTMAX)
    return fail(BSM_ERR_INVALID_ARG,
                "softcap and slopes modify softmax scores only");
  if ((reinterpret_cast<uintptr_t>(mod->alibi_slopes) & 3u) != 0)
    return fail(BSM_ERR_INVALID_ARG, "alibi_slopes must be 4-byte aligned");
  return BSM_OK;
}

// Shape of a cache, its page table and a batch of B sequences with T tokens.
bsm_status check_cache(const bsm_kv_cache* c, int64_t table_stride,
                       int32_t max_pages, int32_t B, int32_t T) {
  if (c == nullptr) return fail(BSM_ERR_INVALID_ARG, "cache is NULL");
  if (B < 0 || T < 0 || max_pages < 0 || c->num_pages < 0 || c->H_kv < 0)
    return fail(BSM_ERR_INVALID_ARG, "negative size");
  if (c->D != 64 && c->D != 128)
    return fail(BSM_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 &&
      c->page_size != 128)
    return fail(BSM_ERR_UNSUPPORTED, "page_size must be 16, 32, 64 or 128");
  if (B > 65535 || c->H_kv > 32767)
    return fail(BSM_ERR_UNSUPPORTED, "too many sequences or heads");
  if (T > (1 << 24) ||
      static_cast<int64_t>(max_pages) * c->page_size > (1 << 30))
    return fail(BSM_ERR_UNSUPPORTED, "more than 2^30 tokens per sequence");
  if (B > 1 && table_stride < max_pages)
    return fail(BSM_ERR_INVALID_ARG, "table_stride must be >= max_pages");
  return BSM_OK;
}

bsm_status check_cache_memory(const bsm_kv_cache* c, const int32_t* table,
                              int32_t max_pages, const int32_t* lens) {
  if (lens == nullptr || (reinterpret_cast<uintptr_t>(lens) & 3u) != 0)
    return fail(BSM_ERR_INVALID_ARG, "lens must be non-NULL, 4-byte aligned");
  if ((table == nullptr && max_pages > 0) ||
      (reinterpret_cast<uintptr_t>(table) & 3u) != 0)
    return fail(BSM_ERR_INVALID_ARG,
                "page_table must be non-NULL, 4-byte aligned");
  if (c->k == nullptr || c->v == nullptr || !aligned16(c->k) || !aligned16(c->v))
    return fail(BSM_ERR_INVALID_ARG,
                "the cache's pages must be non-NULL and 16-byte aligned");
  if (c->k_scale == nullptr || c->v_scale == nullptr ||
      (reinterpret_cast<uintptr_t>(c->k_scale) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(c->v_scale) & 3u) != 0)
    return fail(BSM_ERR_INVALID_ARG,
                "the cache's scales must be non-NULL, 4-byte aligned");
  return BSM_OK;
}

// A [B][heads][S][D] view: aligned data, positive strides, multiples of 8.
bsm_status check_view(const bsm_tensor* t, int64_t B, int64_t heads, int64_t S,
                      const char* name) {
  if (t->data == nullptr || !aligned16(t->data))
    return fail(BSM_ERR_INVALID_ARG,
                std::string(name) + " must be non-NULL and 16-byte aligned");
  const int64_t sizes[3] = {B, heads, S};
  for (int d = 0; d < 3; ++d)
    if (sizes[d] > 1 && (t->strides[d] <= 0 || t->strides[d] % 8 != 0))
      return fail(BSM_ERR_INVALID_ARG,
                  std::string(name) +
                      " strides must be positive multiples of 8");
  return BSM_OK;
}

// A norm, a rotation and positions of rows of D elements: at least one of the
// first two.
bsm_status check_turn(const bsm_head_norm* norm, const bsm_rope* rope,
                      const bsm_positions* pos, int32_t D,
                      bsm::TurnParams* t) {
  *t = bsm::TurnParams{};
  if (norm == nullptr && rope == nullptr)
    return fail(BSM_ERR_INVALID_ARG, "neither a norm nor a rotation");
  if (norm != nullptr) {
    if (!(norm->eps >= 0.f) || !std::isfinite(norm->eps))
      return fail(BSM_ERR_INVALID_ARG, "eps must be finite and >= 0");
    const uintptr_t low = norm->weights_bf16 ? 1u : 3u;
    for (const void* w : {norm->q_weight, norm->k_weight})
      if ((reinterpret_cast<uintptr_t>(w) & low) != 0)
        return fail(BSM_ERR_INVALID_ARG,
                    "weights must be aligned to their element");
    t->norm = 1;
    t->eps = norm->eps;
    t->q_weight = norm->q_weight;
    t->k_weight = norm->k_weight;
    t->weights_bf16 = norm->weights_bf16 != 0;
  }
  if (rope == nullptr) {
    if (pos != nullptr && pos->data != nullptr)
      return fail(BSM_ERR_INVALID_ARG, "positions without a rotation");
    return BSM_OK;
  }
  if (rope->dim < 16 || rope->dim > 128 || rope->dim % 16 != 0 ||
      rope->axes < 1 || rope->axes > 4)
    return fail(BSM_ERR_INVALID_ARG, "a bsm_rope that bsm_rope_init did not fill");
  if (rope->dim > D)
    return fail(BSM_ERR_INVALID_ARG, "the rotation is wider than head_dim");
  for (int i = 0; i < rope->dim / 2; ++i)
    if (rope->axis[i] >= rope->axes)
      return fail(BSM_ERR_INVALID_ARG, "a bsm_rope that bsm_rope_init did not fill");
  t->rope = *rope;
  if (pos != nullptr && pos->data != nullptr) {
    if ((reinterpret_cast<uintptr_t>(pos->data) & 3u) != 0)
      return fail(BSM_ERR_INVALID_ARG, "positions must be 4-byte aligned");
    t->pos = pos->data;
    t->pos_sa = pos->strides[0];
    t->pos_sb = pos->strides[1];
    t->pos_ss = pos->strides[2];
  }
  return BSM_OK;
}

// The sizes of a norm and rotation; rows are counted in 31 bits.
bsm_status check_rows(int32_t B, int32_t H, int32_t H_kv, int32_t S,
                      int32_t D) {
  if (B < 0 || H < 0 || H_kv < 0 || S < 0)
    return fail(BSM_ERR_INVALID_ARG, "negative size");
  if (D != 64 && D != 128)
    return fail(BSM_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  const double rows = static_cast<double>(B) * S *
                      (static_cast<double>(H) + H_kv);
  if (rows > 2147483647.0 || static_cast<double>(B) * S > 2147483647.0)
    return fail(BSM_ERR_UNSUPPORTED, "more than 2^31 - 1 rows");
  return BSM_OK;
}

// A result that begins where its input does must lie as that does, or rows are
// written that are still to be read.
bsm_status check_in_place(const bsm_tensor* in, const bsm_tensor* out,
                          int64_t B, int64_t heads, int64_t S,
                          const char* name) {
  const int64_t sizes[3] = {B, heads, S};
  for (int d = 0; d < 3 && in->data == out->data; ++d)
    if (sizes[d] > 1 && in->strides[d] != out->strides[d])
      return fail(BSM_ERR_INVALID_ARG,
                  std::string(name) + " in place must have its input's strides");
  return BSM_OK;
}

bsm::RowView row_view(const bsm_tensor* t) {
  if (t == nullptr) return bsm::RowView{nullptr, 0, 0, 0};
  return bsm::RowView{static_cast<uint16_t*>(t->data), t->strides[0],
                      t->strides[1], t->strides[2]};
}

// A new epoch for every mask-info build (40 bits, never 0), starting at a
// value that differs between processes, so that a ticket word left in a
// reused buffer by an earlier build never matches.
uint64_t next_build_epoch() {
  static std::atomic<uint64_t> counter{
      (static_cast<uint64_t>(
           std::chrono::steady_clock::now().time_since_epoch().count()) *
       0x9E3779B97F4A7C15ull) ^
      static_cast<uint64_t>(reinterpret_cast<uintptr_t>(&counter))};
  constexpr uint64_t kMask = (uint64_t{1} << 40) - 1;
  uint64_t e = 0;
  while (e == 0) e = counter.fetch_add(1, std::memory_order_relaxed) & kMask;
  return e;
}

}  // namespace

namespace bsm {
void set_last_error(const char* msg) { g_last_error = msg; }
}  // namespace bsm

extern "C" {

size_t bsm_mask_info_bytes(const bsm_mask_spec* spec, int32_t B, int32_t Sq,
                           int32_t Skv, int32_t block_q, int32_t block_kv) {
  if (check_mi_shape(spec, B, Sq, Skv, block_q, block_kv) != BSM_OK) return 0;
  const bool seg = (spec->flags & BSM_MASK_SEGMENT) != 0;
  const int64_t tables = seg ? B : 1;
  const int64_t nq = (Sq + block_q - 1) / block_q;
  const int64_t nk = (Skv + block_kv - 1) / block_kv;
  return mi_layout(tables, nq, nk, seg ? static_cast<int64_t>(B) * Sq : 0,
                   super_pairs(tables, Sq))
      .total;
}

bsm_status bsm_build_mask_info(const bsm_mask_spec* spec,
                               const int32_t* q_segment_ids,
                               const int32_t* kv_segment_ids, int32_t B,
                               int32_t Sq, int32_t Skv, int32_t block_q,
                               int32_t block_kv, void* buffer,
                               size_t buffer_bytes, bsm_mask_info* info,
                               void* stream) {
  g_last_error.clear();
  bsm_status s = check_mi_shape(spec, B, Sq, Skv, block_q, block_kv);
  if (s != BSM_OK) return s;
  if (info == nullptr) return fail(BSM_ERR_INVALID_ARG, "info is NULL");
  const bool seg = (spec->flags & BSM_MASK_SEGMENT) != 0;
  if (seg && (q_segment_ids == nullptr || kv_segment_ids == nullptr))
    return fail(BSM_ERR_INVALID_ARG,
                "BSM_MASK_SEGMENT needs both q and kv segment ids");
  if (!seg && (q_segment_ids != nullptr || kv_segment_ids != nullptr))
    return fail(BSM_ERR_INVALID_ARG,
                "segment ids given without BSM_MASK_SEGMENT");
  if (seg && B < 1) return fail(BSM_ERR_INVALID_ARG, "B must be >= 1");
  const bool dense = (spec->flags & BSM_MASK_DENSE) != 0;
  if (dense && (spec->dense_bits == nullptr ||
                spec->dense_row_words < (static_cast<int64_t>(Skv) + 31) / 32))
    return fail(BSM_ERR_INVALID_ARG,
                "BSM_MASK_DENSE needs dense_bits and dense_row_words >= "
                "ceil(Skv / 32)");
  const int64_t tables = seg ? B : 1;
  const int64_t nq = (Sq + block_q - 1) / block_q;
  const int64_t nk = (Skv + block_kv - 1) / block_kv;
  if (tables > 65535)
    return fail(BSM_ERR_UNSUPPORTED, "too many mask tables");
  const int64_t pairs = super_pairs(tables, Sq);
  const MiLayout L = mi_layout(
      tables, nq, nk, seg ? static_cast<int64_t>(B) * Sq : 0, pairs);
  if (buffer == nullptr) return fail(BSM_ERR_INVALID_ARG, "buffer is NULL");
  if ((reinterpret_cast<uintptr_t>(buffer) & 255u) != 0)
    return fail(BSM_ERR_INVALID_ARG, "buffer must be 256-byte aligned");
  if (buffer_bytes < L.total)
    return fail(BSM_ERR_INVALID_ARG,
                "buffer too small: need " + std::to_string(L.total) +
                    " bytes");
  s = check_device(nullptr);
  if (s != BSM_OK) return s;

  uint8_t* base = static_cast<uint8_t*>(buffer);
  bsm_mask_info mi;
  mi.flags = spec->flags;
  mi.window = (spec->flags & BSM_MASK_LOCAL) ? spec->window : 0;
  mi.num_tables = static_cast<int32_t>(tables);
  mi.Sq = Sq;
  mi.Skv = Skv;
  mi.block_q = block_q;
  mi.block_kv = block_kv;
  mi.nq = static_cast<int32_t>(nq);
  mi.nk = static_cast<int32_t>(nk);
  mi.block_mask = reinterpret_cast<int8_t*>(base + L.off_bm);
  mi.data_next = reinterpret_cast<int32_t*>(base + L.off_dn);
  mi.row_ptr = reinterpret_cast<int32_t*>(base + L.off_rp);
  mi.kv_idx = reinterpret_cast<int32_t*>(base + L.off_idx);
  mi.kv_cls = reinterpret_cast<int8_t*>(base + L.off_cls);
  mi.seg_range = reinterpret_cast<int32_t*>(base + L.off_sr);
  mi.seg_flags = reinterpret_cast<int32_t*>(base + L.off_sf);
  mi.num_super = static_cast<int32_t>((Sq + bsm::kUnitRows - 1) / bsm::kUnitRows);
  mi.dense_bits = dense ? spec->dense_bits : nullptr;
  mi.dense_row_words = dense ? spec->dense_row_words : 0;
  mi.super_order = pairs <= bsm::kMaxSuperOrder
                       ? reinterpret_cast<int32_t*>(base + L.off_so)
                       : nullptr;

  bsm::MaskInfoParams p;
  p.flags = mi.flags;
  p.window = mi.window;
  p.Sq = Sq;
  p.Skv = Skv;
  p.bq = block_q;
  p.bkv = block_kv;
  p.nq = mi.nq;
  p.nk = mi.nk;
  p.tables = mi.num_tables;
  p.q_seg = q_segment_ids;
  p.kv_seg = kv_segment_ids;
  p.block_mask = mi.block_mask;
  p.data_next = mi.data_next;
  p.row_ptr = mi.row_ptr;
  p.kv_idx = mi.kv_idx;
  p.kv_cls = mi.kv_cls;
  p.seg_range = mi.seg_range;
  p.seg_flags = mi.seg_flags;
  p.n_super = mi.num_super;
  p.super_order = mi.super_order;
  p.dense = mi.dense_bits;
  p.dense_words = mi.dense_row_words;
  p.fused = bsm::mask_info_fused(tables, nq, nk) ? 1 : 0;
  p.staged = reinterpret_cast<uint16_t*>(base + L.off_stage);
  p.ticket = reinterpret_cast<unsigned long long*>(base + L.off_ticket);
  p.epoch = next_build_epoch();
  cudaError_t e =
      bsm::launch_mask_info(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "mask-info launch");
  *info = mi;
  return BSM_OK;
}

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
                          void* stream) {
  return bsm_splash_fwd_mod(q, k, v, q_strides, k_strides, v_strides,
                            o_strides, B, H, H_kv, Sq, Skv, D, info,
                            q_segment_ids, kv_segment_ids, scale, score,
                            nullptr, out, lse, workspace, workspace_bytes,
                            stream);
}

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
                              size_t workspace_bytes, void* stream) {
  g_last_error.clear();
  if (B < 0 || H < 0 || H_kv < 0 || Sq < 0 || Skv < 0)
    return fail(BSM_ERR_INVALID_ARG, "negative size");
  if (H_kv == 0 ? H != 0 : (H % H_kv) != 0)
    return fail(BSM_ERR_INVALID_ARG, "H must be a multiple of H_kv");
  if (D != 64 && D != 128)
    return fail(BSM_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (Sq > bsm::kMaxSeq || Skv > bsm::kMaxSeq)
    return fail(BSM_ERR_UNSUPPORTED, "sequence length above 262144");
  if (score != BSM_SCORE_SOFTMAX && score != BSM_SCORE_POINTWISE)
    return fail(BSM_ERR_INVALID_ARG, "unknown score path");
  if (score == BSM_SCORE_POINTWISE && lse != nullptr)
    return fail(BSM_ERR_INVALID_ARG,
                "the pointwise score path has no logsumexp; pass lse = NULL");
  if (!std::isfinite(scale)) return fail(BSM_ERR_INVALID_ARG, "scale not finite");
  bsm::ScoreMod sm_mod;
  if (const bsm_status ms = check_mod(mod, scale, score, &sm_mod); ms != BSM_OK)
    return ms;
  if (info == nullptr) return fail(BSM_ERR_INVALID_ARG, "mask info is NULL");
  if (info->Sq != Sq || info->Skv != Skv)
    return fail(BSM_ERR_INVALID_ARG,
                "mask info was built for other sequence lengths");
  const bool seg = (info->flags & BSM_MASK_SEGMENT) != 0;
  if (info->num_tables != (seg ? B : 1))
    return fail(BSM_ERR_INVALID_ARG,
                "mask info was built for another batch size");
  if (!is_block_size(info->block_q) || !is_block_size(info->block_kv) ||
      info->nq != (Sq + info->block_q - 1) / info->block_q ||
      info->nk != (Skv + info->block_kv - 1) / info->block_kv ||
      info->num_super != (Sq + bsm::kUnitRows - 1) / bsm::kUnitRows)
    return fail(BSM_ERR_INVALID_ARG, "inconsistent mask info");
  if (seg && (q_segment_ids == nullptr || kv_segment_ids == nullptr))
    return fail(BSM_ERR_INVALID_ARG,
                "BSM_MASK_SEGMENT needs both q and kv segment ids");
  if (!seg && (q_segment_ids != nullptr || kv_segment_ids != nullptr))
    return fail(BSM_ERR_INVALID_ARG,
                "segment ids given without BSM_MASK_SEGMENT");
  if ((info->flags & BSM_MASK_DENSE) &&
      (info->dense_bits == nullptr ||
       info->dense_row_words < (static_cast<int64_t>(Skv) + 31) / 32))
    return fail(BSM_ERR_INVALID_ARG, "mask info lacks its dense mask");
  if (seg && (info->seg_range == nullptr || info->seg_flags == nullptr))
    return fail(BSM_ERR_INVALID_ARG, "mask info lacks segment ranges");
  const int64_t n_super = (Sq + bsm::kUnitRows - 1) / bsm::kUnitRows;
  const int64_t units = static_cast<int64_t>(B) * H * n_super;
  if (units == 0) return BSM_OK;
  if (units > 0x7fffffff) return fail(BSM_ERR_UNSUPPORTED, "too many tiles");
  if (q == nullptr || out == nullptr || (Skv > 0 && (k == nullptr || v == nullptr)))
    return fail(BSM_ERR_INVALID_ARG, "NULL tensor");
  if (workspace == nullptr || workspace_bytes < bsm::kFwdWorkspaceBytes ||
      !aligned16(workspace))
    return fail(BSM_ERR_INVALID_ARG,
                "workspace must be >= bsm_splash_fwd_workspace_bytes() bytes, "
                "16-byte aligned");
  if (q_strides == nullptr || k_strides == nullptr || v_strides == nullptr ||
      o_strides == nullptr)
    return fail(BSM_ERR_INVALID_ARG, "NULL strides");
  if (!aligned16(q) || !aligned16(out) || (Skv > 0 && (!aligned16(k) || !aligned16(v))))
    return fail(BSM_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
  const int64_t sizes_q[3] = {B, H, Sq};
  const int64_t sizes_kv[3] = {B, H_kv, Skv};
  for (int d = 0; d < 3; ++d) {
    if (sizes_q[d] > 1 && ((q_strides[d] % 8) != 0 || q_strides[d] <= 0))
      return fail(BSM_ERR_INVALID_ARG, "q strides must be positive multiples of 8");
    if (sizes_q[d] > 1 && ((o_strides[d] % 8) != 0 || o_strides[d] <= 0))
      return fail(BSM_ERR_INVALID_ARG, "out strides must be positive multiples of 8");
    if (Skv > 0 && sizes_kv[d] > 1 && ((k_strides[d] % 8) != 0 || k_strides[d] <= 0 ||
                            (v_strides[d] % 8) != 0 || v_strides[d] <= 0))
      return fail(BSM_ERR_INVALID_ARG, "k/v strides must be positive multiples of 8");
  }
  int num_sms = 0;
  bsm_status s = check_device(&num_sms);
  if (s != BSM_OK) return s;

  CUtensorMap tq, tk, tv;
  std::memset(&tk, 0, sizeof(tk));
  std::memset(&tv, 0, sizeof(tv));
  s = make_map(&tq, q, B, H, Sq, D, q_strides, "q");
  if (s != BSM_OK) return s;
  if (Skv > 0) {
    s = make_map(&tk, k, B, H_kv, Skv, D, k_strides, "k");
    if (s != BSM_OK) return s;
    s = make_map(&tv, v, B, H_kv, Skv, D, v_strides, "v");
    if (s != BSM_OK) return s;
  }

  bsm::FwdParams p;
  p.B = B;
  p.H = H;
  p.Hkv = H_kv;
  p.Sq = Sq;
  p.Skv = Skv;
  p.D = D;
  p.n_super = static_cast<int32_t>(n_super);
  p.n_kvtiles = (Skv + bsm::kTileN - 1) / bsm::kTileN;
  p.num_units = static_cast<int32_t>(units);
  p.flags = info->flags;
  p.window = info->window;
  p.block_mask = info->block_mask;
  p.mi_nq = info->nq;
  p.mi_nk = info->nk;
  p.bq = info->block_q;
  p.bkv = info->block_kv;
  p.tables = info->num_tables;
  p.q_seg = q_segment_ids;
  p.kv_seg = kv_segment_ids;
  p.seg_range = info->seg_range;
  p.seg_flags = info->seg_flags;
  p.super_order = info->super_order;
  p.dense = (info->flags & BSM_MASK_DENSE) ? info->dense_bits : nullptr;
  p.dense_words = info->dense_row_words;
  p.score = score;
  p.mod = sm_mod;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.scale = scale;
  p.inv_sq = Sq > 0 ? static_cast<float>(1.0 / static_cast<double>(Sq)) : 0.f;
  // pointwise: x sigmoid(x) / Sq = g (1 + tanh(x / 2)), x = scale s,
  // g = x / (2 Sq)
  p.pw_half = static_cast<float>(0.5 * static_cast<double>(scale));
  p.pw_g = Sq > 0 ? static_cast<float>(0.5 * static_cast<double>(scale) /
                                        static_cast<double>(Sq))
                  : 0.f;
  p.out = static_cast<uint16_t*>(out);
  p.o_sb = o_strides[0];
  p.o_sh = o_strides[1];
  p.o_ss = o_strides[2];
  p.o_vec8 = (reinterpret_cast<uintptr_t>(out) % 32 == 0 &&
              o_strides[0] % 16 == 0 && o_strides[1] % 16 == 0 &&
              o_strides[2] % 16 == 0)
                 ? 1
                 : 0;
  p.lse = lse;
  p.unit_counter = static_cast<int32_t*>(workspace);
  p.lists = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + 256);
  if (bsm::fwd_grid_size(p, num_sms) > bsm::kMaxCtas)
    return fail(BSM_ERR_UNSUPPORTED, "more than 256 SMs");
  p.timeout_ns = wait_timeout_ns();
  p.trace = nullptr;
  p.trace_cap = 0;
  {
    std::lock_guard<std::mutex> lk(g_trace_mu);
    const int grid = bsm::fwd_grid_size(p, num_sms);
    if (g_trace_buf != nullptr && grid > 0) {
      const size_t per = g_trace_bytes / 16 / static_cast<size_t>(grid);
      if (per >= 8) {
        p.trace = g_trace_buf;
        p.trace_cap = static_cast<uint32_t>(per - 2);
      }
    }
  }
  cudaError_t e;
  if (sm_mod.kind != 0 && bsm::fwd_mod_dt(p) && units <= num_sms) {
    // every unit has a CTA of its own: nothing to count (small calls are bound
    // by latency, and the reset is a node of its own on the stream)
    p.unit_counter = nullptr;
  } else {
    e = cudaMemsetAsync(workspace, 0, sizeof(int32_t),
                        static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "workspace reset");
  }
  e = bsm::launch_splash_fwd(p, tq, tk, tv, num_sms,
                             static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "splash_fwd launch");
  return BSM_OK;
}

bsm_status bsm_pack_dense_mask(const uint8_t* mask, int64_t mask_row_stride,
                               int32_t Sq, int32_t Skv, uint32_t* words,
                               int32_t row_words, void* stream) {
  g_last_error.clear();
  if (Sq < 0 || Skv < 0)
    return fail(BSM_ERR_INVALID_ARG, "Sq and Skv must be >= 0");
  if (row_words < (static_cast<int64_t>(Skv) + 31) / 32)
    return fail(BSM_ERR_INVALID_ARG, "row_words must be >= ceil(Skv / 32)");
  if (mask_row_stride < Skv)
    return fail(BSM_ERR_INVALID_ARG, "mask_row_stride must be >= Skv");
  if (static_cast<int64_t>(Sq) * row_words == 0) return BSM_OK;
  if (mask == nullptr || words == nullptr)
    return fail(BSM_ERR_INVALID_ARG, "mask and words must be non-NULL");
  int num_sms = 0;
  bsm_status s = check_device(&num_sms);
  if (s != BSM_OK) return s;
  const cudaError_t e = bsm::launch_pack_dense(
      mask, mask_row_stride, Sq, Skv, words, row_words, num_sms,
      static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "pack_dense launch");
  return BSM_OK;
}

size_t bsm_splash_fwd_workspace_bytes(void) { return bsm::kFwdWorkspaceBytes; }

size_t bsm_splash_bwd_workspace_bytes(int32_t B, int32_t H, int32_t Sq,
                                      int32_t score) {
  if (B < 0 || H < 0 || Sq < 0) return 0;
  if (score != BSM_SCORE_SOFTMAX) return 0;
  return align_up(static_cast<size_t>(B) * H * Sq * sizeof(float), 256);
}

size_t bsm_splash_bwd_mod_workspace_bytes(int32_t B, int32_t H, int32_t H_kv,
                                          int32_t Sq, int32_t Skv, int32_t D) {
  const size_t base = bsm_splash_bwd_workspace_bytes(B, H, Sq,
                                                     BSM_SCORE_SOFTMAX);
  if (B < 0 || H < 0 || H_kv < 1 || H % H_kv != 0 || Sq < 0 || Skv < 0 || D < 0)
    return base;
  const size_t parts = bsm::bwd_parts(B, H, H_kv, Sq, Skv);
  return parts < 2 ? base
                   : base + parts * 2 * sizeof(float) * static_cast<size_t>(B) *
                                H_kv * Skv * D;
}

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
                          void* stream) {
  return bsm_splash_bwd_mod(q, k, v, out, lse, dout, B, H, H_kv, Sq, Skv, D,
                            info, q_segment_ids, kv_segment_ids, scale, score,
                            nullptr, dq, dk, dv, workspace, workspace_bytes,
                            stream);
}

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
                              size_t workspace_bytes, void* stream) {
  g_last_error.clear();
  if (B < 0 || H < 0 || H_kv < 0 || Sq < 0 || Skv < 0)
    return fail(BSM_ERR_INVALID_ARG, "negative size");
  if (H_kv == 0 ? H != 0 : (H % H_kv) != 0)
    return fail(BSM_ERR_INVALID_ARG, "H must be a multiple of H_kv");
  if (D != 64 && D != 128)
    return fail(BSM_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (Sq > bsm::kMaxSeq || Skv > bsm::kMaxSeq)
    return fail(BSM_ERR_UNSUPPORTED, "sequence length above 262144");
  if (score != BSM_SCORE_SOFTMAX && score != BSM_SCORE_POINTWISE)
    return fail(BSM_ERR_INVALID_ARG, "unknown score path");
  if (!std::isfinite(scale)) return fail(BSM_ERR_INVALID_ARG, "scale not finite");
  bsm::ScoreMod sm_mod;
  if (const bsm_status ms = check_mod(mod, scale, score, &sm_mod); ms != BSM_OK)
    return ms;
  const bool sm = score == BSM_SCORE_SOFTMAX;
  if (q == nullptr || k == nullptr || v == nullptr || dout == nullptr ||
      dq == nullptr || dk == nullptr || dv == nullptr || (sm && out == nullptr))
    return fail(BSM_ERR_INVALID_ARG, "NULL tensor view");
  if (sm && lse == nullptr)
    return fail(BSM_ERR_INVALID_ARG,
                "the softmax backward needs the forward's out and lse");
  if (info == nullptr) return fail(BSM_ERR_INVALID_ARG, "mask info is NULL");
  if (info->Sq != Sq || info->Skv != Skv)
    return fail(BSM_ERR_INVALID_ARG,
                "mask info was built for other sequence lengths");
  const bool seg = (info->flags & BSM_MASK_SEGMENT) != 0;
  if (info->num_tables != (seg ? B : 1))
    return fail(BSM_ERR_INVALID_ARG,
                "mask info was built for another batch size");
  if (!is_block_size(info->block_q) || !is_block_size(info->block_kv) ||
      info->nq != (Sq + info->block_q - 1) / info->block_q ||
      info->nk != (Skv + info->block_kv - 1) / info->block_kv)
    return fail(BSM_ERR_INVALID_ARG, "inconsistent mask info");
  if (seg && (q_segment_ids == nullptr || kv_segment_ids == nullptr))
    return fail(BSM_ERR_INVALID_ARG,
                "BSM_MASK_SEGMENT needs both q and kv segment ids");
  if (!seg && (q_segment_ids != nullptr || kv_segment_ids != nullptr))
    return fail(BSM_ERR_INVALID_ARG,
                "segment ids given without BSM_MASK_SEGMENT");
  if ((info->flags & BSM_MASK_DENSE) &&
      (info->dense_bits == nullptr ||
       info->dense_row_words < (static_cast<int64_t>(Skv) + 31) / 32))
    return fail(BSM_ERR_INVALID_ARG, "mask info lacks its dense mask");
  if (static_cast<int64_t>(B) * H * Sq == 0 &&
      static_cast<int64_t>(B) * H_kv * Skv == 0)
    return BSM_OK;
  const size_t ws_need = bsm_splash_bwd_workspace_bytes(B, H, Sq, score);
  if (ws_need > 0 && (workspace == nullptr || workspace_bytes < ws_need ||
                      !aligned16(workspace)))
    return fail(BSM_ERR_INVALID_ARG,
                "workspace must be >= bsm_splash_bwd_workspace_bytes() bytes, "
                "16-byte aligned");
  // every view: aligned data, positive strides that are multiples of 8
  struct View {
    const bsm_tensor* t;
    int64_t heads, S;
    const char* name;
  };
  const View views[] = {{q, H, Sq, "q"},       {k, H_kv, Skv, "k"},
                        {v, H_kv, Skv, "v"},   {dout, H, Sq, "dout"},
                        {dq, H, Sq, "dq"},     {dk, H_kv, Skv, "dk"},
                        {dv, H_kv, Skv, "dv"}, {sm ? out : dout, H, Sq, "out"}};
  for (const View& w : views) {
    if (w.S == 0) continue;
    if (w.t->data == nullptr || !aligned16(w.t->data))
      return fail(BSM_ERR_INVALID_ARG,
                  std::string(w.name) + " must be non-NULL and 16-byte aligned");
    const int64_t sizes[3] = {B, w.heads, w.S};
    for (int d = 0; d < 3; ++d)
      if (sizes[d] > 1 && (w.t->strides[d] <= 0 || w.t->strides[d] % 8 != 0))
        return fail(BSM_ERR_INVALID_ARG,
                    std::string(w.name) +
                        " strides must be positive multiples of 8");
  }
  int num_sms = 0;
  bsm_status s = check_device(&num_sms);
  if (s != BSM_OK) return s;
  CUtensorMap tq, tk, tv, tdo;
  std::memset(&tq, 0, sizeof(tq));
  std::memset(&tk, 0, sizeof(tk));
  std::memset(&tv, 0, sizeof(tv));
  std::memset(&tdo, 0, sizeof(tdo));
  if (Sq > 0) {
    s = make_map(&tq, q->data, B, H, Sq, D, q->strides, "q");
    if (s != BSM_OK) return s;
    s = make_map(&tdo, dout->data, B, H, Sq, D, dout->strides, "dout");
    if (s != BSM_OK) return s;
  }
  if (Skv > 0) {
    s = make_map(&tk, k->data, B, H_kv, Skv, D, k->strides, "k");
    if (s != BSM_OK) return s;
    s = make_map(&tv, v->data, B, H_kv, Skv, D, v->strides, "v");
    if (s != BSM_OK) return s;
  }
  bsm::BwdParams p;
  p.B = B;
  p.H = H;
  p.Hkv = H_kv;
  p.Sq = Sq;
  p.Skv = Skv;
  p.D = D;
  p.flags = info->flags;
  p.window = info->window;
  p.block_mask = info->block_mask;
  p.mi_nq = info->nq;
  p.mi_nk = info->nk;
  p.bq = info->block_q;
  p.bkv = info->block_kv;
  p.q_seg = q_segment_ids;
  p.kv_seg = kv_segment_ids;
  p.dense = (info->flags & BSM_MASK_DENSE) ? info->dense_bits : nullptr;
  p.dense_words = info->dense_row_words;
  p.score = score;
  p.mod = sm_mod;
  p.scale = scale;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.inv_sq = Sq > 0 ? static_cast<float>(1.0 / static_cast<double>(Sq)) : 0.f;
  p.lse = lse;
  p.delta = static_cast<float*>(workspace);
  p.out = sm ? static_cast<const uint16_t*>(out->data) : nullptr;
  p.o_sb = sm ? out->strides[0] : 0;
  p.o_sh = sm ? out->strides[1] : 0;
  p.o_ss = sm ? out->strides[2] : 0;
  p.dout = static_cast<const uint16_t*>(dout->data);
  p.do_sb = dout->strides[0];
  p.do_sh = dout->strides[1];
  p.do_ss = dout->strides[2];
  p.dq = static_cast<uint16_t*>(dq->data);
  p.dq_sb = dq->strides[0];
  p.dq_sh = dq->strides[1];
  p.dq_ss = dq->strides[2];
  p.dk = static_cast<uint16_t*>(dk->data);
  p.dk_sb = dk->strides[0];
  p.dk_sh = dk->strides[1];
  p.dk_ss = dk->strides[2];
  p.dv = static_cast<uint16_t*>(dv->data);
  p.dv_sb = dv->strides[0];
  p.dv_sh = dv->strides[1];
  p.dv_ss = dv->strides[2];
  p.parts = 1;
  p.part_sums = nullptr;
  if (sm_mod.kind != 0 &&
      workspace_bytes >=
          bsm_splash_bwd_mod_workspace_bytes(B, H, H_kv, Sq, Skv, D)) {
    p.parts = bsm::bwd_parts(B, H, H_kv, Sq, Skv);
    p.part_sums =
        reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + ws_need);
  }
  p.timeout_ns = wait_timeout_ns();
  cudaError_t e = bsm::launch_splash_bwd(p, tq, tk, tv, tdo,
                                         static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "splash_bwd launch");
  return BSM_OK;
}

namespace {
// freq / (2 pi) turns, |freq| <= 64, without the whole ones, in units of 2^-64 and
// off by half of one: the product with 1 / (2 pi) in two f64 (either alone would
// leave 53 bits, which 2^31 positions multiply to an error of 2^-21 and, at a
// frequency of 64, 2^-17).
uint64_t turn_step(double freq) {
  constexpr double kHigh = 0.15915494309189535, kLow = -9.839338337591243e-18;
  const double high = freq * kHigh;
  const double low = std::fma(freq, kHigh, -high) + freq * kLow;
  const double units = std::ldexp(high, 64);  // below 2^68
  const __int128 whole = static_cast<__int128>(units);
  const double rest =
      (units - static_cast<double>(whole)) + std::ldexp(low, 64);
  return static_cast<uint64_t>(whole + std::llrint(rest));
}
}  // namespace

bsm_status bsm_rope_init(bsm_rope* rope, int32_t dim, int32_t interleaved,
                         const double* inv_freq, const int32_t* axis,
                         int32_t axes) {
  g_last_error.clear();
  if (rope == nullptr || inv_freq == nullptr)
    return fail(BSM_ERR_INVALID_ARG, "NULL rope or inv_freq");
  if (dim < 16 || dim > 128 || dim % 16 != 0)
    return fail(BSM_ERR_INVALID_ARG,
                "a rotation's dim must be a multiple of 16 from 16 to 128");
  if (axes < 1 || axes > 4)
    return fail(BSM_ERR_INVALID_ARG, "axes must be from 1 to 4");
  bsm_rope r = {};
  r.dim = dim;
  r.interleaved = interleaved != 0;
  r.axes = axes;
  for (int i = 0; i < dim / 2; ++i) {
    if (!(std::fabs(inv_freq[i]) <= 64.0))
      return fail(BSM_ERR_INVALID_ARG, "inv_freq must be within [-64, 64]");
    const int32_t a = axis != nullptr ? axis[i] : 0;
    if (a < 0 || a >= axes)
      return fail(BSM_ERR_INVALID_ARG, "axis must be within [0, axes)");
    r.axis[i] = static_cast<uint8_t>(a);
    r.step[i] = turn_step(inv_freq[i]);
  }
  *rope = r;
  return BSM_OK;
}

bsm_status bsm_norm_rope(const bsm_tensor* q, const bsm_tensor* k, int32_t B,
                         int32_t H, int32_t H_kv, int32_t S, int32_t D,
                         const bsm_head_norm* norm, const bsm_rope* rope,
                         const bsm_positions* pos, const bsm_tensor* q_out,
                         const bsm_tensor* k_out, void* stream) {
  g_last_error.clear();
  bsm_status s = check_rows(B, H, H_kv, S, D);
  if (s != BSM_OK) return s;
  bsm::NormRopeParams p = {};
  s = check_turn(norm, rope, pos, D, &p.turn);
  if (s != BSM_OK) return s;
  if (q == nullptr || q_out == nullptr ||
      (H_kv > 0 && (k == nullptr || k_out == nullptr)))
    return fail(BSM_ERR_INVALID_ARG, "NULL tensor view");
  if (B == 0 || S == 0 || H + static_cast<int64_t>(H_kv) == 0) return BSM_OK;
  if (H > 0) {
    s = check_view(q, B, H, S, "q");
    if (s == BSM_OK) s = check_view(q_out, B, H, S, "q_out");
    if (s == BSM_OK) s = check_in_place(q, q_out, B, H, S, "q_out");
  }
  if (s == BSM_OK && H_kv > 0) {
    s = check_view(k, B, H_kv, S, "k");
    if (s == BSM_OK) s = check_view(k_out, B, H_kv, S, "k_out");
    if (s == BSM_OK) s = check_in_place(k, k_out, B, H_kv, S, "k_out");
  }
  int num_sms = 0;
  if (s == BSM_OK) s = check_device(&num_sms);
  if (s != BSM_OK) return s;
  p.B = B;
  p.S = S;
  p.D = D;
  p.heads[0] = H;
  p.heads[1] = H_kv;
  p.x[0] = row_view(q);
  p.x[1] = row_view(k);
  p.out[0] = row_view(q_out);
  p.out[1] = row_view(k_out);
  const cudaError_t e =
      bsm::launch_norm_rope(p, num_sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "norm_rope launch");
  return BSM_OK;
}

size_t bsm_norm_rope_bwd_workspace_bytes(void) {
  return static_cast<size_t>(bsm::kNormRopeMaxBlocks) * 128 * sizeof(float);
}

bsm_status bsm_norm_rope_bwd(const bsm_tensor* gq, const bsm_tensor* gk,
                             const bsm_tensor* q, const bsm_tensor* k,
                             int32_t B, int32_t H, int32_t H_kv, int32_t S,
                             int32_t D, const bsm_head_norm* norm,
                             const bsm_rope* rope, const bsm_positions* pos,
                             const bsm_tensor* dq, const bsm_tensor* dk,
                             float* dq_weight, float* dk_weight,
                             void* workspace, size_t workspace_bytes,
                             void* stream) {
  g_last_error.clear();
  bsm_status s = check_rows(B, H, H_kv, S, D);
  if (s != BSM_OK) return s;
  bsm::NormRopeParams p = {};
  s = check_turn(norm, rope, pos, D, &p.turn);
  if (s != BSM_OK) return s;
  const bool keys = H_kv > 0;
  if (gq == nullptr || dq == nullptr || (keys && (gk == nullptr || dk == nullptr)) ||
      (norm != nullptr && (q == nullptr || (keys && k == nullptr))))
    return fail(BSM_ERR_INVALID_ARG, "NULL tensor view");
  const bool dw = dq_weight != nullptr || dk_weight != nullptr;
  if (dw && norm == nullptr)
    return fail(BSM_ERR_INVALID_ARG, "weight gradients without a norm");
  if (((reinterpret_cast<uintptr_t>(dq_weight) |
        reinterpret_cast<uintptr_t>(dk_weight)) & 3u) != 0)
    return fail(BSM_ERR_INVALID_ARG, "weight gradients must be 4-byte aligned");
  if (dw && (workspace == nullptr || !aligned16(workspace) ||
             workspace_bytes < bsm_norm_rope_bwd_workspace_bytes()))
    return fail(BSM_ERR_INVALID_ARG,
                "workspace must be >= bsm_norm_rope_bwd_workspace_bytes() "
                "bytes, 16-byte aligned");
  const bool rows = B > 0 && S > 0 && H + static_cast<int64_t>(H_kv) > 0;
  if (!rows && !dw) return BSM_OK;
  const bsm_tensor* views[2][3] = {{gq, dq, q}, {gk, dk, k}};
  static const char* const names[2][3] = {{"gq", "dq", "q"}, {"gk", "dk", "k"}};
  for (int i = 0; i < 2 && rows; ++i)
    for (int j = 0; j < (norm != nullptr ? 3 : 2) && (i ? H_kv : H) > 0; ++j)
      if (s == BSM_OK)
        s = check_view(views[i][j], B, i ? H_kv : H, S, names[i][j]);
  for (int i = 0; i < 2 && rows && s == BSM_OK; ++i)
    if ((i ? H_kv : H) > 0)
      s = check_in_place(views[i][0], views[i][1], B, i ? H_kv : H, S,
                         names[i][1]);
  int num_sms = 0;
  if (s == BSM_OK) s = check_device(&num_sms);
  if (s != BSM_OK) return s;
  p.B = B;
  p.S = S;
  p.D = D;
  p.heads[0] = H;
  p.heads[1] = H_kv;
  for (int i = 0; i < 2; ++i) {
    p.g[i] = row_view(views[i][0]);
    p.out[i] = row_view(views[i][1]);
    p.x[i] = row_view(views[i][2]);
  }
  p.dw[0] = dq_weight;
  p.dw[1] = dk_weight;
  p.partial = static_cast<float*>(workspace);
  const cudaError_t e =
      bsm::launch_norm_rope_bwd(p, num_sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "norm_rope_bwd launch");
  return BSM_OK;
}

namespace {
// bsm_kv_append, and bsm_kv_append_rope with `turn`.
bsm_status append(const bsm_kv_cache* cache, const int32_t* page_table,
                  int64_t table_stride, int32_t max_pages, const int32_t* lens,
                  const int32_t* n_new, const bsm_tensor* k_new,
                  const bsm_tensor* v_new, int32_t B, int32_t T,
                  const bsm::TurnParams* turn, void* stream) {
  bsm_status s = check_cache(cache, table_stride, max_pages, B, T);
  if (s != BSM_OK) return s;
  if (k_new == nullptr || v_new == nullptr)
    return fail(BSM_ERR_INVALID_ARG, "NULL tensor view");
  if (B == 0 || T == 0 || cache->H_kv == 0) return BSM_OK;
  s = check_cache_memory(cache, page_table, max_pages, lens);
  if (s != BSM_OK) return s;
  if ((reinterpret_cast<uintptr_t>(n_new) & 3u) != 0)
    return fail(BSM_ERR_INVALID_ARG, "n_new must be 4-byte aligned");
  s = check_view(k_new, B, cache->H_kv, T, "k_new");
  if (s == BSM_OK) s = check_view(v_new, B, cache->H_kv, T, "v_new");
  if (s == BSM_OK) s = check_device(nullptr);
  if (s != BSM_OK) return s;
  bsm::AppendParams p;
  p.k = static_cast<uint8_t*>(cache->k);
  p.v = static_cast<uint8_t*>(cache->v);
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.num_pages = cache->num_pages;
  p.H_kv = cache->H_kv;
  p.page_size = cache->page_size;
  p.D = cache->D;
  p.table = page_table;
  p.table_stride = table_stride;
  p.max_pages = max_pages;
  p.lens = lens;
  p.n_new = n_new;
  p.B = B;
  p.T = T;
  p.k_new = static_cast<const uint16_t*>(k_new->data);
  p.v_new = static_cast<const uint16_t*>(v_new->data);
  p.k_sb = k_new->strides[0];
  p.k_sh = k_new->strides[1];
  p.k_ss = k_new->strides[2];
  p.v_sb = v_new->strides[0];
  p.v_sh = v_new->strides[1];
  p.v_ss = v_new->strides[2];
  const auto st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = turn != nullptr
                            ? bsm::launch_kv_append_rope(p, *turn, st)
                            : bsm::launch_kv_append(p, st);
  if (e != cudaSuccess) return cuda_fail(e, "kv_append launch");
  return BSM_OK;
}
}  // namespace

bsm_status bsm_kv_append(const bsm_kv_cache* cache, const int32_t* page_table,
                         int64_t table_stride, int32_t max_pages,
                         const int32_t* lens, const int32_t* n_new,
                         const bsm_tensor* k_new, const bsm_tensor* v_new,
                         int32_t B, int32_t T, void* stream) {
  g_last_error.clear();
  return append(cache, page_table, table_stride, max_pages, lens, n_new, k_new,
                v_new, B, T, nullptr, stream);
}

bsm_status bsm_kv_append_rope(const bsm_kv_cache* cache,
                              const int32_t* page_table, int64_t table_stride,
                              int32_t max_pages, const int32_t* lens,
                              const int32_t* n_new, const bsm_tensor* k_new,
                              const bsm_tensor* v_new, int32_t B, int32_t T,
                              const bsm_head_norm* norm, const bsm_rope* rope,
                              const bsm_positions* pos, void* stream) {
  g_last_error.clear();
  if (cache == nullptr) return fail(BSM_ERR_INVALID_ARG, "cache is NULL");
  bsm::TurnParams turn;
  const bsm_status s = check_turn(norm, rope, pos, cache->D, &turn);
  if (s != BSM_OK) return s;
  return append(cache, page_table, table_stride, max_pages, lens, n_new, k_new,
                v_new, B, T, &turn, stream);
}

size_t bsm_paged_attention_workspace_bytes(void) {
  return bsm::kPaWorkspaceBytes;
}

namespace {
// What bsm_paged_attention_tree has beside bsm_paged_attention.
struct Drafts {
  const int32_t* n_new;
  const uint32_t* tree;
  int64_t sb, st;
};

bsm_status paged(const bsm_tensor* q, const bsm_kv_cache* cache,
                 const int32_t* page_table, int64_t table_stride,
                 int32_t max_pages, const int32_t* lens, int32_t B, int32_t H,
                 int32_t T, float scale, int32_t window,
                 const bsm_score_mod* mod, const Drafts* drafts,
                 const bsm_tensor* out, float* lse, void* workspace,
                 size_t workspace_bytes, void* stream) {
  bsm_status s = check_cache(cache, table_stride, max_pages, B, T);
  if (s != BSM_OK) return s;
  if (H < 0 || (cache->H_kv == 0 ? H != 0 : H % cache->H_kv != 0))
    return fail(BSM_ERR_INVALID_ARG, "H must be a multiple of H_kv");
  if (!std::isfinite(scale)) return fail(BSM_ERR_INVALID_ARG, "scale not finite");
  if (window < 0) return fail(BSM_ERR_INVALID_ARG, "window must be >= 0");
  if (q == nullptr || out == nullptr)
    return fail(BSM_ERR_INVALID_ARG, "NULL tensor view");
  bsm::PagedParams p;
  s = check_mod(mod, scale, BSM_SCORE_SOFTMAX, &p.mod);
  if (s != BSM_OK) return s;
  p.scale_x = p.mod.kind & bsm::kModCap
                  ? p.mod.cap_e
                  : static_cast<float>(static_cast<double>(scale) *
                                       1.4426950408889634);
  if (B == 0 || T == 0 || H == 0) return BSM_OK;
  s = check_cache_memory(cache, page_table, max_pages, lens);
  if (s == BSM_OK) s = check_view(q, B, H, T, "q");
  if (s == BSM_OK) s = check_view(out, B, H, T, "out");
  if (s != BSM_OK) return s;
  const int64_t rows = static_cast<int64_t>(H / cache->H_kv) * T;
  if (rows * cache->H_kv > 8 * 65535)
    return fail(BSM_ERR_UNSUPPORTED, "too many query rows");
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0)
    return fail(BSM_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  const bool tc = drafts != nullptr && bsm::tree_tiles(rows) > 0;
  const size_t need = drafts != nullptr
                          ? bsm::tree_workspace_bytes(rows, cache->D)
                          : bsm::kPaWorkspaceBytes;
  if (workspace == nullptr || workspace_bytes < need || !aligned16(workspace))
    return fail(BSM_ERR_INVALID_ARG,
                std::string("workspace must be >= bsm_paged_attention") +
                    (drafts != nullptr ? "_tree" : "") +
                    "_workspace_bytes() bytes, 16-byte aligned");
  int num_sms = 0;
  s = check_device(&num_sms);
  if (s != BSM_OK) return s;
  if (num_sms > (tc ? bsm::kTreeMaxSms : bsm::kPaMaxSms))
    return fail(BSM_ERR_UNSUPPORTED, "too many SMs");
  p.parts = static_cast<float*>(workspace);
  p.k = static_cast<const uint8_t*>(cache->k);
  p.v = static_cast<const uint8_t*>(cache->v);
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.num_pages = cache->num_pages;
  p.H_kv = cache->H_kv;
  p.page_size = cache->page_size;
  for (p.page_shift = 4; (1 << p.page_shift) < p.page_size;) ++p.page_shift;
  p.D = cache->D;
  p.table = page_table;
  p.table_stride = table_stride;
  p.max_pages = max_pages;
  p.lens = lens;
  p.B = B;
  p.H = H;
  p.T = T;
  p.window = window < (1 << 30) ? window : 1 << 30;  // no sequence is longer
  p.q = static_cast<const uint16_t*>(q->data);
  p.q_sb = q->strides[0];
  p.q_sh = q->strides[1];
  p.q_ss = q->strides[2];
  p.out = static_cast<uint16_t*>(out->data);
  p.o_sb = out->strides[0];
  p.o_sh = out->strides[1];
  p.o_ss = out->strides[2];
  p.lse = lse;
  const auto st = static_cast<cudaStream_t>(stream);
  p.n_new = nullptr;
  p.tree = nullptr;
  p.tree_sb = p.tree_st = 0;
  if (drafts != nullptr) {
    p.n_new = drafts->n_new;
    p.tree = drafts->tree;
    p.tree_sb = drafts->sb;
    p.tree_st = drafts->st;
  }
  const cudaError_t e =
      tc ? bsm::launch_tree_tc(p, num_sms, wait_timeout_ns(), st)
      : drafts != nullptr ? bsm::launch_paged_tree(p, num_sms, st)
                          : bsm::launch_paged_attention(p, num_sms, st);
  if (e != cudaSuccess) return cuda_fail(e, "paged_attention launch");
  return BSM_OK;
}
}  // namespace

bsm_status bsm_paged_attention(const bsm_tensor* q, const bsm_kv_cache* cache,
                               const int32_t* page_table, int64_t table_stride,
                               int32_t max_pages, const int32_t* lens,
                               int32_t B, int32_t H, int32_t T, float scale,
                               int32_t window, const bsm_score_mod* mod,
                               const bsm_tensor* out, float* lse,
                               void* workspace, size_t workspace_bytes,
                               void* stream) {
  g_last_error.clear();
  return paged(q, cache, page_table, table_stride, max_pages, lens, B, H, T,
               scale, window, mod, nullptr, out, lse, workspace,
               workspace_bytes, stream);
}

size_t bsm_paged_attention_tree_workspace_bytes(int32_t H, int32_t H_kv,
                                                int32_t T, int32_t D) {
  if (H < 0 || H_kv <= 0 || T < 0) return 0;
  return bsm::tree_workspace_bytes(static_cast<int64_t>(H / H_kv) * T, D);
}

bsm_status bsm_paged_attention_tree(
    const bsm_tensor* q, const bsm_kv_cache* cache, const int32_t* page_table,
    int64_t table_stride, int32_t max_pages, const int32_t* lens,
    const int32_t* n_new, const uint32_t* tree, int64_t tree_stride_b,
    int64_t tree_stride_t, int32_t B, int32_t H, int32_t T, float scale,
    int32_t window, const bsm_score_mod* mod, const bsm_tensor* out,
    float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  g_last_error.clear();
  if (T > 1024 && tree != nullptr)
    return fail(BSM_ERR_UNSUPPORTED, "more than 1024 drafts in a tree");
  if (((reinterpret_cast<uintptr_t>(n_new) |
        reinterpret_cast<uintptr_t>(tree)) & 3u) != 0)
    return fail(BSM_ERR_INVALID_ARG, "n_new and tree must be 4-byte aligned");
  if (tree_stride_b < 0 || tree_stride_t < 0)
    return fail(BSM_ERR_INVALID_ARG, "tree strides must be >= 0");
  const Drafts d = {n_new, tree, tree_stride_b, tree_stride_t};
  return paged(q, cache, page_table, table_stride, max_pages, lens, B, H, T,
               scale, window, mod, &d, out, lse, workspace, workspace_bytes,
               stream);
}

bsm_status bsm_device_status(void* stream, int32_t* detail) {
  g_last_error.clear();
  int32_t rec[4] = {0, 0, 0, 0}, brec[4] = {0, 0, 0, 0};
  int32_t crec[4] = {0, 0, 0, 0}, trec[4] = {0, 0, 0, 0};
  cudaError_t e = bsm::read_device_error(rec, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "device status");
  e = bsm::read_bwd_error(brec);
  if (e != cudaSuccess) return cuda_fail(e, "device status");
  if (rec[0] == 0 && brec[0] != 0) std::memcpy(rec, brec, sizeof(rec));
  if (rec[0] == 0) e = bsm::read_tree_error(1, trec);
  if (e != cudaSuccess) return cuda_fail(e, "device status");
  if (trec[0] != 0) std::memcpy(rec, trec, sizeof(rec));
  // read, and so cleared, only where no timeout is reported before it: else
  // the next call reports it
  if (rec[0] == 0) e = bsm::read_cache_error(crec);
  if (e != cudaSuccess) return cuda_fail(e, "device status");
  if (rec[0] == 0 && crec[0] == 0) e = bsm::read_tree_error(2, crec);
  if (e != cudaSuccess) return cuda_fail(e, "device status");
  if (crec[0] != 0) {
    if (detail != nullptr) std::memcpy(detail, crec, sizeof(crec));
    return fail(BSM_ERR_INVALID_ARG,
                (crec[2] < 0 ? "a length is out of range (sequence "
                             : "a page is out of range (sequence ") +
                    std::to_string(crec[1]) +
                    (crec[2] < 0 ? "" : ", slot " + std::to_string(crec[2])) +
                    ", value " + std::to_string(crec[3]) + ")");
  }
  if (detail != nullptr) std::memcpy(detail, rec, sizeof(rec));
  if (rec[0] != 0)
    return fail(BSM_ERR_DEVICE_TIMEOUT,
                "a kernel gave up on a bounded wait (block " +
                    std::to_string(rec[1]) + ", role " + std::to_string(rec[2]) +
                    ", phase " + std::to_string(rec[3]) + ")");
  return BSM_OK;
}

namespace {
bsm_status selftest(cudaError_t (*launch)(uint64_t, cudaStream_t),
                    int64_t timeout_ns, void* stream) {
  g_last_error.clear();
  if (timeout_ns < 1000 || timeout_ns > 10000000000LL)
    return fail(BSM_ERR_INVALID_ARG, "timeout_ns must be in [1e3, 1e10]");
  bsm_status s = check_device(nullptr);
  if (s != BSM_OK) return s;
  const cudaError_t e = launch(static_cast<uint64_t>(timeout_ns),
                               static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "self-test launch");
  return BSM_OK;
}
}  // namespace

bsm_status bsm_selftest_wait_timeout(int64_t timeout_ns, void* stream) {
  return selftest(bsm::launch_wait_selftest, timeout_ns, stream);
}

bsm_status bsm_selftest_tree_timeout(int64_t timeout_ns, void* stream) {
  return selftest(bsm::launch_tree_selftest, timeout_ns, stream);
}

bsm_status bsm_debug_set_trace(void* buffer, size_t bytes) {
  g_last_error.clear();
  if (buffer != nullptr && (reinterpret_cast<uintptr_t>(buffer) & 15u) != 0)
    return fail(BSM_ERR_INVALID_ARG, "trace buffer must be 16-byte aligned");
  std::lock_guard<std::mutex> lk(g_trace_mu);
  g_trace_buf = bytes >= 32 ? buffer : nullptr;
  g_trace_bytes = g_trace_buf != nullptr ? bytes : 0;
  return BSM_OK;
}

int32_t bsm_debug_fwd_grid(int32_t B, int32_t H, int32_t Sq) {
  int num_sms = 0;
  if (check_device(&num_sms) != BSM_OK) return -1;
  bsm::FwdParams p;
  p.num_units = B * H * ((Sq + bsm::kUnitRows - 1) / bsm::kUnitRows);
  return bsm::fwd_grid_size(p, num_sms);
}

const char* bsm_last_error(void) { return g_last_error.c_str(); }

int32_t bsm_version(void) { return 302; }

}  // extern "C"
