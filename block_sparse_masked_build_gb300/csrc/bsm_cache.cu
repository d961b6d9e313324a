// Paged key/value cache in 8-bit floating point for sm_103a (GB300): writing
// new tokens into it, and attention of one or a few query tokens per
// sequence over it.
//
// A page holds `page_size` consecutive tokens of one sequence for every
// key/value head: e4m3 codes [H_kv][page_size][D], and one f32 scale per
// (page, head); element = code * scale.
//
// Append.  For a page and head, amax over the finite magnitudes of the new
// tokens gives the smallest e in [-40, 40] with amax <= 448 * 2^e (448 is the
// largest e4m3 value).  A page that holds tokens already keeps the larger of
// its scale and 2^e; where its scale grows the old codes are rounded again.
// Power-of-two scales make every quotient exact, so the only roundings are
// the ones to e4m3 itself (half a step: 2^-4 of a normal value), and rounding
// an old code again loses only what falls below the new smallest step.
//
// Attention.  For query row r = (head of the group, token t) at position
// pos = len - T + t and the keys j it sees (j <= pos, and pos - j < window):
//     x_j = scale q.k_j,  z_j = cap tanh(x_j / cap) - slope (pos - j),
//     out = sum_j e^(z_j - m) v_j / sum_j e^(z_j - m)
// with the running maximum m of a one-pass softmax, in f32.
#include <cstdint>

#include "bsm_internal.h"
#include "bsm_paged.cuh"
#include "bsm_ptx.cuh"
#include "bsm_rope.cuh"

namespace bsm {

// Error record: [0] code (2 = a page table or length out of range), [1]
// sequence, [2] page slot, [3] the value found.
__device__ int g_cache_error[4];

namespace {

__device__ __forceinline__ void record_bad_index(int b, int slot, int value) {
  if (atomicCAS(&g_cache_error[0], 0, 2) == 0) {
    g_cache_error[1] = b;
    g_cache_error[2] = slot;
    g_cache_error[3] = value;
  }
}

__device__ __forceinline__ float f16_lo(uint32_t w) {
  float f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}"
      : "=f"(f)
      : "r"(w));
  return f;
}
__device__ __forceinline__ float f16_hi(uint32_t w) {
  float f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, h;\n\t}"
      : "=f"(f)
      : "r"(w));
  return f;
}
// Four f32 as e4m3 codes, nearest even, magnitudes above 448 to 448, NaN to
// NaN.
__device__ __forceinline__ uint32_t f32x4_to_e4m3(float a, float b, float c,
                                                  float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// ------------------------------------------------------------------ append

constexpr int kAppendThreads = 128;

// 2^e with e the smallest integer in [-40, 40] for which amax <= 448 * 2^e;
// amax >= 0 is finite.  448 = 1.75 * 2^8.
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 127 - 8 +
          ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = min(max(e, -40), 40);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// One CTA writes the new tokens of one page of one head's keys or values.
// A thread owns NCH pieces of 8 elements (16 bytes in, 8 out) of the page and
// keeps its new ones in registers between the maximum and the rounding, so
// new elements are read once; old codes are read only where the scale grows.
// Bound by memory for prompts and by latency for single tokens (a load, a
// block maximum, a store).
template <int NCH>
__global__ void __launch_bounds__(kAppendThreads, NCH <= 8 ? 8 : 4)
    kv_append_kernel(const AppendParams p) {
  const int b = blockIdx.z;
  const int h = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  int len = p.lens[b];
  int n = p.n_new != nullptr ? p.n_new[b] : p.T;
  const int capacity = p.max_pages * p.page_size;
  const bool bad = len < 0 || n < 0 || n > p.T || len > capacity - n;
  if (bad) {  // nothing of such a sequence is written
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0)
      record_bad_index(b, -1, len < 0 || len > capacity ? len : n);
    return;
  }
  const int slot = len / p.page_size + blockIdx.x;
  const int tok0 = slot * p.page_size;
  const int lo = max(len, tok0) - tok0;  // new tokens [lo, hi) of the page
  const int hi = min(len + n - tok0, p.page_size);
  if (lo >= hi) return;
  // the new elements and, beside them, the page: neither waits for the other
  const int pid = p.table[static_cast<int64_t>(b) * p.table_stride + slot];
  const int per_shift = p.D == 128 ? 4 : 3;  // log2 of the pieces per token
  const uint16_t* src = is_v ? p.v_new : p.k_new;
  const int64_t sb = is_v ? p.v_sb : p.k_sb, sh = is_v ? p.v_sh : p.k_sh,
                ss = is_v ? p.v_ss : p.k_ss;
  src += b * sb + h * sh;
  uint4 x[NCH];
  uint32_t top = 0;  // two running maxima, one per half word
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = threadIdx.x + i * kAppendThreads;
    const int tok = c >> per_shift;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tok >= lo && tok < hi)
      x[i] = *reinterpret_cast<const uint4*>(
          src + (tok0 + tok - len) * ss + (c & ((1 << per_shift) - 1)) * 8);
  }
  if (pid < 0 || pid >= p.num_pages) {
    if (threadIdx.x == 0) record_bad_index(b, slot, pid);
    return;
  }
  const int64_t block = static_cast<int64_t>(pid) * p.H_kv + h;
  uint8_t* dst = (is_v ? p.v : p.k) + block * p.page_size * p.D;
  float* scale_at = (is_v ? p.v_scale : p.k_scale) + block;
  const float was = lo > 0 ? *scale_at : 0.f;
  // the largest |bits| (bf16 magnitudes compare as integers)
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) top = max_u16x2(top, w[j] & 0x7fff7fffu);
  }
  __shared__ uint32_t warp_top[2][kAppendThreads / 32];
  auto block_max = [&](int which) {
    top = max(top & 0xffffu, top >> 16);
    top = __reduce_max_sync(0xffffffffu, top);
    if (threadIdx.x % 32 == 0) warp_top[which][threadIdx.x / 32] = top;
    __syncthreads();  // (the first: every thread has read the old scale)
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w)
      top = max(top, warp_top[which][w]);
  };
  block_max(0);
  if (top >= 0x7f80u) {  // an infinity or NaN: once more over the finite ones
    top = 0;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a = w[j] & 0x7fff7fffu;
        top = max_u16x2(top, a & __vcmpltu2(a, 0x7f807f80u));
      }
    }
    block_max(1);
  }
  const float want = block_scale(__uint_as_float(top << 16));
  const float scale = lo > 0 ? fmaxf(was, want) : want;
  const float inv = __frcp_rn(scale);  // exact: a power of two from this kernel
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = threadIdx.x + i * kAppendThreads;
    const int tok = c >> per_shift;
    if (tok >= lo && tok < hi) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint2 q;
      q.x = f32x4_to_e4m3(bf16_lo(w[0]) * inv, bf16_hi(w[0]) * inv,
                          bf16_lo(w[1]) * inv, bf16_hi(w[1]) * inv);
      q.y = f32x4_to_e4m3(bf16_lo(w[2]) * inv, bf16_hi(w[2]) * inv,
                          bf16_lo(w[3]) * inv, bf16_hi(w[3]) * inv);
      *reinterpret_cast<uint2*>(dst + c * 8) = q;
    } else if (tok < lo && scale > was) {
      const float ratio = was * inv;
      uint2 q = *reinterpret_cast<const uint2*>(dst + c * 8);
      uint32_t r[2] = {q.x, q.y};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t f0 = e4m3x2_to_f16x2(r[j]), f1 = e4m3x2_to_f16x2_hi(r[j]);
        r[j] = f32x4_to_e4m3(f16_lo(f0) * ratio, f16_hi(f0) * ratio,
                             f16_lo(f1) * ratio, f16_hi(f1) * ratio);
      }
      *reinterpret_cast<uint2*>(dst + c * 8) = make_uint2(r[0], r[1]);
    }
  }
  if (threadIdx.x == 0) *scale_at = scale;
}

// The same with the keys normalised and rotated first, in f32 from the load to
// the rounding to e4m3.  A token's row lies in D / 16 neighbouring lanes,
// sixteen elements each, the two elements of a rotated pair in one lane: the
// only exchange is the norm's sum.  8 prompts of 500-2048 tokens, 8 heads of 128:
// 27-35 us (eight elements a lane, partners exchanged and every angle worked out
// twice, took 7 us more at the same angles' cost); one token for each of 64
// sequences 10, 20-48 drafts for 16 of them 9.  The prompts' 63 MB would take 9
// us: bound by instructions, which issue in 67 % of the cycles, half of them the
// angles'.  Working these out once for two or four heads of a page (35-38 us: a
// block's heads then wait one after another) or ahead of the elements into
// shared memory (32) gained nothing, nor did blocks of 512 threads (36).
constexpr int kTurnThreads = 256;

template <int D, int NCH>
__global__ void __launch_bounds__(kTurnThreads, NCH > 2 ? 2 : 4)
    kv_append_rope_kernel(const AppendParams p,
                          const __grid_constant__ TurnParams turn) {
  constexpr int kPer = D / 16;  // lanes of a token's row
  const int b = blockIdx.z;
  const int h = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const int len = p.lens[b];
  const int n = p.n_new != nullptr ? p.n_new[b] : p.T;
  const int capacity = p.max_pages * p.page_size;
  if (len < 0 || n < 0 || n > p.T || len > capacity - n) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0)
      record_bad_index(b, -1, len < 0 || len > capacity ? len : n);
    return;  // nothing of such a sequence is written
  }
  const int slot = len / p.page_size + blockIdx.x;
  const int tok0 = slot * p.page_size;
  const int lo = max(len, tok0) - tok0;  // new tokens [lo, hi) of the page
  const int hi = min(len + n - tok0, p.page_size);
  if (lo >= hi) return;
  const int pid = p.table[static_cast<int64_t>(b) * p.table_stride + slot];
  const bsm_rope& rope = turn.rope;
  const bool pairs = rope.interleaved != 0;
  const int row0 = threadIdx.x / kPer;
  constexpr int kRows = kTurnThreads / kPer;  // rows of one step
  const LanePart part =
      lane_part(threadIdx.x % kPer, rope.dim, !pairs);
  const uint16_t* src = is_v ? p.v_new : p.k_new;
  const int64_t sb = is_v ? p.v_sb : p.k_sb, sh = is_v ? p.v_sh : p.k_sh,
                ss = is_v ? p.v_ss : p.k_ss;
  src += b * sb + h * sh;
  uint4 raw[NCH][2];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int tok = row0 + i * kRows;
    raw[i][0] = raw[i][1] = make_uint4(0u, 0u, 0u, 0u);
    if (tok >= lo && tok < hi) {
      const uint16_t* row = src + (tok0 + tok - len) * ss;
      raw[i][0] = *reinterpret_cast<const uint4*>(row + part.at0);
      raw[i][1] = *reinterpret_cast<const uint4*>(row + part.at1);
    }
  }
  // steps and weights in shared memory while the elements are on their way
  // (read from the parameters, where lanes of a warp want different words, the
  // steps cost 11 us of 49 on those prompts)
  __shared__ __align__(16) uint64_t steps[64];
  __shared__ __align__(16) float weights[D];
  if (!is_v) {
    if (threadIdx.x < 64) steps[threadIdx.x] = rope.step[threadIdx.x];
    if (turn.norm && threadIdx.x >= 128 && threadIdx.x < 128 + D / 8)
      weights_of(turn.k_weight, turn.weights_bf16, (threadIdx.x - 128) * 8,
                 weights + (threadIdx.x - 128) * 8);
  }
  if (pid < 0 || pid >= p.num_pages) {
    if (threadIdx.x == 0) record_bad_index(b, slot, pid);
    return;
  }
  const int64_t block = static_cast<int64_t>(pid) * p.H_kv + h;
  uint8_t* dst = (is_v ? p.v : p.k) + block * p.page_size * p.D;
  float* scale_at = (is_v ? p.v_scale : p.k_scale) + block;
  const float was = lo > 0 ? *scale_at : 0.f;
  __syncthreads();
  float x[NCH][16];
  float top = 0.f;  // the largest finite magnitude
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    unpack_bf16x8(raw[i][0], x[i]);
    unpack_bf16x8(raw[i][1], x[i] + 8);
    const int tok = row0 + i * kRows;
    const bool fresh = tok >= lo && tok < hi;
    // (whole warps: the lanes add up their squares)
    if (!is_v && __any_sync(0xffffffffu, fresh)) {
      if (turn.norm) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) sum = fmaf(x[i][e], x[i][e], sum);
#pragma unroll
        for (int d = 1; d < kPer; d *= 2)
          sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const float r = rsqrtf(fmaf(sum, 1.f / D, turn.eps));
#pragma unroll
        for (int e = 0; e < 16; ++e)
          x[i][e] *= r;  // (and then the weight, as in norm_rope)
        if (turn.k_weight != nullptr) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            x[i][e] *= weights[(e < 8 ? part.at0 : part.at1 - 8) + e];
        }
      }
      if (part.freq >= 0 && fresh) {
        const int t = tok0 + tok - len;
        const int32_t* pos =
            turn.pos != nullptr
                ? turn.pos + b * turn.pos_sb + t * turn.pos_ss
                : nullptr;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float c, s;
          turns_of<1>(rope, steps + part.freq + e, part.freq + e, pos,
                      turn.pos_sa, tok0 + tok, &c, &s);
          if (pairs) {
            const float u = x[i][2 * e], v = x[i][2 * e + 1];
            x[i][2 * e] = u * c - v * s;
            x[i][2 * e + 1] = v * c + u * s;
          } else {
            const float u = x[i][e], v = x[i][8 + e];
            x[i][e] = u * c - v * s;
            x[i][8 + e] = v * c + u * s;
          }
        }
      }
    }
    if (fresh) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float a = fabsf(x[i][e]);
        top = fmaxf(top, a < __int_as_float(0x7f800000) ? a : 0.f);
      }
    }
  }
  __shared__ uint32_t warp_top[kTurnThreads / 32];
  const uint32_t mine =
      __reduce_max_sync(0xffffffffu, __float_as_uint(top));
  if (threadIdx.x % 32 == 0) warp_top[threadIdx.x / 32] = mine;
  __syncthreads();  // (and every thread has read the old scale)
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < kTurnThreads / 32; ++i) most = max(most, warp_top[i]);
  const float want = block_scale(__uint_as_float(most));
  const float scale = lo > 0 ? fmaxf(was, want) : want;
  const float inv = __frcp_rn(scale);  // exact: a power of two from this kernel
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int tok = row0 + i * kRows;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float* y = x[i] + 8 * k;
      uint2* at =
          reinterpret_cast<uint2*>(dst + tok * D + (k ? part.at1 : part.at0));
      if (tok >= lo && tok < hi) {
        *at = make_uint2(
            f32x4_to_e4m3(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
            f32x4_to_e4m3(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
      } else if (tok < lo && scale > was) {
        const float ratio = was * inv;
        const uint2 q = *at;
        uint32_t r[2] = {q.x, q.y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t f0 = e4m3x2_to_f16x2(r[j]),
                         f1 = e4m3x2_to_f16x2_hi(r[j]);
          r[j] = f32x4_to_e4m3(f16_lo(f0) * ratio, f16_hi(f0) * ratio,
                               f16_lo(f1) * ratio, f16_hi(f1) * ratio);
        }
        *at = make_uint2(r[0], r[1]);
      }
    }
  }
  if (threadIdx.x == 0) *scale_at = scale;
}

// --------------------------------------------------------------- attention

constexpr int kPaWarps = 4;
constexpr int kPaThreads = 32 * kPaWarps;
// The deal (see PaPlan): a unit is a group of 16 tokens for each warp.
template <bool TREE>
struct PaDeal {
  static constexpr bool kTree = TREE;
  static constexpr int kUnit = kPaWarps, kRunCost = 4, kLeast = 2;
};
constexpr float kPUp = 512.f; // p's factor before it becomes f16

template <int D, int NT>
struct PaCfg {
  // groups of a warp's ring, one of them being read: what three CTAs of an SM
  // have room for at D = 128.  (At 64, where six fit, they were no faster: 94
  // us on 64 sequences of 300-12000 tokens, with four 91.)
  static constexpr int kPaStages = 4;
  static constexpr int kHalf = kPaGroup * D;  // bytes of a group's K or V
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kOffScale = kPaWarps * kPaStages * kStage;
  // two row tiles: their query fragments
  static constexpr int kOffQ = kOffScale + kPaWarps * kPaStages * 8;
  static constexpr int kSmem = kOffQ + (NT > 1 ? NT * D / 32 * 512 : 0);
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src,
                                           bool keep) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(src), "r"(keep ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src,
                                          bool keep) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst),
               "l"(src), "r"(keep ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(a)
               : "memory");
  return r;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y,
                                       uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x),
               "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
               : "=r"(r.x), "=r"(r.y)
               : "r"(a)
               : "memory");
  return r;
}
// d += a b: a 16 x 16 f16 (rows = tokens or dims), b 16 x 8 f16, d f32.
__device__ __forceinline__ void mma16816(float d[4], uint32_t a0, uint32_t a1,
                                         uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;"
               : "=r"(r)
               : "r"(x));
  return r;
}

// Byte offset of 16-byte piece c of token row tr within a group's K or V.
// D = 128: one 128-byte line per token, pieces exchanged by an xor with
// (tr & 1) * 4 + (tr >> 1 & 3); D = 64: two tokens per line.  With the
// pieces' assignment to lanes below, every warp-wide read and write touches
// each bank once.
template <int D>
__device__ __forceinline__ uint32_t piece_at(int tr, int c) {
  if (D == 128)
    return tr * 128 + ((c ^ (((tr & 1) << 2) | ((tr >> 1) & 3))) << 4);
  return (tr >> 1) * 128 +
         (((((tr & 1) << 2) | c) ^ (((tr >> 1) & 3) << 1)) << 4);
}

// Starts the copy of one group of 16 tokens from `tok` on into a stage (whole
// warp).  Tokens outside [lo, hi) and pages out of range (pid < 0) are filled
// with zeros; a scale of zero marks the latter.
template <int D>
__device__ __forceinline__ void load_group(const PagedParams& p,
                                           uint32_t stage, uint32_t scale_at,
                                           int head, int pid, int tok, int lo,
                                           int hi) {
  const int lane = threadIdx.x % 32;
  const bool ok = pid >= 0;
  const int64_t block = static_cast<int64_t>(ok ? pid : 0) * p.H_kv + head;
  const int64_t off =
      ((block << p.page_shift) + (tok & (p.page_size - 1))) * D + lane * 16;
  constexpr int kPieces = kPaGroup * D / 16;
  // piece i * 32 + lane lies at first + i * 512 but for the exchange, which
  // differs in one bit between odd and even i (D = 128).  (Groups that end
  // inside take the other branch: with the tests in one loop 64 sequences of
  // 300-12000 tokens took 135 us, so 131; of four query tokens 206 and 198.)
  const uint32_t first = stage + piece_at<D>(lane / (D / 16), lane % (D / 16));
  const uint8_t* k = p.k + off;
  const uint8_t* v = p.v + off;
  if (ok && tok >= lo && tok + kPaGroup <= hi) {  // whole (warp-uniform)
#pragma unroll
    for (int i = 0; i < kPieces / 32; ++i) {
      const uint32_t at = (D == 128 && (i & 1) ? first ^ 32u : first) + i * 512;
      cp_async16(at, k + i * 512);
      cp_async16(at + kPaGroup * D, v + i * 512);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPieces / 32; ++i) {
      const int t = tok + i * (512 / D) + lane / (D / 16);
      const bool keep = ok && t >= lo && t < hi;
      const uint32_t at = (D == 128 && (i & 1) ? first ^ 32u : first) + i * 512;
      cp_async16(at, k + i * 512, keep);
      cp_async16(at + kPaGroup * D, v + i * 512, keep);
    }
  }
  if (lane < 2)
    cp_async4(scale_at + lane * 4, (lane == 0 ? p.k_scale : p.v_scale) + block,
              ok);
}

// One run of units: query rows [row0, row0 + 8 NT) of one (sequence,
// key/value head), groups [g0, g1) of its plan.  Warp w takes groups
// g1 - 1 - w, g1 - 5 - w, ... of 16 tokens.  Per group, with the group as the 16-row
// operand so that 8 query rows fill the other one:
//     S^T [16 tokens][8 rows] = K q^T,   O^T [D][8 rows] += V^T P^T.
// K and V go from shared memory to registers as they lie (16 bytes per lane)
// and become f16, which holds every e4m3 value, as do P (11 bits; its
// rounding is 2^-11) and q, scaled by a power of two per row.
// `part`: where to leave o [row][D], m and l of an item cut across CTAs, or
// null to write the result.
template <int D, int NT, bool TREE>
__device__ __forceinline__ void attend_run(const PagedParams& p, uint8_t* smem,
                                           int b, const PaPlan& plan, int hkv,
                                           int row0, int g0, int g1,
                                           float* part) {
  using C = PaCfg<D, NT>;
  constexpr int kSteps = D / 16, kPaStages = C::kPaStages;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  const int G = p.H / p.H_kv, rows = G * p.T;
  const float NEG_INF = __int_as_float(0xff800000);
  // a row's maximum before it has seen a key: the lowest finite value, from
  // which -inf - m and m - m need no special case
  const float kLowest = __int_as_float(0xff7fffff);
  const int len = plan.len, lo = plan.lo, first_group = plan.first_group;
  const int base = len - plan.drafts;  // tokens before the drafts (TREE)

  // the copies start first; the queries are loaded while they run
  const uint32_t ring = smem_u32(smem) + warp * kPaStages * C::kStage;
  const uint32_t scales = smem_u32(smem) + C::kOffScale + warp * kPaStages * 8;
  const int* table = p.table + static_cast<int64_t>(b) * p.table_stride;
  // the run's groups from the last to the first: with a bias that falls with
  // the distance the maximum is then met early and o is seldom rescaled (64
  // sequences of 300-12000 tokens with a bias: 158 us in rising order, 137 in
  // this one)
  const int n = g1 - g0;
  auto group_of = [&](int k) { return first_group + g1 - 1 - k; };
  // the page of the run's k-th group; -1 past its end and for a page out of
  // range
  auto page_of = [&](int k) {
    if (k >= n) return -1;
    const int slot = group_of(k) >> (p.page_shift - 4);
    const int pid = table[slot];
    if (static_cast<uint32_t>(pid) < static_cast<uint32_t>(p.num_pages))
      return pid;
    if (lane == 0) record_bad_index(b, slot, pid);
    __syncwarp();  // (matrix instructions are a whole warp's, here as below)
    return -1;
  };
  auto issue = [&](int k, int st, int pid) {
    if (k < n)
      load_group<D>(p, ring + st * C::kStage, scales + st * 8, hkv, pid,
                    group_of(k) * kPaGroup, lo, len);
    cp_async_commit();
  };
  // the ring's first groups, their pages looked up together; from then on a
  // group's page is looked up one turn before its copy starts
  int pid[kPaStages];
#pragma unroll
  for (int i = 0; i < kPaStages; ++i) pid[i] = page_of(warp + i * kPaWarps);
#pragma unroll
  for (int i = 0; i < kPaStages - 1; ++i)
    issue(warp + i * kPaWarps, i, pid[i]);
  int next_pid = pid[kPaStages - 1];

  // query fragments: row row0 + 8 nt + g, elements 64 h + 16 t .. + 15.  One
  // tile's stay in registers; two tiles' (32 registers at D = 128, which the
  // third CTA of an SM would not get) are read from shared memory, where the
  // four warps, which hold the same ones, leave them
  uint32_t qf[NT][kSteps][2];
  const uint32_t q_at = smem_u32(smem) + C::kOffQ + lane * 16;
  // of rows 8 nt + 2 t, + 1: 2^(row's exponent) times what makes q.k the
  // exponent of e^(2 x / cap), or x, in log2 units
  float q_mul[NT][2];
  float slope2[NT][2];
  int pos[NT][2];  // positions of those rows; -1 for rows that do not exist
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = row0 + nt * 8 + g;
    uint32_t w[kSteps][2];
    uint32_t top = 0;
    const uint16_t* src =
        p.q + b * p.q_sb +
        static_cast<int64_t>(hkv * G + min(r, rows - 1) / p.T) * p.q_sh +
        static_cast<int64_t>(min(r, rows - 1) % p.T) * p.q_ss;
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(src + 64 * h + 16 * t +
                                                        8 * i);
        w[4 * h + 2 * i][0] = v.x;
        w[4 * h + 2 * i][1] = v.y;
        w[4 * h + 2 * i + 1][0] = v.z;
        w[4 * h + 2 * i + 1][1] = v.w;
      }
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) top = max_u16x2(top, w[s][i] & 0x7fff7fffu);
    top = max(top & 0xffffu, top >> 16);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // the row's largest magnitude becomes [1, 2): f16 then keeps bf16's 8
    // bits of every element above 2^-17 of it, and 2^-25 of it of the rest.
    // Exponents at the ends of the range stay finite factors.
    const int e = min(max(static_cast<int>(top >> 7) - 127, -120), 120);
    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        qf[nt][s][i] = pack_f16x2(bf16_lo(w[s][i]) * down,
                                  bf16_hi(w[s][i]) * down);
    if (NT > 1) {
#pragma unroll
      for (int s = 0; s < kSteps; s += 2)
        if (warp == nt * 2 + (s / 2 & 1))
          sts128(q_at + (nt * (kSteps / 2) + s / 2) * 512, qf[nt][s][0],
                 qf[nt][s][1], qf[nt][s + 1][0], qf[nt][s + 1][1]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // lane (2 t + i) * 4 holds row 2 t + i's factor
      const float u = __shfl_sync(0xffffffffu, up, (2 * t + i) * 4);
      const int rr = row0 + nt * 8 + 2 * t + i;
      const bool live = rr < rows;
      q_mul[nt][i] = u * p.scale_x;
      pos[nt][i] = live ? len - p.T + rr % p.T : -1;
      if (TREE) {
        const int t = live ? rr % p.T : 0;
        const int depth =
            live && t < plan.drafts ? draft_depth(p, b, t, plan.drafts) : -1;
        pos[nt][i] = depth >= 0 ? base + depth : -1;
      }
      slope2[nt][i] = (p.mod.kind & kModBias) && live
                          ? p.mod.slopes[hkv * G + rr / p.T] *
                                1.4426950408889634f
                          : 0.f;
    }
  }
  if (NT > 1) __syncthreads();
  // a group none of whose tokens any live row masks
  const int pos_min = TREE ? base - 1 : len - p.T, pos_max = len - 1;

  float o[NT][kSteps][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[nt][s][i] = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      m[nt][i] = kLowest;
      l[nt][i] = 0.f;
    }
  }
  float v_ref = 1.f;  // o is in units of this value scale

  // distance of the lane's first token to the rows' positions (negative),
  // kept as it moves on: exact in f32
  float dist[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c)
      dist[nt][c] =
          static_cast<float>(group_of(warp) * kPaGroup + g - pos[nt][c]);

  int st = 0;
  float v_inv = 1.f;  // 1 / v_ref
  for (int k = warp; k < n;
       k += kPaWarps, st = st + 1 == kPaStages ? 0 : st + 1) {
    cp_async_wait<kPaStages - 2>();
    __syncwarp();  // the group is in shared memory, and the one before it read
    issue(k + (kPaStages - 1) * kPaWarps, st == 0 ? kPaStages - 1 : st - 1,
          next_pid);
    next_pid = page_of(k + kPaStages * kPaWarps);
    const uint32_t k_at = ring + st * C::kStage, v_at = k_at + C::kHalf;
    const uint2 sc = lds64(scales + st * 8);
    const float k_scale = __uint_as_float(sc.x);
    const float v_scale = __uint_as_float(sc.y);
    float d[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        d[nt][c] = dist[nt][c];
        dist[nt][c] -= static_cast<float>(kPaGroup * kPaWarps);
      }
    if (k_scale == 0.f) continue;  // a page that is not there (whole warp)
    const int tok = group_of(k) * kPaGroup;

    // ---- S^T = K q^T
    // (in two chains of accumulation, as each product waits for the one before)
    float s[NT][4], s1[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[nt][i] = s1[nt][i] = 0.f;
    uint4 qs[NT];
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
      const uint4 x = lds128(k_at + piece_at<D>(g, 4 * h + t));
      const uint4 y = lds128(k_at + piece_at<D>(g + 8, 4 * h + t));
      const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
      const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a0 = e4m3x2_to_f16x2(xw[j]), a2 = e4m3x2_to_f16x2_hi(xw[j]);
        const uint32_t a1 = e4m3x2_to_f16x2(yw[j]), a3 = e4m3x2_to_f16x2_hi(yw[j]);
        if (NT == 1) {
          mma16816((j & 1) ? s1[0] : s[0], a0, a1, a2, a3,
                   qf[0][4 * h + j][0], qf[0][4 * h + j][1]);
        } else {
          if ((j & 1) == 0)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              qs[nt] = lds128(q_at + (nt * (kSteps / 2) + 2 * h + j / 2) * 512);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816((j & 1) ? s1[nt] : s[nt], a0, a1, a2, a3,
                     (j & 1) ? qs[nt].z : qs[nt].x,
                     (j & 1) ? qs[nt].w : qs[nt].y);
        }
      }
    }

    // ---- the cap: tanh(y) = 1 - 2 / (1 + 2^x), x = 2 y log2(e), off by 2^-23
    // of the cap; above a cap of about 200 that would show in the logits, and
    // small y take the forward's polynomial instead
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s[nt][i] = (s[nt][i] + s1[nt][i]) * (q_mul[nt][i & 1] * k_scale);
    if (p.mod.kind & kModCap) {
      if (p.mod.cap_log2 > 300.f) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = s[nt][i], y = x * 0.34657359f, y2 = y * y;
            const float z = fmaf(-2.f, rcp_approx(ex2_approx(x) + 1.f), 1.f);
            const float t = fmaf(y2, fmaf(y2, fmaf(y2, -0.04439273843f,
                                                   0.1318993943f),
                                          -0.3332628423f),
                                 0.999999451f);
            s[nt][i] = p.mod.cap_log2 * (y2 <= 0.25f ? y * t : z);
          }
      } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            s[nt][i] = fmaf(-2.f * p.mod.cap_log2,
                            rcp_approx(ex2_approx(s[nt][i]) + 1.f),
                            p.mod.cap_log2);
      }
    }

    // ---- logits in log2 units, mask, running maximum
    const bool inner = tok + kPaGroup - 1 <= pos_min &&
                       (p.window <= 0 || pos_max - tok < p.window);
    // of drafts among the group: what each row sees of the lane's two tokens,
    // and their distances, which depths give
    bool hidden[NT][4];
    if (TREE && !inner) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = tok + g + h * 8;
        const bool draft = j >= base && j < len;
        const int at =
            draft && (p.window > 0 || (p.mod.kind & kModBias))
                ? base + draft_depth(p, b, j - base, plan.drafts)
                : j;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int rr = row0 + nt * 8 + 2 * t + c;
            bool hide = j >= len || pos[nt][c] < 0;
            if (draft && !hide)
              hide = !(draft_bits(p, b, rr % p.T, (j - base) / 32,
                                  plan.drafts) >> ((j - base) % 32) & 1u);
            hidden[nt][2 * h + c] =
                hide || (p.window > 0 && pos[nt][c] - at >= p.window);
            if (draft && (p.mod.kind & kModBias))
              s[nt][2 * h + c] = fmaf(
                  slope2[nt][c],
                  -fabsf(static_cast<float>(pos[nt][c] - at)) -
                      (d[nt][c] + h * 8.f),
                  s[nt][2 * h + c]);  // (less what is added below)
          }
      }
      __syncwarp();
    }
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = i & 1, j = tok + g + (i >> 1) * 8;
        float x = s[nt][i];
        if (p.mod.kind & kModBias)
          x = fmaf(slope2[nt][c], d[nt][c] + (i >> 1) * 8.f, x);
        if (!inner &&
            (TREE ? hidden[nt][i]
                  : j > pos[nt][c] ||
                        (p.window > 0 && pos[nt][c] - j >= p.window)))
          x = NEG_INF;
        s[nt][i] = x;
        grow = grow || !(x <= m[nt][c]);
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = fmaxf(s[nt][c], s[nt][c + 2]);
#pragma unroll
          for (int d = 4; d < 32; d *= 2)
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
          // (selected, not branched on: the lanes stay together)
          const bool more = mx > m[nt][c];
          const float alpha = more ? ex2_approx(m[nt][c] - mx) : 1.f;
          m[nt][c] = more ? mx : m[nt][c];
          l[nt][c] *= alpha;
#pragma unroll
          for (int d = 0; d < kSteps; ++d) {
            o[nt][d][c] *= alpha;
            o[nt][d][c + 2] *= alpha;
          }
        }
    }
    // ---- the value scale: o is kept in units of v_ref / kPUp, and a
    // group's scale multiplies p while it is within 2^6 of v_ref; past that o
    // moves to the new unit.  p <= 1, so p * kPUp * 2^6 <= 2^15 fits f16, and
    // what f16 flushes to zero is p below 2^-27: 2^18 such keys together
    // weigh less than the 2^-8 of the output's own rounding
    float v_mul = v_scale * v_inv;
    if (!(v_mul >= 0.015625f && v_mul <= 64.f)) {
      const float r = v_ref / v_scale;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int d = 0; d < kSteps; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[nt][d][i] *= r;
      v_ref = v_scale;
      v_inv = 1.f / v_scale;
      v_mul = 1.f;
    }
    v_mul *= kPUp;

    // ---- p and its transpose as the second operand
    uint32_t pb[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float pr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pr[i] = ex2_approx(s[nt][i] - m[nt][i & 1]);
        l[nt][i & 1] += pr[i];
        pr[i] *= v_mul;
      }
      pb[nt][0] = transpose8x8(pack_f16x2(pr[0], pr[1]));
      pb[nt][1] = transpose8x8(pack_f16x2(pr[2], pr[3]));
    }

    // ---- O^T += V^T P^T: lane (g, t) holds elements of tokens 2t, 2t + 1,
    // 2t + 8, 2t + 9: 16 (D = 128) or 8 (D = 64) consecutive dims
    uint32_t vw[4][D / 32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tr = 2 * t + (i & 1) + (i >> 1) * 8;
      if (D == 128) {
        const uint4 v =
            lds128(v_at + piece_at<D>(tr, ((g & 1) << 2) | (g >> 1)));
        vw[i][0] = v.x;
        vw[i][1] = v.y;
        vw[i][D / 32 - 2] = v.z;
        vw[i][D / 32 - 1] = v.w;
      } else {
        const uint2 v = lds64(v_at + piece_at<D>(tr, g >> 1) + (g & 1) * 8);
        vw[i][0] = v.x;
        vw[i][1] = v.y;
      }
    }
    // Where the rows see different tokens (T > 1 only), a NaN value that a
    // row does not see must not reach it as 0 * NaN: such elements are taken
    // out of V, and the rows that do see one get NaN there.
    if (!inner && (TREE || p.T > 1)) {
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < D / 32; ++j) any |= nan_codes(vw[i][j]);
      if (__any_sync(0xffffffffu, any != 0)) {
        uint32_t seen[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int j = tok + g + 8 * hh;
            float f[2];
#pragma unroll
            for (int c = 0; c < 2; ++c)
              f[c] = (TREE ? hidden[nt][2 * hh + c]
                           : j > pos[nt][c] ||
                                 (p.window > 0 && pos[nt][c] - j >= p.window))
                         ? 0.f
                         : 1.f;
            seen[nt][hh] = transpose8x8(pack_f16x2(f[0], f[1]));
          }
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          uint32_t one[4];  // 1.0 (code 0x38) where V holds a NaN
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t bytes = (nan_codes(vw[i][j]) >> 7) * 0xffu;
            one[i] = bytes & 0x38383838u;
            vw[i][j] &= ~bytes;
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t sel = u == 0 ? 0x5140u : 0x7362u;
            const uint32_t x = __byte_perm(one[0], one[1], sel);
            const uint32_t y = __byte_perm(one[2], one[3], sel);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float n[4] = {0.f, 0.f, 0.f, 0.f};
              mma16816(n, e4m3x2_to_f16x2(x), e4m3x2_to_f16x2_hi(x),
                       e4m3x2_to_f16x2(y), e4m3x2_to_f16x2_hi(y), seen[nt][0],
                       seen[nt][1]);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (n[i] > 0.f)
                  o[nt][2 * j + u][i] = __int_as_float(0x7fffffff);
            }
          }
        }
        __syncwarp();
      }
    }
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t sel = u == 0 ? 0x5140u : 0x7362u;
        const uint32_t x = __byte_perm(vw[0][j], vw[1][j], sel);
        const uint32_t y = __byte_perm(vw[2][j], vw[3][j], sel);
        const uint32_t a0 = e4m3x2_to_f16x2(x), a1 = e4m3x2_to_f16x2_hi(x);
        const uint32_t a2 = e4m3x2_to_f16x2(y), a3 = e4m3x2_to_f16x2_hi(y);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma16816(o[nt][2 * j + u], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
      }
  }
  cp_async_wait<0>();
  __syncthreads();  // the rings become the warps' results

  // ---- join the warps: o [warp][row][D], then m and l [warp][row]
  constexpr int R = 8 * NT;
  float* so = reinterpret_cast<float*>(smem);
  float* sm = so + kPaWarps * R * D;
  float* sl = sm + kPaWarps * R;
  static_assert((kPaWarps * R * (D + 2)) * 4 <= C::kOffScale, "join area");
  const float unit = v_ref / kPUp;
  const int dim0 = D == 128 ? 16 * (((g & 1) << 2) | (g >> 1)) : 8 * g;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float sum = l[nt][c];
#pragma unroll
      for (int d = 4; d < 32; d *= 2)
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
      const int r = nt * 8 + 2 * t + c;
      if (TREE && pos[nt][c] < 0) {  // an empty row, whatever it gathered
        sum = 0.f;
        m[nt][c] = kLowest;
#pragma unroll
        for (int d = 0; d < kSteps; ++d) o[nt][d][c] = o[nt][d][c + 2] = 0.f;
      }
      if (g == 0) {
        sm[warp * R + r] = m[nt][c];
        sl[warp * R + r] = sum;
      }
#pragma unroll
      for (int d = 0; d < kSteps; d += 2)
        *reinterpret_cast<float4*>(so + (warp * R + r) * D + dim0 + 2 * d) =
            make_float4(o[nt][d][c] * unit, o[nt][d][c + 2] * unit,
                        o[nt][d + 1][c] * unit, o[nt][d + 1][c + 2] * unit);
    }
  __syncthreads();
  for (int i = threadIdx.x; i < R * (D / 2); i += kPaThreads) {
    const int r = i / (D / 2), d = i % (D / 2) * 2;
    const int rr = row0 + r;
    if (rr >= rows) break;
    float base = kLowest;
#pragma unroll
    for (int w = 0; w < kPaWarps; ++w) base = fmaxf(base, sm[w * R + r]);
    float sum = 0.f, xy[2] = {0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kPaWarps; ++w) {
      const float f = ex2_approx(sm[w * R + r] - base);
      sum = fmaf(sl[w * R + r], f, sum);
      const float2 v = *reinterpret_cast<float2*>(so + (w * R + r) * D + d);
      xy[0] = fmaf(v.x, f, xy[0]);
      xy[1] = fmaf(v.y, f, xy[1]);
    }
    if (part != nullptr) {
      *reinterpret_cast<float2*>(part + r * D + d) = make_float2(xy[0], xy[1]);
      if (d == 0) {
        part[R * D + r] = base;
        part[R * D + R + r] = sum;
      }
      continue;
    }
    write_row<2>(p, b, hkv * G + rr / p.T, rr % p.T, d, base, sum, xy);
  }
  __syncthreads();  // the join area becomes the rings again
}

// CTAs per SM of the attention kernel: three rings fit an SM's shared memory
// at head dim 128.  At 64 four fit its registers (64 sequences of 300-12000
// tokens, one row tile: 86 us, with five 91; two: 128, with three 131).
template <int D, int NT>
constexpr int kPaPerSm = D == 64 ? 4 : 3;

static_assert(kPaPerSm<64, 2> <= kPaMaxPerSm, "workspace");

template <int D, int NT, bool TREE>
__global__ void __launch_bounds__(kPaThreads, kPaPerSm<D, NT>)
    paged_attention_kernel(const PagedParams p) {
  using X = PaDeal<TREE>;
  extern __shared__ __align__(128) uint8_t smem[];
  // the join kernel may be scheduled once every CTA here runs; it waits for
  // this grid's end before it reads the parts
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int rows = p.H / p.H_kv * p.T;
  const int tiles = (rows + 8 * NT - 1) / (8 * NT);
  const int per = p.H_kv * tiles;
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.B; b += kPaThreads) {
      const int len = p.lens[b];
      const PaPlan plan = plan_of<X>(p, b);
      if (len != plan.len) record_bad_index(b, -1, len);
      if (TREE && p.n_new != nullptr && p.n_new[b] != plan.drafts)
        record_bad_index(b, -1, p.n_new[b]);
    }
  int64_t u = -1, end = -1, start;
  int b = find_sequence<X>(
      p, per,
      [&](int64_t all) {
        const int64_t units = all * per;
        const int64_t busy = busy_ctas<X>(units, gridDim.x);
        if (blockIdx.x < busy) {
          u = mul_div(blockIdx.x, units, busy);
          end = mul_div(blockIdx.x + 1, units, busy);
        }
        return u;
      },
      &start);
  if (b < 0) return;
  while (u < end) {
    const PaPlan plan = plan_of<X>(p, b);
    const int64_t row_cost = static_cast<int64_t>(plan.n_cost) * per;
    if (u >= start + row_cost) {
      start += row_cost;
      ++b;
      continue;
    }
    const int64_t within = u - start;
    const int item = within < (int64_t{1} << 31)
                         ? static_cast<int>(static_cast<uint32_t>(within) /
                                            static_cast<uint32_t>(plan.n_cost))
                         : static_cast<int>(within / plan.n_cost);
    const int off =
        static_cast<int>(within - static_cast<int64_t>(item) * plan.n_cost);
    const int n = static_cast<int>(
        min(static_cast<int64_t>(plan.n_cost - off), end - u));
    // units [r0, r1) of the item
    const int r0 = max(off - X::kRunCost, 0), r1 = off + n - X::kRunCost;
    if (r1 > r0) {
      float* part = nullptr;
      if (r0 > 0 || r1 < plan.n_units)  // slot 0: an earlier CTA has the start
        part = p.parts + (blockIdx.x * 2 + (r0 > 0 ? 0 : 1)) *
                             static_cast<int64_t>(8 * NT * (D + 2));
      attend_run<D, NT, TREE>(p, smem, b, plan, item / tiles,
                              item % tiles * 8 * NT, r0 * kPaWarps,
                              min(r1 * kPaWarps, plan.n_groups), part);
    }
    u += n;
  }
}

template <int D, int NT, bool TREE>
cudaError_t launch_paged(const PagedParams& p, int num_sms,
                         cudaStream_t stream) {
  using X = PaDeal<TREE>;
  auto kern = paged_attention_kernel<D, NT, TREE>;
  cudaError_t e = cudaFuncSetAttribute(
      kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PaCfg<D, NT>::kSmem);
  if (e != cudaSuccess) return e;
  const int rows = p.H / p.H_kv * p.T;
  const int tiles = (rows + 8 * NT - 1) / (8 * NT);
  const int grid = num_sms * kPaPerSm<D, NT>;
  kern<<<grid, kPaThreads, PaCfg<D, NT>::kSmem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_join<X, D, 8 * NT>(p, grid, num_sms, stream);
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t stream) {
  const int slots = (p.T + p.page_size - 2) / p.page_size + 1;
  const dim3 grid(slots, 2 * p.H_kv, p.B);
  switch (p.page_size * p.D / (8 * kAppendThreads)) {
    case 1: kv_append_kernel<1><<<grid, kAppendThreads, 0, stream>>>(p); break;
    case 2: kv_append_kernel<2><<<grid, kAppendThreads, 0, stream>>>(p); break;
    case 4: kv_append_kernel<4><<<grid, kAppendThreads, 0, stream>>>(p); break;
    case 8: kv_append_kernel<8><<<grid, kAppendThreads, 0, stream>>>(p); break;
    case 16: kv_append_kernel<16><<<grid, kAppendThreads, 0, stream>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

template <int D>
static cudaError_t append_rope(const AppendParams& p, const TurnParams& t,
                               cudaStream_t stream) {
  const int slots = (p.T + p.page_size - 2) / p.page_size + 1;
  const dim3 grid(slots, 2 * p.H_kv, p.B);
  // steps of the block over a page's pieces (the smallest pages: part of one)
  switch (p.page_size * D / (16 * kTurnThreads)) {
    case 0:
    case 1: kv_append_rope_kernel<D, 1><<<grid, kTurnThreads, 0, stream>>>(p, t); break;
    case 2: kv_append_rope_kernel<D, 2><<<grid, kTurnThreads, 0, stream>>>(p, t); break;
    case 4: kv_append_rope_kernel<D, 4><<<grid, kTurnThreads, 0, stream>>>(p, t); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t launch_kv_append_rope(const AppendParams& p, const TurnParams& t,
                                  cudaStream_t stream) {
  return p.D == 128 ? append_rope<128>(p, t, stream)
                    : append_rope<64>(p, t, stream);
}

template <bool TREE>
static cudaError_t launch_rows(const PagedParams& p, int num_sms,
                               cudaStream_t stream) {
  // one tile of 8 query rows, or two where the group and the tokens fill them
  const bool two = static_cast<int64_t>(p.H / p.H_kv) * p.T > 8;
  if (p.D == 128)
    return two ? launch_paged<128, 2, TREE>(p, num_sms, stream)
               : launch_paged<128, 1, TREE>(p, num_sms, stream);
  if (p.D == 64)
    return two ? launch_paged<64, 2, TREE>(p, num_sms, stream)
               : launch_paged<64, 1, TREE>(p, num_sms, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_paged_attention(const PagedParams& p, int num_sms,
                                   cudaStream_t stream) {
  return launch_rows<false>(p, num_sms, stream);
}

cudaError_t launch_paged_tree(const PagedParams& p, int num_sms,
                              cudaStream_t stream) {
  return launch_rows<true>(p, num_sms, stream);
}

cudaError_t read_cache_error(int32_t out[4]) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_cache_error, 4 * sizeof(int32_t));
  if (e != cudaSuccess) return e;
  const int32_t zero[4] = {0, 0, 0, 0};
  return cudaMemcpyToSymbol(g_cache_error, zero, 4 * sizeof(int32_t));
}

}  // namespace bsm
