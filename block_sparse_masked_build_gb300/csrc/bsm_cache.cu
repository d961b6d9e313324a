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
#include "bsm_ptx.cuh"

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

__device__ __forceinline__ float bf16_lo(uint32_t w) {
  return __uint_as_float(w << 16);
}
__device__ __forceinline__ float bf16_hi(uint32_t w) {
  return __uint_as_float(w & 0xffff0000u);
}

// Two e4m3 codes (the low 16 bits) as f16x2; exact, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
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
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
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

// --------------------------------------------------------------- attention

constexpr int kPaWarps = 4;
constexpr int kPaThreads = 32 * kPaWarps;
constexpr int kPaGroup = 16;  // tokens a warp works on at a time
constexpr int kPaRunCost = 4; // see PaPlan
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

// The high bit of every byte of w that is a NaN code (0x7f or 0xff).
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
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

// Writes N elements of one result row from dim d on: x / sum in bf16 and, with
// d = 0, the logsumexp of base + log2(sum).  sum = 0: the row saw no key.
template <int N>
__device__ __forceinline__ void write_row(const PagedParams& p, int b,
                                          int head, int t, int d, float base,
                                          float sum, const float* x) {
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  uint16_t* dst = p.out + b * p.o_sb + head * p.o_sh + t * p.o_ss + d;
#pragma unroll
  for (int i = 0; i < N; i += 2)
    *reinterpret_cast<uint32_t*>(dst + i) =
        pack_bf16x2(x[i] * inv, x[i + 1] * inv);
  if (d == 0 && p.lse != nullptr)
    p.lse[(static_cast<int64_t>(b) * p.H + head) * p.T + t] =
        sum != 0.f ? (base + log2f(sum)) * 0.6931471805599453f
                   : __int_as_float(0xff800000);
}

// How the tokens are dealt out.  An item is (sequence, key/value head, tile of
// 8 NT query rows); its work is its sequence's visible tokens in units of 64
// (a group of 16 for each warp).  All units of all items, in order, are cut
// into equal runs, one per CTA, so that unequal lengths and few long
// sequences load every SM alike.  An item counts kPaRunCost units more than
// it has, before its first: what starting and ending a run costs (64
// sequences of 300-12000 tokens: 160 us without, 140 with).  A CTA may start and end inside an item;
// then it leaves its part (o, m, l) in the workspace and the join kernel adds
// the parts up.  The cut depends on the lengths alone, which both kernels
// read.
struct PaPlan {
  int len, lo;      // of one sequence: tokens, first visible one
  int first_group;  // of 16 tokens
  int n_groups, n_units;
  int n_cost;  // n_units + kPaRunCost, or 0 without units
};

__device__ __forceinline__ PaPlan plan_of(const PagedParams& p, int len) {
  PaPlan s;
  s.len = min(max(len, 0), p.max_pages * p.page_size);
  s.lo = p.window > 0 ? max(0, s.len - p.T - p.window + 1) : 0;
  s.first_group = s.lo / kPaGroup;
  s.n_groups = (s.len + kPaGroup - 1) / kPaGroup - s.first_group;
  s.n_units = (s.n_groups + kPaWarps - 1) / kPaWarps;
  s.n_cost = s.n_units > 0 ? s.n_units + kPaRunCost : 0;
  return s;
}

// a * b / c, in 32 bits where that is enough (a 64-bit division takes some
// hundred instructions, and small calls are bound by latency).
__device__ __forceinline__ int64_t mul_div(int64_t a, int64_t b, int64_t c) {
  if (((a | b) < (1 << 15) || (a < 1024 && b < (1 << 21))) &&
      c < (int64_t{1} << 31))
    return static_cast<uint32_t>(a) * static_cast<uint32_t>(b) /
           static_cast<uint32_t>(c);
  return a * b / c;
}

// Where the units of an item row (one head and row tile) lie: the sum over all
// sequences, and of those before one of them.
struct PaScan {
  int64_t all, before;
};

// One warp's scan of the lengths, every warp on its own (no barrier): lane i
// takes `chunk` sequences in order.  n: its sequences' units.
__device__ __forceinline__ int lane_units(const PagedParams& p, int chunk,
                                          int64_t* n) {
  const int b0 = (threadIdx.x % 32) * chunk;
  int64_t sum = 0;
  for (int i = 0; i < chunk; ++i)
    if (b0 + i < p.B) sum += plan_of(p, p.lens[b0 + i]).n_cost;
  *n = sum;
  return b0;
}

__device__ __forceinline__ PaScan scan_before(const PagedParams& p, int seq) {
  const int chunk = (p.B + 31) / 32;
  int64_t all = 0, head = 0;
  // interleaved: both sums, whatever the order
  for (int i = 0; i < chunk; ++i) {
    const int b = i * 32 + threadIdx.x % 32;
    if (b < p.B) {
      const int n = plan_of(p, p.lens[b]).n_cost;
      all += n;
      if (b < seq) head += n;
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) {
    all += __shfl_xor_sync(0xffffffffu, all, d);
    head += __shfl_xor_sync(0xffffffffu, head, d);
  }
  return PaScan{all, head};
}

// Sums all units (of one item row) and finds the sequence that holds the unit
// `u_of(total)` of `per` item rows per sequence: the b with start(b) <= u <
// start(b + 1).  Whole warps; the same in every one.
template <class F>
__device__ __forceinline__ int find_sequence(const PagedParams& p, int per,
                                             F&& u_of, int64_t* start) {
  const int lane = threadIdx.x % 32;
  const int chunk = (p.B + 31) / 32;
  int64_t n;
  int b = lane_units(p, chunk, &n);
  int64_t inc = n;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += v;
  }
  const int64_t u = u_of(__shfl_sync(0xffffffffu, inc, 31));
  int64_t at = (inc - n) * per;
  const unsigned has =
      __ballot_sync(0xffffffffu, u >= 0 && n > 0 && at <= u && u < inc * per);
  if (has == 0) return -1;
  const int owner = __ffs(has) - 1;
  if (lane == owner)
    for (;; ++b) {
      const int64_t m =
          static_cast<int64_t>(plan_of(p, p.lens[b]).n_cost) * per;
      if (u < at + m) break;
      at += m;
    }
  *start = __shfl_sync(0xffffffffu, at, owner);
  return __shfl_sync(0xffffffffu, b, owner);
}

// CTAs that get work: at least two units each, so that a CTA's first loads
// and its join are spread over more than one round of groups.
__device__ __forceinline__ int64_t busy_ctas(int64_t units, int64_t grid) {
  const int64_t n = (units + 1) / 2;
  return n < grid ? n : grid;
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
template <int D, int NT>
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
      slope2[nt][i] = (p.mod.kind & kModBias) && live
                          ? p.mod.slopes[hkv * G + rr / p.T] *
                                1.4426950408889634f
                          : 0.f;
    }
  }
  if (NT > 1) __syncthreads();
  // a group none of whose tokens any live row masks
  const int pos_min = len - p.T, pos_max = len - 1;

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
            (j > pos[nt][c] || (p.window > 0 && pos[nt][c] - j >= p.window)))
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
          if (mx > m[nt][c]) {
            const float alpha = ex2_approx(m[nt][c] - mx);  // 0 from -inf
            m[nt][c] = mx;
            l[nt][c] *= alpha;
#pragma unroll
            for (int d = 0; d < kSteps; ++d) {
              o[nt][d][c] *= alpha;
              o[nt][d][c + 2] *= alpha;
            }
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
    if (!inner && p.T > 1) {
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
              f[c] = j > pos[nt][c] ||
                             (p.window > 0 && pos[nt][c] - j >= p.window)
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

template <int D, int NT>
__global__ void __launch_bounds__(kPaThreads, kPaPerSm<D, NT>)
    paged_attention_kernel(const PagedParams p) {
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
      if (len != plan_of(p, len).len) record_bad_index(b, -1, len);
    }
  int64_t u = -1, end = -1, start;
  int b = find_sequence(
      p, per,
      [&](int64_t all) {
        const int64_t units = all * per;
        const int64_t busy = busy_ctas(units, gridDim.x);
        if (blockIdx.x < busy) {
          u = mul_div(blockIdx.x, units, busy);
          end = mul_div(blockIdx.x + 1, units, busy);
        }
        return u;
      },
      &start);
  if (b < 0) return;
  while (u < end) {
    const PaPlan plan = plan_of(p, p.lens[b]);
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
    const int r0 = max(off - kPaRunCost, 0), r1 = off + n - kPaRunCost;
    if (r1 > r0) {
      float* part = nullptr;
      if (r0 > 0 || r1 < plan.n_units)  // slot 0: an earlier CTA has the start
        part = p.parts + (blockIdx.x * 2 + (r0 > 0 ? 0 : 1)) *
                             static_cast<int64_t>(8 * NT * (D + 2));
      attend_run<D, NT>(p, smem, b, plan, item / tiles, item % tiles * 8 * NT,
                        r0 * kPaWarps, min(r1 * kPaWarps, plan.n_groups), part);
    }
    u += n;
  }
}

// Joins the parts of the items that were cut and writes the rows of sequences
// without tokens: a warp per query row, or (WIDE) a block, whose warps share
// the parts.
template <int D, int NT, bool WIDE>
__global__ void __launch_bounds__(kPaThreads)
    paged_join_kernel(const PagedParams p, const int grid) {
  constexpr int R = 8 * NT, kPer = D / 32;
  const int rows = p.H / p.H_kv * p.T;
  const int tiles = (rows + R - 1) / R;
  const int per = p.H_kv * tiles;
  const int b = blockIdx.z, item = blockIdx.y;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int r = WIDE ? blockIdx.x : blockIdx.x * kPaWarps + warp;
  const int rr = item % tiles * R + r;
  const PaScan scan = scan_before(p, b);
  const int64_t units = scan.all * per;
  const int n = plan_of(p, p.lens[b]).n_units;
  // every block waits for the attention grid, so that work after this kernel
  // on the stream sees what that grid wrote itself
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (rr >= rows || r >= R) return;
  const int head = item / tiles * (p.H / p.H_kv) + rr / p.T, t = rr % p.T;
  float x[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) x[i] = 0.f;
  if (n == 0) {
    write_row<kPer>(p, b, head, t, lane * kPer, 0.f, 0.f, x);
    return;
  }
  const int64_t busy = busy_ctas(units, grid);
  // the CTAs that hold its first and last unit
  const int64_t u0 = scan.before * per +
                     static_cast<int64_t>(item) * (n + kPaRunCost) + kPaRunCost;
  auto cta_of = [&](int64_t u) {  // the last c with c * units / busy <= u
    const int64_t c = mul_div(u + 1, busy, units);
    return c - (c * units == (u + 1) * busy);
  };
  const int64_t c0 = cta_of(u0), c1 = cta_of(u0 + n - 1);
  if (c0 == c1) return;  // whole in one CTA, which wrote it
  // the item's first unit is in the first CTA, which leaves its part in slot 1
  constexpr int64_t kPart = R * (D + 2);
  auto part_of = [&](int64_t c) {
    return p.parts + (c * 2 + (c == c0 ? 1 : 0)) * kPart;
  };
  float base = __int_as_float(0xff7fffff);  // as every part's before a key
  for (int64_t c = c0 + lane; c <= c1; c += 32)
    base = fmaxf(base, part_of(c)[R * D + r]);
#pragma unroll
  for (int d = 16; d > 0; d /= 2)
    base = fmaxf(base, __shfl_xor_sync(0xffffffffu, base, d));
  float sum = 0.f;
  constexpr int kStep = WIDE ? kPaWarps : 1;
  const int64_t first = c0 + (WIDE ? warp : 0);
  for (int64_t c = first; c <= c1; c += 32 * kStep) {
    // lane i: the weight of part c + i kStep
    float f = 0.f;
    if (c + lane * kStep <= c1) {
      const float* part = part_of(c + lane * kStep) + R * D + r;
      f = ex2_approx(part[0] - base);
      sum = fmaf(part[R], f, sum);
    }
    const int m = static_cast<int>(
        min((c1 - c) / kStep + 1, static_cast<int64_t>(32)));
#pragma unroll 8
    for (int i = 0; i < m; ++i) {
      const float w = __shfl_sync(0xffffffffu, f, i);
      const float* o = part_of(c + i * kStep) + r * D + lane * kPer;
      float v[kPer];
      if (kPer == 4) {
        const float4 q = *reinterpret_cast<const float4*>(o);
        v[0] = q.x;
        v[1] = q.y;
        v[kPer - 2] = q.z;
        v[kPer - 1] = q.w;
      } else {
        const float2 q = *reinterpret_cast<const float2*>(o);
        v[0] = q.x;
        v[1] = q.y;
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j) x[j] = fmaf(v[j], w, x[j]);
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (WIDE) {  // (all warps of the block come here, or none: one row)
    __shared__ float shared_x[kPaWarps][D], shared_sum[kPaWarps];
#pragma unroll
    for (int i = 0; i < kPer; ++i) shared_x[warp][lane * kPer + i] = x[i];
    if (lane == 0) shared_sum[warp] = sum;
    __syncthreads();
    if (warp > 0) return;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = 0.f;
#pragma unroll
    for (int w = 0; w < kPaWarps; ++w) {
      sum += shared_sum[w];
#pragma unroll
      for (int i = 0; i < kPer; ++i) x[i] += shared_x[w][lane * kPer + i];
    }
  }
  write_row<kPer>(p, b, head, t, lane * kPer, base, sum, x);
}

template <int D, int NT>
cudaError_t launch_paged(const PagedParams& p, int num_sms,
                         cudaStream_t stream) {
  auto kern = paged_attention_kernel<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(
      kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PaCfg<D, NT>::kSmem);
  if (e != cudaSuccess) return e;
  const int rows = p.H / p.H_kv * p.T;
  const int tiles = (rows + 8 * NT - 1) / (8 * NT);
  const int grid = num_sms * kPaPerSm<D, NT>;
  kern<<<grid, kPaThreads, PaCfg<D, NT>::kSmem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  // few rows, which may each have many parts: a block per row (one sequence of
  // 8000 tokens and one K/V head: 20 us with a warp per row, 12.4 so)
  const int tile_rows = min(rows, 8 * NT);
  const bool wide =
      static_cast<int64_t>(p.B) * p.H_kv * tiles * tile_rows <= 4 * num_sms;
  cfg.gridDim = dim3(wide ? tile_rows : (tile_rows + kPaWarps - 1) / kPaWarps,
                     p.H_kv * tiles, p.B);
  cfg.blockDim = dim3(kPaThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return wide
             ? cudaLaunchKernelEx(&cfg, paged_join_kernel<D, NT, true>, p, grid)
             : cudaLaunchKernelEx(&cfg, paged_join_kernel<D, NT, false>, p,
                                  grid);
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

cudaError_t launch_paged_attention(const PagedParams& p, int num_sms,
                                   cudaStream_t stream) {
  // one tile of 8 query rows, or two where the group and the tokens fill them
  const bool two = static_cast<int64_t>(p.H / p.H_kv) * p.T > 8;
  if (p.D == 128)
    return two ? launch_paged<128, 2>(p, num_sms, stream)
               : launch_paged<128, 1>(p, num_sms, stream);
  if (p.D == 64)
    return two ? launch_paged<64, 2>(p, num_sms, stream)
               : launch_paged<64, 1>(p, num_sms, stream);
  return cudaErrorInvalidValue;
}

cudaError_t read_cache_error(int32_t out[4]) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_cache_error, 4 * sizeof(int32_t));
  if (e != cudaSuccess) return e;
  const int32_t zero[4] = {0, 0, 0, 0};
  return cudaMemcpyToSymbol(g_cache_error, zero, 4 * sizeof(int32_t));
}

}  // namespace bsm
