// What the kernels over the paged 8-bit cache share: conversions of e4m3 codes,
// the deal of a call's tokens over the CTAs, drafted tokens, and the kernel
// that joins the parts of rows whose keys were split.
#pragma once

#include <cstdint>

#include "bsm_internal.h"
#include "bsm_ptx.cuh"

namespace bsm {
namespace {

constexpr int kPaGroup = 16;  // tokens that share a page and its scales

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

// The high bit of every byte of w that is a NaN code (0x7f or 0xff).
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
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

// How the tokens are dealt out; X is a kernel's deal.  An item is (sequence,
// key/value head, tile of query rows: 8 or 16 in the kernel of few rows, 128 or
// 256 in the trees'); its work is its sequence's visible tokens in units of
// X::kUnit groups (64 tokens, a group for each warp; the trees' 128, a full
// step).  All units of all items, in order, are cut into equal runs, one per CTA,
// so that unequal lengths and few long sequences load every SM alike.  An item
// counts X::kRunCost units more than it has, before its first: what starting and
// ending a run costs (the kernel of few rows, 64 sequences of 300-12000 tokens:
// 160 us without, 140 with).  A CTA may start and end inside an item; then it
// leaves its part (o, m, l) in the workspace and a join kernel adds the parts up.
// The cut depends on the lengths and numbers of drafts alone, which both kernels
// read.
struct PaPlan {
  int len, lo;      // of one sequence: tokens, first visible one
  int drafts;       // query tokens that are there: its last ones
  int first_group;  // of 16 tokens
  int n_groups, n_units;
  int n_cost;  // n_units + X::kRunCost, or 0 without units
};

template <class X>
__device__ __forceinline__ PaPlan plan_of(const PagedParams& p, int b) {
  PaPlan s;
  s.len = min(max(p.lens[b], 0), p.max_pages * p.page_size);
  s.drafts = p.T;
  if (X::kTree) {
    s.drafts = min(p.T, s.len);
    if (p.n_new != nullptr) s.drafts = min(max(p.n_new[b], 0), s.drafts);
  }
  s.lo = p.window > 0 ? max(0, s.len - s.drafts - p.window + 1) : 0;
  s.first_group = s.lo / kPaGroup;
  s.n_groups = (s.len + kPaGroup - 1) / kPaGroup - s.first_group;
  s.n_units = (s.n_groups + X::kUnit - 1) / X::kUnit;
  if (X::kTree && s.drafts == 0) s.n_groups = s.n_units = 0;
  s.n_cost = s.n_units > 0 ? s.n_units + X::kRunCost : 0;
  return s;
}

// Drafted tokens.  Draft t of a sequence with n of them lies n - t places
// before its end; it sees every token before the drafts, and draft j where bit
// j of its row is set (without a tree: j <= t).  Bits of drafts that are not
// there count as clear.  Its depth, which gives its position behind the tokens
// before the drafts, is the number of drafts it sees, less itself; -1: it sees
// none, and its row is empty.
__device__ __forceinline__ uint32_t draft_bits(const PagedParams& p, int b,
                                               int t, int word, int n) {
  const int left = (p.tree != nullptr ? n : min(n, t + 1)) - 32 * word;
  const uint32_t there = left <= 0 ? 0u : left >= 32 ? ~0u : (1u << left) - 1u;
  // (past the drafts' words there may be no memory)
  if (p.tree == nullptr || there == 0u) return there;
  return p.tree[b * p.tree_sb + t * p.tree_st + word] & there;
}
__device__ __forceinline__ int draft_depth(const PagedParams& p, int b, int t,
                                           int n) {
  if (p.tree == nullptr) return t;
  int seen = 0;
  for (int w = 0; w * 32 < n; ++w) seen += __popc(draft_bits(p, b, t, w, n));
  return seen - 1;
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
template <class X>
__device__ __forceinline__ int lane_units(const PagedParams& p, int chunk,
                                          int64_t* n) {
  const int b0 = (threadIdx.x % 32) * chunk;
  int64_t sum = 0;
  for (int i = 0; i < chunk; ++i)
    if (b0 + i < p.B) sum += plan_of<X>(p, b0 + i).n_cost;
  *n = sum;
  return b0;
}

template <class X>
__device__ __forceinline__ PaScan scan_before(const PagedParams& p, int seq) {
  const int chunk = (p.B + 31) / 32;
  int64_t all = 0, head = 0;
  // interleaved: both sums, whatever the order
  for (int i = 0; i < chunk; ++i) {
    const int b = i * 32 + threadIdx.x % 32;
    if (b < p.B) {
      const int n = plan_of<X>(p, b).n_cost;
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
template <class X, class F>
__device__ __forceinline__ int find_sequence(const PagedParams& p, int per,
                                             F&& u_of, int64_t* start) {
  const int lane = threadIdx.x % 32;
  const int chunk = (p.B + 31) / 32;
  int64_t n;
  int b = lane_units<X>(p, chunk, &n);
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
          static_cast<int64_t>(plan_of<X>(p, b).n_cost) * per;
      if (u < at + m) break;
      at += m;
    }
  *start = __shfl_sync(0xffffffffu, at, owner);
  return __shfl_sync(0xffffffffu, b, owner);
}

// CTAs that get work: at least X::kLeast units each (two in the kernel of few
// rows, so that a CTA's first loads and its join are spread over more than one
// round of groups; one of the trees', which are twice as long).
template <class X>
__device__ __forceinline__ int64_t busy_ctas(int64_t units, int64_t grid) {
  const int64_t n = (units + X::kLeast - 1) / X::kLeast;
  return n < grid ? n : grid;
}

// Joins the parts of the items that were cut and writes the rows of sequences
// without tokens: a warp per query row, or (WIDE) a block, whose warps share
// the parts.
template <class X, int D, int R, bool WIDE>
__global__ void __launch_bounds__(128)
    paged_join_kernel(const PagedParams p, const int grid) {
  constexpr int kPer = D / 32, kPaWarps = 4;
  const int rows = p.H / p.H_kv * p.T;
  const int tiles = (rows + R - 1) / R;
  const int per = p.H_kv * tiles;
  const int b = blockIdx.z, item = blockIdx.y;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int r = WIDE ? blockIdx.x : blockIdx.x * kPaWarps + warp;
  const int rr = item % tiles * R + r;
  const PaScan scan = scan_before<X>(p, b);
  const int64_t units = scan.all * per;
  const int n = plan_of<X>(p, b).n_units;
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
  const int64_t busy = busy_ctas<X>(units, grid);
  // the CTAs that hold its first and last unit
  const int64_t u0 = scan.before * per +
                     static_cast<int64_t>(item) * (n + X::kRunCost) + X::kRunCost;
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

// The join's launch behind an attention kernel of `grid` CTAs whose items are
// tiles of R query rows.
template <class X, int D, int R>
cudaError_t launch_join(const PagedParams& p, int grid, int num_sms,
                        cudaStream_t stream) {
  const int rows = p.H / p.H_kv * p.T;
  const int tiles = (rows + R - 1) / R;
  cudaLaunchConfig_t cfg = {};
  // few rows, which may each have many parts: a block per row (one sequence of
  // 8000 tokens and one K/V head: 20 us with a warp per row, 12.4 so)
  const int tile_rows = min(rows, R);
  const bool wide =
      static_cast<int64_t>(p.B) * p.H_kv * tiles * tile_rows <= 4 * num_sms;
  cfg.gridDim = dim3(wide ? tile_rows : (tile_rows + 4 - 1) / 4,
                     p.H_kv * tiles, p.B);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return wide ? cudaLaunchKernelEx(&cfg, paged_join_kernel<X, D, R, true>, p,
                                   grid)
              : cudaLaunchKernelEx(&cfg, paged_join_kernel<X, D, R, false>, p,
                                   grid);
}

}  // namespace
}  // namespace bsm
