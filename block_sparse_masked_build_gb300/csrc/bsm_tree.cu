// Attention of many query rows over the paged 8-bit cache for sm_103a (GB300):
// trees of drafted tokens.  With G query heads per key/value head and T drafts
// a key serves G T rows, and from a few dozen on the work is a matrix product:
//     S = Q K^T,   P = 2^(z - m),   O += P V
// on the 5th-generation tensor core, 128 rows to a tile, one tile (R = 1) or
// two (R = 2) per CTA, 128 tokens at a time.
//
// The tensor core's operands are f16, which holds every e4m3 value: codes go
// from global memory through registers, where they are converted, into tiles
// of shared memory; a key's scale multiplies its column of S, a value's scale
// its tokens' rows of V.  Per 128 tokens and head dim 128 an SM reads 32 KB
// (1400 cycles at its share of the memory's rate), converts 32768 elements, and
// per tile of rows spends 1024 cycles on the tensor core and as many on the
// exponentials: one tile is bound by memory, two by the tensor core and the
// exponentials.
//
// Roles (512 threads, four warpgroups, registers shared out by setmaxnreg):
//   warp 0      deals the CTA's runs out in steps of up to 8 groups of 16
//               tokens: looks up pages and scales, up to 8 steps ahead.
//   warp 1      issues the MMAs (and owns the 512 TMEM columns).
//   converters  warpgroup 1, and with one tile of rows warpgroup 3 as well (one
//               takes the keys then, the other the values): the next 128
//               tokens' codes are on their way into registers while these are
//               converted.
//   score       warpgroup 2 (and 3 with two tiles): one thread per query row,
//               its TMEM lane: mask, running maximum, exponentials, P back to
//               TMEM over S, and at a run's end the row's result.
// TMEM columns: S and P [0, 128) and [128, 256), by turns with one tile, one
// for each of two; O [256, 256 + D), of a second tile from 384 on.
//
// A step's tokens go from a run's end to its start: the drafts come first, and
// with a bias that falls with the distance the maximum is met early.
#include <cstdint>

#include "bsm_internal.h"
#include "bsm_paged.cuh"
#include "bsm_ptx.cuh"

namespace bsm {

// Error record: [0] code (1: a wait gave up, then block, role, phase; 2: a
// page table or length out of range, then sequence, page slot, value).
__device__ int g_tree_error[4];

namespace {

constexpr int kTcThreads = 512;
constexpr int kTcRows = 128;    // of a tile: one accumulator
constexpr int kTcTokens = 128;  // of a full step
constexpr int kTcGroups = kTcTokens / kPaGroup;
constexpr int kTcSteps = 8;     // ring of steps
constexpr uint32_t kTcTmem = 512;
constexpr int kTreeFewRows = 16;  // see tree_tiles
constexpr int kRolePlan = 1, kRoleMma = 2, kRoleConvert = 3, kRoleScore = 4;
// P is scaled by 2^9 before it becomes f16, whose smallest number is 2^-24: a
// key's weight is lost below 2^-34 of the largest (as in the attention of
// single tokens).  The reference m may lie up to 2^6 below the running maximum
// before O is rescaled; 2^15 still fits f16.
constexpr float kTcUpLog2 = 9.f, kTcRescaleLog2 = 6.f;

// The deal: a unit is a full step.
struct TcDeal {
  static constexpr bool kTree = true;
  static constexpr int kUnit = kTcGroups, kRunCost = 3, kLeast = 1;
};

template <int D, int R>
struct TcCfg {
  static constexpr int kTile = kTcTokens * D * 2;  // Q, K or V in f16
  // K and V tiles in turn: what fits beside Q, with two steps at least
  static constexpr int kSlots = R == 1 ? 5 : 4;
  static constexpr int kOffKv = R * kTile;
  static constexpr int kOffCtl = kOffKv + kSlots * kTile;
  // registers per thread: warpgroup 0, converters, score
  static constexpr uint32_t kRegsPlan = 64, kRegsConvert = R == 1 ? 120 : 96,
                            kRegsScore = R == 1 ? 208 : 176;
  static_assert(kRegsPlan + (3 - R) * kRegsConvert + R * kRegsScore <= 512,
                "register file");
};

// Up to 128 tokens of a run, newest step first.
struct TcStep {
  int32_t groups;    // 1 .. 8 groups of 16 tokens from tok0 on; 0: the end
  int32_t tok0;
  int32_t first, last;  // of its run
  int32_t plain;     // 8 groups, and every row sees every token
  float v_ref;       // V's tile, and so O, is in units of this scale
  // of the run
  int32_t b, hkv, row0, part;  // part: -1 whole, else its slot in the workspace
  int32_t len, lo, n;          // tokens, first visible one, drafts
  int32_t pad;
  float k_scale[kTcGroups];
  float v_mul[kTcGroups];      // scale / v_ref
  int64_t off[kTcGroups];      // of the group's codes; -1: page out of range
};

struct TcCtl {
  uint64_t step_full[kTcSteps], step_empty[kTcSteps];
  uint64_t kv_full[5], kv_empty[5];
  uint64_t q_full[2], s_full[2], p_full[2], pv_done[2], o_free[2], mma_done;
  uint32_t tmem;
  int abort;
  TcStep steps[kTcSteps];
  // of steps that are not plain, by step modulo 4: columns' positions, and the
  // NaN codes of V (16 dims per entry), with the step's number + 1 where there
  // are any.  A slot is written again four steps later, when the tensor core
  // has long taken the P that the rows made with it.
  int32_t pos[4][kTcTokens];
  uint16_t nan[4][kTcTokens][8];
  uint32_t nan_step[4];
};

struct TcParams {
  PagedParams p;
  uint64_t timeout_ns;
};

__device__ __forceinline__ void tc_record(int code, int a, int b, int c) {
  if (atomicCAS(&g_tree_error[0], 0, code) == 0) {
    g_tree_error[1] = a;
    g_tree_error[2] = b;
    g_tree_error[3] = c;
  }
}

// Warp-wide bounded wait (see mbar_wait), alike in every lane.
__device__ __forceinline__ bool tc_wait(const TcParams& t, TcCtl* c,
                                        uint64_t* bar, uint32_t parity,
                                        int role, int phase) {
  const bool ok = __all_sync(
      0xffffffffu, mbar_wait(bar, parity, &c->abort, t.timeout_ns));
  if (!ok && threadIdx.x % 32 == 0) tc_record(1, blockIdx.x, role, phase);
  return ok;
}

__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if (threadIdx.x % 32 == 0) mbar_arrive(bar);
}

__device__ __forceinline__ float pow2(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// ----------------------------------------------------------------- planner

// Value scales of a step lie within these factors of its unit: a code times
// the ratio is then exact in f16 (for ratios that are powers of two), 2^-19 its
// smallest and 448 * 2^6 its largest number.  Pages further apart go in steps
// of their own, between which O moves to the other unit.
__device__ __forceinline__ bool near_scale(float s, float ref) {
  const float r = s / ref;
  return r >= 0x1p-10f && r <= 0x1p6f;
}

// One run: groups [g0, g1) of its sequence's plan.
template <int D, int R>
__device__ __forceinline__ bool plan_run(const TcParams& t, TcCtl* c, int b,
                                         const PaPlan& plan, int hkv, int row0,
                                         int g0, int g1, int part,
                                         uint32_t& step) {
  const PagedParams& p = t.p;
  const int lane = threadIdx.x % 32;
  const int* table = p.table + static_cast<int64_t>(b) * p.table_stride;
  const int base = plan.len - plan.drafts;
  float ref = 0.f;
  for (int top = g1; top > g0; top -= 32) {  // lane i: group top - 1 - i
    const int g = top - 1 - lane;
    const int tok = (plan.first_group + g) * kPaGroup;
    float ks = 0.f, vs = 0.f;
    int64_t off = -1;
    if (g >= g0) {
      const int slot = tok >> p.page_shift;
      const int pid = table[slot];
      if (static_cast<uint32_t>(pid) < static_cast<uint32_t>(p.num_pages)) {
        const int64_t block = static_cast<int64_t>(pid) * p.H_kv + hkv;
        ks = p.k_scale[block];
        vs = p.v_scale[block];
        off = ((block << p.page_shift) + (tok & (p.page_size - 1))) * D;
      } else {
        tc_record(2, b, slot, pid);
      }
    }
    const int here = min(32, top - g0);
    for (int at = 0; at < here;) {
      int n = min(kTcGroups, here - at);
      const bool mine = lane >= at && lane < at + n && off >= 0;
      const unsigned some = __ballot_sync(0xffffffffu, mine);
      unsigned far = __ballot_sync(0xffffffffu, mine && !near_scale(vs, ref));
      if (far & (1u << at) || (ref == 0.f && some != 0)) {
        ref = __shfl_sync(0xffffffffu, vs, __ffs(some) - 1);
        far = __ballot_sync(0xffffffffu, mine && !near_scale(vs, ref));
        // (a scale that is near nothing, itself included, goes alone)
        far &= ~(1u << (__ffs(some) - 1));
      }
      if (far != 0) n = __ffs(far) - 1 - at;
      const uint32_t slot = step % kTcSteps;
      if (!tc_wait(t, c, &c->step_empty[slot], ((step / kTcSteps) & 1) ^ 1,
                   kRolePlan, 0))
        return false;
      TcStep& s = c->steps[slot];
      if (lane >= at && lane < at + n) {
        const int i = at + n - 1 - lane;  // ascending tokens
        s.k_scale[i] = ks;
        s.v_mul[i] = off >= 0 && ref != 0.f ? vs / ref : 0.f;
        s.off[i] = off;
      }
      const int tok0 = (plan.first_group + top - at - n) * kPaGroup;
      const unsigned there = __ballot_sync(0xffffffffu, off >= 0);
      if (lane == 0) {
        s.groups = n;
        s.tok0 = tok0;
        s.first = top == g1 && at == 0;
        s.last = top - at - n == g0;
        s.plain = n == kTcGroups && tok0 + kTcTokens <= base &&
                  tok0 >= plan.lo && (there >> at & 0xffu) == 0xffu &&
                  (p.window <= 0 || plan.len - 1 - tok0 < p.window);
        s.v_ref = ref != 0.f ? ref : 1.f;
        s.b = b;
        s.hkv = hkv;
        s.row0 = row0;
        s.part = part;
        s.len = plan.len;
        s.lo = plan.lo;
        s.n = plan.drafts;
      }
      warp_arrive(&c->step_full[slot]);
      ++step;
      at += n;
    }
  }
  return true;
}

template <int D, int R>
__device__ __forceinline__ void plan_role(const TcParams& t, TcCtl* c) {
  using X = TcDeal;
  const PagedParams& p = t.p;
  const int lane = threadIdx.x % 32;
  const int rows = p.H / p.H_kv * p.T;
  const int tiles = (rows + R * kTcRows - 1) / (R * kTcRows);
  const int per = p.H_kv * tiles;
  if (blockIdx.x == 0)
    for (int b = lane; b < p.B; b += 32) {
      const int len = p.lens[b];
      const PaPlan plan = plan_of<X>(p, b);
      if (len != plan.len) tc_record(2, b, -1, len);
      if (p.n_new != nullptr && p.n_new[b] != plan.drafts)
        tc_record(2, b, -1, p.n_new[b]);
    }
  __syncwarp();
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
  uint32_t step = 0;
  bool ok = true;
  while (ok && b >= 0 && u < end) {
    const PaPlan plan = plan_of<X>(p, b);
    const int64_t row_cost = static_cast<int64_t>(plan.n_cost) * per;
    if (u >= start + row_cost) {
      start += row_cost;
      ++b;
      continue;
    }
    const int64_t within = u - start;
    const int item = static_cast<int>(within / plan.n_cost);
    const int off =
        static_cast<int>(within - static_cast<int64_t>(item) * plan.n_cost);
    const int n = static_cast<int>(
        min(static_cast<int64_t>(plan.n_cost - off), end - u));
    // units [r0, r1) of the item
    const int r0 = max(off - X::kRunCost, 0), r1 = off + n - X::kRunCost;
    if (r1 > r0) {
      int part = -1;
      if (r0 > 0 || r1 < plan.n_units)  // slot 0: an earlier CTA has the start
        part = blockIdx.x * 2 + (r0 > 0 ? 0 : 1);
      ok = plan_run<D, R>(t, c, b, plan, item / tiles,
                          item % tiles * (R * kTcRows), r0 * kTcGroups,
                          min(r1 * kTcGroups, plan.n_groups), part, step);
    }
    u += n;
  }
  if (!ok) return;
  const uint32_t slot = step % kTcSteps;  // the end
  if (!tc_wait(t, c, &c->step_empty[slot], ((step / kTcSteps) & 1) ^ 1,
               kRolePlan, 1))
    return;
  if (lane == 0) c->steps[slot].groups = 0;
  warp_arrive(&c->step_full[slot]);
}

// -------------------------------------------------------------- converters

// The codes of one step's keys or values on their way: the thread's 16-byte
// pieces.  A group of 16 tokens is 16 D bytes in a row: at D = 128 a piece per
// thread of the warpgroup, at 64 one per thread of half of it.
template <int D>
struct TcLoad {
  static constexpr int kPieces = D / 16;
  uint4 x[kPieces];
};

template <int D>
__device__ __forceinline__ void load_codes(const TcStep& s,
                                           const uint8_t* pages,
                                           TcLoad<D>& l) {
  const int i = threadIdx.x % 128;
#pragma unroll
  for (int k = 0; k < TcLoad<D>::kPieces; ++k) {
    const int g = D == 128 ? k : 2 * k + i / 64;
    const int at = D == 128 ? i : i % 64;
    l.x[k] = make_uint4(0u, 0u, 0u, 0u);
    if (g < s.groups) {
      const int64_t off = s.off[g];
      if (off >= 0)
        l.x[k] = __ldcs(
            reinterpret_cast<const uint4*>(pages + off + at * 16));
    }
  }
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// What a step that is not plain needs before its codes are converted: tokens
// that are no sequence's become zeros, and so do NaN codes of values, which are
// noted, as a row that does not see them must not meet 0 * NaN; and the
// positions of its columns.
template <int D>
__device__ __forceinline__ void clean_codes(const PagedParams& p, TcCtl* c,
                                            const TcStep& s, uint32_t step,
                                            bool values, TcLoad<D>& l) {
  constexpr int kPer = D / 16, kRows = 128 / kPer;
  const int i = threadIdx.x % 128;
  const int piece = i % kPer, row = i / kPer;
#pragma unroll
  for (int k = 0; k < TcLoad<D>::kPieces; ++k) {
    const int tr = row + k * kRows, tok = s.tok0 + tr;
    if (tok < s.lo || tok >= s.len) l.x[k] = make_uint4(0u, 0u, 0u, 0u);
    if (values) {
      uint32_t* w = reinterpret_cast<uint32_t*>(&l.x[k]);
      uint32_t found = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t n = nan_codes(w[j]) >> 7;  // one bit per byte
        w[j] &= ~(n * 0xffu);
        // the four bits 0, 8, 16, 24 next to each other
        found |= ((n * 0x00204081u >> 21) & 0xfu) << (4 * j);
      }
      c->nan[step % 4][tr][piece] = static_cast<uint16_t>(found);
      if (found != 0) c->nan_step[step % 4] = step + 1;
    }
  }
  if (values && (p.window > 0 || (p.mod.kind & kModBias))) {
    const int tok = s.tok0 + i, base = s.len - s.n;
    c->pos[step % 4][i] = tok >= base && tok < s.len
                              ? base + draft_depth(p, s.b, tok - base, s.n)
                              : tok;
  }
}

template <int OFF>
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y,
                                       uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0+%5], {%1, %2, %3, %4};" ::"r"(a), "r"(x),
               "r"(y), "r"(z), "r"(w), "n"(OFF)
               : "memory");
}

// Piece K of a thread and the ones behind it into the f16 tile (see
// convert_role); a, b: where the two halves of piece 0 go.
template <int D, int K>
__device__ __forceinline__ void store_codes(const TcStep& s, bool values,
                                            bool flip, uint32_t a, uint32_t b,
                                            const TcLoad<D>& l) {
  constexpr int kRows = 2048 / D;
  const uint32_t w[4] = {l.x[K].x, l.x[K].y, l.x[K].z, l.x[K].w};
  uint32_t h[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    h[2 * j] = e4m3x2_to_f16x2(w[j]);
    h[2 * j + 1] = e4m3x2_to_f16x2_hi(w[j]);
  }
  if (values) {
    const int g = D == 128 ? K : 2 * K + threadIdx.x % 128 / 64;
    const float m = s.v_mul[g];
    if (m != 1.f) {
      const uint32_t mm = pack_f16x2(m, m);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = hmul2(h[j], mm);
    }
  }
  constexpr int off = K * kRows * 128;
  sts128<off>(a, flip ? h[4] : h[0], flip ? h[5] : h[1], flip ? h[6] : h[2],
              flip ? h[7] : h[3]);
  sts128<off>(b, flip ? h[0] : h[4], flip ? h[1] : h[5], flip ? h[2] : h[6],
              flip ? h[3] : h[7]);
  if constexpr (K + 1 < TcLoad<D>::kPieces)
    store_codes<D, K + 1>(s, values, flip, a, b, l);
}

__device__ __forceinline__ bool wait_step(const TcParams& t, TcCtl* c,
                                          uint32_t step, int role) {
  return tc_wait(t, c, &c->step_full[step % kTcSteps], (step / kTcSteps) & 1,
                 role, 9);
}

// A converter warpgroup: with one tile of rows the keys (which = 0) or the
// values (1) of every step, with two tiles both in turn.  The codes of the half
// step after the one in hand are on their way meanwhile.  (One copy of the code
// for keys and values, as the roles together must fit the SM's instruction
// cache: with a copy for each, unrolled by two, and the MMAs unrolled, the
// kernel waited for instructions, 373 us on 32 sequences of 300-12000 tokens
// and 16 drafts.)
//
// Tiles are rows of 64 elements (128 bytes) per token, two such blocks at D =
// 128, in the 128-byte swizzle.  Lanes of the upper block store their second
// half first: eight lanes then touch eight different 16-byte columns.
template <int D, int R>
__device__ __forceinline__ void convert_role(const TcParams& t, TcCtl* c,
                                             uint32_t kv, int which) {
  using C = TcCfg<D, R>;
  constexpr int kPer = D / 16;
  const int i = threadIdx.x % 128, piece = i % kPer;
  const uint32_t row = i / kPer;
  const bool flip = D == 128 && piece >= 4;
  const uint32_t line =
      kv + (D == 128 ? (piece >> 2) * (kTcTokens * 128) : 0) + row * 128;
  const uint32_t chunk = ((2 * piece) & 7) | (flip ? 1u : 0u);
  const uint32_t at_a = line + ((chunk ^ (row & 7)) << 4);
  const uint32_t at_b = line + ((chunk ^ 1u ^ (row & 7)) << 4);
  bool values = which != 0;
  TcLoad<D> now, next;
  if (!wait_step(t, c, 0, kRoleConvert) || c->steps[0].groups == 0) return;
  load_codes<D>(c->steps[0], values ? t.p.v : t.p.k, now);
#pragma unroll 1
  for (uint32_t step = 0;;) {
    // the half step behind this one
    uint32_t step2 = step;
    bool values2 = values, more = true;
    if (R == 2) values2 = !values;
    if (R == 1 || values) {
      ++step2;
      if (!wait_step(t, c, step2, kRoleConvert)) return;
      more = c->steps[step2 % kTcSteps].groups != 0;
    }
    if (more)
      load_codes<D>(c->steps[step2 % kTcSteps], values2 ? t.p.v : t.p.k, next);
    const TcStep& s = c->steps[step % kTcSteps];
    const uint32_t h = 2 * step + (values ? 1 : 0);
    const uint32_t slot = h % C::kSlots;
    if (!tc_wait(t, c, &c->kv_empty[slot], ((h / C::kSlots) & 1) ^ 1,
                 kRoleConvert, values))
      return;
    if (__builtin_expect(!s.plain, 0))
      clean_codes<D>(t.p, c, s, step, values, now);
    store_codes<D, 0>(s, values, flip, at_a + slot * C::kTile,
                      at_b + slot * C::kTile, now);
    fence_proxy_async();
    warp_arrive(&c->kv_full[slot]);
    if (R == 1 || values) warp_arrive(&c->step_empty[step % kTcSteps]);
    if (!more) return;
    now = next;
    step = step2;
    values = values2;
  }
}

// --------------------------------------------------------------------- MMA

// Instruction descriptor as idesc_bf16_f32, with f16 operands.
__device__ __forceinline__ constexpr uint32_t idesc_f16(int N, bool mn_major) {
  return (1u << 4) | ((mn_major ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(kTcRows >> 4) << 24);
}

template <int D, int R>
__device__ __forceinline__ void mma_role(const TcParams& t, TcCtl* c,
                                         uint32_t smem, uint32_t tmem) {
  using C = TcCfg<D, R>;
  constexpr uint32_t kUnits = C::kTile >> 4;
  const uint64_t dq = sdesc_sw128(smem, 16, 1024);
  const uint64_t dk = sdesc_sw128(smem + C::kOffKv, 16, 1024);
  const uint64_t dv = sdesc_sw128(smem + C::kOffKv, kTcTokens * 128, 1024);
  bool ok = true;
  uint32_t runs = 0;  // begun
  int groups = 0, groups_before = 0;  // of the step and of the one before
  bool first = false, first_before = false;
  // buffer of tile r at a step, and how often it was used before
  auto buf = [](uint32_t step, int r) { return R == 2 ? r : int(step & 1); };
  auto use = [](uint32_t step) { return R == 2 ? step : step >> 1; };
  auto wait_kv = [&](uint32_t h) {
    return tc_wait(t, c, &c->kv_full[h % C::kSlots], (h / C::kSlots) & 1,
                   kRoleMma, 2);
  };
#pragma unroll 1
  for (uint32_t step = 0; ok; ++step) {
    ok = wait_step(t, c, step, kRoleMma);
    if (!ok) break;
    const TcStep& s = c->steps[step % kTcSteps];
    groups_before = groups;
    first_before = first;
    groups = s.groups;
    first = s.first != 0;
    const bool more = groups != 0;
    warp_arrive(&c->step_empty[step % kTcSteps]);
    // One tile: S goes ahead of the P V before it, in the other buffer, while
    // that P is in the making.  Two tiles share the steps' S and P in turn: S
    // goes behind the P V that reads its columns (MMAs of one thread run in
    // the order they were issued).  A run's first S waits for its query, which
    // the rows load when the run before is written out.
    const bool ahead = R == 1 && !first;
#pragma unroll 1
    for (int turn = 0; turn < 2 * R; ++turn) {
      const int r = turn >> 1;
      if (((turn & 1) != 0) != ahead) {  // S_r = Q_r K^T
        if (!more) continue;
        if (r == 0) ok = wait_kv(2 * step);
        if (ok && first)
          ok = tc_wait(t, c, &c->q_full[r], runs & 1, kRoleMma, 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a = dq + r * kUnits;
        const uint64_t b = dk + (2 * step) % C::kSlots * kUnits;
        const uint32_t idesc = idesc_f16(groups * kPaGroup, false);
        const uint32_t d = tmem + buf(step, r) * 128;
#pragma unroll 2
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * (kTcTokens * 128 / 16) + (k & 3) * 2;
          mma_ss_elect(d, a + off, b + off, idesc, k > 0);
        }
        mma_commit_elect(&c->s_full[buf(step, r)]);
        if (r == R - 1)
          mma_commit_elect(&c->kv_empty[(2 * step) % C::kSlots]);
      } else {  // O_r (+)= P_r V of the step before
        if (step == 0) continue;
        const uint32_t before = step - 1, h = 2 * before + 1;
        const int bf = buf(before, r);
        if (r == 0) ok = wait_kv(h);
        if (ok)
          ok = tc_wait(t, c, &c->p_full[bf], use(before) & 1, kRoleMma, 3);
        // run k (k = runs - 1 here) finds O free when k runs were written out
        if (ok && first_before)
          ok = tc_wait(t, c, &c->o_free[r], runs & 1, kRoleMma, 4);
        if (!ok) break;
        tc_fence_after();
        const uint64_t b = dv + h % C::kSlots * kUnits;
        constexpr uint32_t idesc = idesc_f16(D, true);
#pragma unroll 2
        for (int k = 0; k < groups_before; ++k)
          mma_ts_elect(tmem + 256 + r * 128, tmem + bf * 128 + k * 8,
                       b + k * (kPaGroup * 128 / 16), idesc,
                       k > 0 || !first_before);
        mma_commit_elect(&c->pv_done[r]);
        if (r == R - 1) mma_commit_elect(&c->kv_empty[h % C::kSlots]);
      }
    }
    if (!more) break;
    if (first) ++runs;
  }
  // every MMA issued above has completed once this arrives
  __syncwarp();
  mma_commit_elect(&c->mma_done);
  if (threadIdx.x % 32 == 0 && !mbar_wait_drain(&c->mma_done, 0, t.timeout_ns))
    tc_record(1, blockIdx.x, kRoleMma, 8);
  __syncwarp();
}

// ------------------------------------------------------------------- score

// A row's query into its tile: f16, scaled so that the row's largest magnitude
// becomes [1, 2) (f16 then keeps bf16's 8 bits of every element above 2^-17 of
// it, and 2^-25 of it of the rest).  Returns the factor that undoes it.
template <int D>
__device__ __forceinline__ float load_query(const uint16_t* src, bool live,
                                            bool negate, uint32_t tile, int r) {
  uint32_t w[D / 2];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (live) v = *reinterpret_cast<const uint4*>(src + 8 * i);
    w[4 * i] = v.x;
    w[4 * i + 1] = v.y;
    w[4 * i + 2] = v.z;
    w[4 * i + 3] = v.w;
  }
#pragma unroll
  for (int i = 0; i < D / 2; ++i) top = max_u16x2(top, w[i] & 0x7fff7fffu);
  top = max(top & 0xffffu, top >> 16);
  // exponents at the ends of the range stay finite factors
  const int e = min(max(static_cast<int>(top >> 7) - 127, -120), 120);
  const float down = negate ? -pow2(-e) : pow2(-e);
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = w[4 * i + j];
      h[j] = pack_f16x2(__uint_as_float(x << 16) * down,
                        __uint_as_float(x & 0xffff0000u) * down);
    }
    const uint32_t at = tile + (i >> 3) * (kTcRows * 128) + r * 128 +
                        (((i & 7) ^ (r & 7)) << 4);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at),
                 "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                 : "memory");
  }
  return pow2(e);
}

// The columns of a step that are not plain that a row sees, 32 to a word.
__device__ __forceinline__ uint32_t visible(const PagedParams& p,
                                            const TcStep& s, int word, int t) {
  const int base = s.len - s.n;
  const int t0 = s.tok0 + 32 * word;
  // tokens [lo, len) of the step's groups
  const int lo = s.lo - t0, hi = min(s.len, s.tok0 + s.groups * kPaGroup) - t0;
  uint32_t keep = hi <= 0 ? 0u : hi >= 32 ? ~0u : (1u << hi) - 1u;
  if (lo > 0) keep = lo >= 32 ? 0u : keep & (~0u << lo);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (2 * word + i < s.groups && s.off[2 * word + i] < 0)
      keep &= ~(0xffffu << (16 * i));
  const int d0 = t0 - base;  // draft of the word's first column
  if (d0 > -32) {
    uint32_t bits;
    if (d0 >= 0) {
      const int w = d0 / 32, sh = d0 % 32;
      bits = draft_bits(p, s.b, t, w, s.n) >> sh;
      if (sh > 0 && (w + 1) * 32 < s.n)
        bits |= draft_bits(p, s.b, t, w + 1, s.n) << (32 - sh);
    } else {
      bits = (draft_bits(p, s.b, t, 0, s.n) << -d0) | ((1u << -d0) - 1u);
    }
    keep &= bits;
  }
  return keep;
}

// cap * tanh(x / cap) of a row's scores S = q.k, in log2 units: polynomials
// where the warp's scores allow them (|y| <= 0.5, <= 1.2), else exponentials.
__device__ __forceinline__ void cap_scores(const ScoreMod& m, float* s) {
  float a0 = 0.f, a1 = 0.f;
#pragma unroll
  for (int c = 0; c < kTcTokens; c += 4) {
    a0 = fmax3_abs_nan(a0, s[c], s[c + 1]);
    a1 = fmax3_abs_nan(a1, s[c + 2], s[c + 3]);
  }
  const float top = fmax3_abs_nan(a0, a1, a1);
  if (__all_sync(0xffffffffu, top <= m.poly_max)) {
#pragma unroll
    for (int c = 0; c < kTcTokens; c += 2) {
      float h0, h1;
      poly_sq2<4>(h0, h1, s[c], s[c + 1], m.poly);
      fmul2v(s[c], s[c + 1], s[c], s[c + 1], h0, h1);
    }
  } else if (__all_sync(0xffffffffu, top <= m.wide_max)) {
#pragma unroll
    for (int c = 0; c < kTcTokens; c += 2) {
      float h0, h1;
      poly_sq2<7>(h0, h1, s[c], s[c + 1], m.wide);
      fmul2v(s[c], s[c + 1], s[c], s[c + 1], h0, h1);
    }
  } else {
    // tanh(y) = 1 - 2 / (1 + e^(2 y)), off by 2^-23 of the cap
    const float k2 = -2.f * m.cap_log2;
#pragma unroll
    for (int c = 0; c < kTcTokens; ++c) {
      const float y = s[c] * m.cap_e;
      float z = fmaf(k2, rcp_approx(ex2_approx(y) + 1.f), m.cap_log2);
      if (m.cap_log2 > 300.f) {  // where that would show in the logits
        const float h = y * 0.34657359f, h2 = h * h;
        const float q = fmaf(h2, fmaf(h2, fmaf(h2, -0.04439273843f,
                                               0.1318993943f),
                                      -0.3332628423f),
                             0.999999451f);
        z = h2 <= 0.25f ? m.cap_log2 * (h * q) : z;
      }
      s[c] = z;
    }
  }
}

template <int D, int R, bool MOD>
__device__ __forceinline__ void score_role(const TcParams& tp, TcCtl* c,
                                           uint32_t smem, uint32_t tmem,
                                           const int t) {
  using C = TcCfg<D, R>;
  const PagedParams& p = tp.p;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int quarter = warp % 4;
  const int r = quarter * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t o_addr = tmem + lane_off + 256 + t * 128;
  const float NEG_INF = __int_as_float(0xff800000);
  const int G = p.H / p.H_kv, rows = G * p.T;
  const bool capped = MOD && (p.mod.kind & kModCap);
  const bool biased = MOD && (p.mod.kind & kModBias);
  const bool negate = !capped && p.scale_x < 0.f;
  uint32_t pv = 0;  // P tiles given to the tensor core
  // of the run
  float q_mul = 0.f, slope2 = 0.f, m_used = NEG_INF, l_sum = 0.f, ref = 1.f;
  int row = 0, tq = 0, pos = -1;
  uint32_t nans[D / 32];
  uint32_t run_pv = 0;
  for (uint32_t step = 0;; ++step) {
    if (!wait_step(tp, c, step, kRoleScore)) return;
    const TcStep& s = c->steps[step % kTcSteps];
    if (s.groups == 0) return;
    if (s.first) {
      row = s.row0 + t * kTcRows + r;
      const bool live = row < rows;
      const int at = live ? row : 0;
      const int head = s.hkv * G + at / p.T;
      tq = at % p.T;
      const float up = load_query<D>(
          p.q + s.b * p.q_sb + head * p.q_sh + tq * p.q_ss, live, negate,
          smem + t * C::kTile, r);
      fence_proxy_async();
      mbar_arrive(&c->q_full[t]);
      // with a cap: to S itself; else to log2 units
      q_mul = capped ? up : up * fabsf(p.scale_x);
      slope2 = biased ? p.mod.slopes[head] * 1.4426950408889634f : 0.f;
      const int depth =
          live && tq < s.n ? draft_depth(p, s.b, tq, s.n) : -1;
      pos = depth >= 0 ? s.len - s.n + depth : -1;
      m_used = NEG_INF;
      l_sum = 0.f;
      ref = s.v_ref;
      run_pv = 0;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) nans[i] = 0u;
    }
    const int buf = R == 2 ? t : static_cast<int>(step & 1);
    const uint32_t use = R == 2 ? step : step >> 1;
    const uint32_t s_addr = tmem + lane_off + buf * 128;
    uint32_t keep[4] = {~0u, ~0u, ~0u, ~0u};
    if (__builtin_expect(!s.plain, 0)) {
      // positions and NaN codes come with the values
      const uint32_t h = 2 * step + 1;
      if (!tc_wait(tp, c, &c->kv_full[h % C::kSlots], (h / C::kSlots) & 1,
                   kRoleScore, 5))
        return;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        keep[w] = pos >= 0 ? visible(p, s, w, tq) : 0u;
        if (p.window > 0)
#pragma unroll 4
          for (int j = 0; j < 32; ++j)
            if (pos - c->pos[step % 4][32 * w + j] >= p.window)
              keep[w] &= ~(1u << j);
      }
      if (c->nan_step[step % 4] == step + 1) {
        // values that are NaN: a row that sees one has NaN in that place
#pragma unroll
        for (int w = 0; w < 4; ++w)
          for (uint32_t k = keep[w]; k != 0; k &= k - 1) {
            const uint16_t* n = c->nan[step % 4][32 * w + __ffs(k) - 1];
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
              nans[i] |= *reinterpret_cast<const uint32_t*>(n + 2 * i);
          }
      }
    }
    float f[kTcGroups];
#pragma unroll
    for (int g = 0; g < kTcGroups; ++g) f[g] = q_mul * s.k_scale[g];
    if (!tc_wait(tp, c, &c->s_full[buf], use & 1, kRoleScore, 1)) return;
    tc_fence_after();
    uint32_t raw[kTcTokens];
#pragma unroll
    for (int q = 0; q < kTcTokens / 32; ++q)
      tmem_ld32(s_addr + q * 32, raw + q * 32);
    tmem_ld_wait();
    float* x = reinterpret_cast<float*>(raw);
    if (MOD || !s.plain) {
#pragma unroll
      for (int j = 0; j < kTcTokens; j += 2)
        fmul2(x[j], x[j + 1], x[j], x[j + 1], f[j / kPaGroup]);
#pragma unroll
      for (int g = 0; g < kTcGroups; ++g) f[g] = 1.f;
    }
    if (MOD) {
      // columns that are not seen may hold anything; 0 costs the cap nothing
      if (!s.plain)
#pragma unroll
        for (int j = 0; j < kTcTokens; ++j)
          if (!(keep[j / 32] >> (j % 32) & 1u)) x[j] = 0.f;
      if (capped) cap_scores(p.mod, x);
      if (biased) {
        if (s.plain) {
          const float d0 = static_cast<float>(s.tok0 - pos);
#pragma unroll
          for (int j = 0; j < kTcTokens; ++j)
            x[j] = fmaf(slope2, d0 + static_cast<float>(j), x[j]);
        } else {
#pragma unroll
          for (int j = 0; j < kTcTokens; ++j)
            x[j] = fmaf(-slope2,
                        fabsf(static_cast<float>(pos - c->pos[step % 4][j])),
                        x[j]);
        }
      }
    }
    if (__builtin_expect(!s.plain, 0)) {
#pragma unroll
      for (int j = 0; j < kTcTokens; ++j)
        if (!(keep[j / 32] >> (j % 32) & 1u)) x[j] = NEG_INF;
    }
    // the running maximum
    float top = NEG_INF;
#pragma unroll
    for (int g = 0; g < kTcGroups; ++g) {
      const float* v = x + g * kPaGroup;
      const float a = fmax3(v[0], v[1], v[2]), b = fmax3(v[3], v[4], v[5]);
      const float d = fmax3(v[6], v[7], v[8]), e = fmax3(v[9], v[10], v[11]);
      const float m = fmax3(fmax3(a, b, d), fmax3(e, v[12], v[13]),
                            fmaxf(v[14], v[15]));
      top = fmaxf(top, m * f[g]);
    }
    float scale_o = 1.f;
    if (top > m_used + kTcRescaleLog2) {
      const float alpha = ex2_approx(m_used - top);  // 0 from -inf
      l_sum *= alpha;
      scale_o = alpha;
      m_used = top;
    }
    if (s.v_ref != ref) {
      scale_o *= ref / s.v_ref;
      ref = s.v_ref;
    }
    // 2^9 goes along with P and the sums
    const float add = m_used == NEG_INF ? kTcUpLog2 : kTcUpLog2 - m_used;
    float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
    for (int q = 0; q < kTcTokens / 32; ++q) {
      uint32_t pk[16];
#pragma unroll
      for (int j = 32 * q; j < 32 * q + 32; j += 4) {
        float x0, x1, x2, x3;
        ffma2(x0, x1, x[j], x[j + 1], f[j / kPaGroup], add);
        ffma2(x2, x3, x[j + 2], x[j + 3], f[j / kPaGroup], add);
        const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
        const float p2 = ex2_approx(x2), p3 = ex2_approx(x3);
        fadd2(l0, l1, l0, l1, p0, p1);
        fadd2(l2, l3, l2, l3, p2, p3);
        pk[(j & 31) / 2] = pack_f16x2(p0, p1);
        pk[(j & 31) / 2 + 1] = pack_f16x2(p2, p3);
      }
      tmem_st16(s_addr + q * 16, pk);
    }
    l_sum += (l0 + l1) + (l2 + l3);
    if (__any_sync(0xffffffffu, scale_o != 1.f) && run_pv > 0) {
      if (!tc_wait(tp, c, &c->pv_done[t], (pv - 1) & 1, kRoleScore, 2)) return;
      tc_fence_after();
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        uint32_t o[32];
        tmem_ld32(o_addr + q * 32, o);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j)
          o[j] = __float_as_uint(__uint_as_float(o[j]) * scale_o);
        tmem_st32(o_addr + q * 32, o);
      }
    }
    tmem_st_wait();
    tc_fence_before();
    mbar_arrive(&c->p_full[buf]);
    ++pv;
    ++run_pv;
    if (!s.last) {
      warp_arrive(&c->step_empty[step % kTcSteps]);
      continue;
    }
    // ---- the row's result, or its part of it
    if (!tc_wait(tp, c, &c->pv_done[t], (pv - 1) & 1, kRoleScore, 3)) return;
    tc_fence_after();
    const int b = s.b, head = s.hkv * G + (row < rows ? row : 0) / p.T;
    const bool there = pos >= 0;  // else an empty row, whatever it gathered
    if (!there) l_sum = 0.f;
    const float unit = there ? ref * pow2(-static_cast<int>(kTcUpLog2)) : 0.f;
    const float sum = l_sum * pow2(-static_cast<int>(kTcUpLog2));
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    constexpr int kPartRows = R * kTcRows;
    float* part = s.part < 0 ? nullptr
                             : p.parts + static_cast<int64_t>(s.part) *
                                             (kPartRows * (D + 2));
    const int in_part = t * kTcRows + r;
#pragma unroll 1
    for (int q = 0; q < D / 32; ++q) {
      uint32_t raw_o[32];
      tmem_ld32(o_addr + q * 32, raw_o);
      tmem_ld_wait();
      uint32_t nan = 0;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) nan = i == q ? nans[i] : nan;
      float* o = reinterpret_cast<float*>(raw_o);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        o[j] = there ? o[j] * unit : 0.f;
        if (nan >> j & 1u) o[j] = __int_as_float(0x7fffffff);
      }
      if (row >= rows) continue;
      if (part != nullptr) {
        float* dst = part + in_part * D + q * 32;
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          *reinterpret_cast<float4*>(dst + j) =
              make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
      } else {
        uint16_t* dst = p.out + b * p.o_sb + head * p.o_sh + tq * p.o_ss +
                        q * 32;
#pragma unroll
        for (int j = 0; j < 32; j += 8)
          st_global_v4(dst + j, pack_bf16x2(o[j] * inv, o[j + 1] * inv),
                       pack_bf16x2(o[j + 2] * inv, o[j + 3] * inv),
                       pack_bf16x2(o[j + 4] * inv, o[j + 5] * inv),
                       pack_bf16x2(o[j + 6] * inv, o[j + 7] * inv));
      }
    }
    tc_fence_before();
    mbar_arrive(&c->o_free[t]);
    if (row < rows) {
      // (a row without a key in this part: the join's lowest reference)
      const float base = there && m_used != NEG_INF
                             ? m_used
                             : __int_as_float(0xff7fffff);
      if (part != nullptr) {
        part[kPartRows * D + in_part] = base;
        part[kPartRows * D + kPartRows + in_part] = sum;
      } else if (p.lse != nullptr) {
        p.lse[(static_cast<int64_t>(b) * p.H + head) * p.T + tq] =
            sum != 0.f ? (base + log2f(sum)) * 0.6931471805599453f : NEG_INF;
      }
    }
    warp_arrive(&c->step_empty[step % kTcSteps]);
  }
}

template <int D, int R, bool MOD>
__global__ void __launch_bounds__(kTcThreads, 1)
    paged_tree_kernel(const __grid_constant__ TcParams t) {
  using C = TcCfg<D, R>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
      ~static_cast<uintptr_t>(1023));
  TcCtl* c = reinterpret_cast<TcCtl*>(smem + C::kOffCtl);
  const int warp = threadIdx.x / 32, wg = threadIdx.x / 128;
  // the join kernel may be scheduled once every CTA here runs; it waits for
  // this grid's end before it reads the parts
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kConvertWarps = 4 * (3 - R), kScoreWarps = 4 * R;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kTcSteps; ++i) {
      mbar_init(&c->step_full[i], 1);
      mbar_init(&c->step_empty[i], kConvertWarps + 1 + kScoreWarps);
    }
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&c->kv_full[i], 4);
      mbar_init(&c->kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c->q_full[i], kTcRows);
      mbar_init(&c->s_full[i], 1);
      mbar_init(&c->p_full[i], kTcRows);
      mbar_init(&c->pv_done[i], 1);
      mbar_init(&c->o_free[i], kTcRows);
    }
    mbar_init(&c->mma_done, 1);
    c->abort = 0;
    for (int i = 0; i < 4; ++i) c->nan_step[i] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&c->tmem, kTcTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem, base = smem_u32(smem);
  if (wg == 0) {
    setmaxnreg_dec<C::kRegsPlan>();
    if (warp == 0)
      plan_role<D, R>(t, c);
    else if (warp == 1)
      mma_role<D, R>(t, c, base, tmem);
  } else if (wg == 1 || (R == 1 && wg == 3)) {
    setmaxnreg_dec<C::kRegsConvert>();
    convert_role<D, R>(t, c, base + C::kOffKv, wg >> 1);
  } else {
    setmaxnreg_inc<C::kRegsScore>();
    score_role<D, R, MOD>(t, c, base, tmem, wg - 2);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTcTmem);
}

template <int D, int R, bool MOD>
cudaError_t launch_tc(const TcParams& t, int num_sms, cudaStream_t stream) {
  using C = TcCfg<D, R>;
  auto kern = paged_tree_kernel<D, R, MOD>;
  constexpr int smem = C::kOffCtl + static_cast<int>(sizeof(TcCtl)) + 1024;
  static_assert(smem <= 232448, "shared memory budget");
  // the registers that the roles take sum up to those of the launch
  cudaFuncAttributes a;
  cudaError_t e = cudaFuncGetAttributes(&a, kern);
  if (e != cudaSuccess) return e;
  if (a.numRegs * 4 < static_cast<int>(C::kRegsPlan + (3 - R) * C::kRegsConvert +
                                       R * C::kRegsScore))
    return cudaErrorLaunchOutOfResources;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           smem);
  if (e != cudaSuccess) return e;
  kern<<<num_sms, kTcThreads, smem, stream>>>(t);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_join<TcDeal, D, R * kTcRows>(t.p, num_sms, num_sms, stream);
}

template <int D, int R>
cudaError_t launch_mod(const TcParams& t, int num_sms, cudaStream_t stream) {
  return t.p.mod.kind != 0 ? launch_tc<D, R, true>(t, num_sms, stream)
                           : launch_tc<D, R, false>(t, num_sms, stream);
}

}  // namespace

int tree_tiles(int64_t rows) {
  return rows <= kTreeFewRows ? 0 : rows <= kTcRows ? 1 : 2;
}

size_t tree_workspace_bytes(int64_t rows, int D) {
  const int tiles = tree_tiles(rows);
  if (tiles == 0) return kPaWorkspaceBytes;
  return static_cast<size_t>(kTreeMaxSms) * 2 * tiles * kTcRows * (D + 2) * 4;
}

cudaError_t launch_tree_tc(const PagedParams& p, int num_sms,
                           uint64_t timeout_ns, cudaStream_t stream) {
  TcParams t;
  t.p = p;
  t.timeout_ns = timeout_ns;
  const int tiles = tree_tiles(static_cast<int64_t>(p.H / p.H_kv) * p.T);
  if (p.D == 128)
    return tiles == 1 ? launch_mod<128, 1>(t, num_sms, stream)
                      : launch_mod<128, 2>(t, num_sms, stream);
  return tiles == 1 ? launch_mod<64, 1>(t, num_sms, stream)
                    : launch_mod<64, 2>(t, num_sms, stream);
}

cudaError_t read_tree_error(int32_t out[4]) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_tree_error, 4 * sizeof(int32_t));
  if (e != cudaSuccess) return e;
  const int32_t zero[4] = {0, 0, 0, 0};
  return cudaMemcpyToSymbol(g_tree_error, zero, 4 * sizeof(int32_t));
}

}  // namespace bsm
