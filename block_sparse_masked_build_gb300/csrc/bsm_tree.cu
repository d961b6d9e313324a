// Attention of many query rows over the paged 8-bit cache for sm_103a (GB300):
// trees of drafted tokens.  With G query heads per key/value head and T drafts
// a key serves G T rows, and from a few dozen on the work is a matrix product:
//     S = Q K^T,   P = 2^(z - m),   O += P V
// on the 5th-generation tensor core, 128 rows to a tile, one tile (R = 1) or
// two (R = 2) per CTA, 128 tokens at a time.
//
// The tensor core's operands are f16, which holds every e4m3 value: codes come
// by bulk copies into a ring of shared memory and are converted from there into
// f16 tiles; a key's scale multiplies its column of S, a value's scale that of
// P.  Per 128 tokens and head dim 128 an SM reads 32 KB (1400
// cycles at its share of the memory's rate), converts 32768 elements, and per
// tile of rows spends 1024 cycles on the tensor core and as many on the
// exponentials: one tile is bound by memory, two by the tensor core and the
// exponentials.
//
// Roles (512 threads, four warpgroups):
//   warp 0      deals the CTA's runs out in steps of up to 8 groups of 16
//               tokens: looks up pages and scales, up to 8 steps ahead.
//   warp 3      starts the copies of the codes, up to two steps ahead of their
//               conversion.
//   warps 1, 2  issue the MMAs (warp 1 owns the 512 TMEM columns).
//   converter   warpgroup 1.
//   score       warpgroups 2 and 3: one thread per query row, its TMEM lane, or
//               with one tile two, each with half of the columns: mask, running
//               maximum, exponentials, P back to TMEM over S, and at a run's
//               end the row's result.
// The roles' loops are kept short, one copy of each and 32 columns of a row at
// a time: together they must stay in the SM's instruction cache.  (With 128
// columns unrolled and codes on their way in registers, a third of all
// instruction fetches went past it: 32 sequences of 300-12000 tokens with up to
// 16 drafts took 250 us.)
// TMEM columns: S and P [0, 128) and [128, 256), by turns with one tile, one
// for each of two; O [256, 256 + D), of a second tile from 384 on.
//
// Measured over several boxes (32/8 heads of 128): 32 sequences of 300-12000
// tokens, 7-16 drafts, one tile, 149-171 us (2.4-2.7 TB/s: the conversion and the
// chain from S over the softmax to P take ~2300 cycles per 128 tokens, the tensor
// pipe is active in 28-31 %); 16 sequences of 2000-12000 tokens, 64 drafts, two
// tiles, 152-179 us (650-780 TFLOP/s, ~5000 cycles per 128 tokens); 2 sequences of
// 100000-131072 tokens, 25 drafts, 144-164 us, with capped scores, which pass
// through registers once more, 243-264.  A bias costs as much as a cap: the first
// two 235 and 224 (cap 50: 271 and 266), on a box where they took 168 and 167.
//
// A step's tokens go from a run's end to its start: the drafts come first, and
// with a bias that falls with the distance the maximum is met early.
#include <cstddef>
#include <cstdint>

#include "bsm_internal.h"
#include "bsm_paged.cuh"
#include "bsm_ptx.cuh"

namespace bsm {

// Error records, the first of each kind: code 1 (a wait gave up), block, role,
// phase; code 2 (a page table or length out of range), sequence, page slot, value.
__device__ int g_tree_error[2][4];

namespace {

constexpr int kTcThreads = 512;
constexpr int kTcRows = 128;    // of a tile: one accumulator
constexpr int kTcTokens = 128;  // of a full step
constexpr int kTcGroups = kTcTokens / kPaGroup;
constexpr int kTcSteps = 8;     // ring of steps
constexpr uint32_t kTcTmem = 512;
// Up to so many query rows per key/value head go to the kernel of single tokens,
// which reads the cache once for each 16: 32 sequences of 300-12000 tokens with 8
// rows took it 94 us (this one 167), with 16 130 (170), with 24 246 (172).  (One
// sequence of 2000 tokens with 32 rows: 21.9 us, this one 24.4.)
constexpr int kTreeFewRows = 16;
constexpr int kRolePlan = 1, kRoleMma = 2, kRoleConvert = 3, kRoleScore = 4,
              kRoleLoad = 5;
// P is scaled by 2^9 before it becomes f16, whose smallest number is 2^-24: a
// key's weight is lost below 2^-33 of the largest, with the least of the values'
// scales (2^-6) below 2^-27.  The reference m may lie up to 2^6 below the running
// maximum before O is rescaled; 2^15 still fits f16.
constexpr float kTcUpLog2 = 9.f, kTcRescaleLog2 = 6.f;

// The deal: a unit is a full step.
struct TcDeal {
  static constexpr bool kTree = true;
  static constexpr int kUnit = kTcGroups, kRunCost = 6, kLeast = 1;
};

template <int D, int R>
struct TcCfg {
  static constexpr int kTile = kTcTokens * D * 2;  // Q, K or V in f16
  static constexpr int kCodes = kTcTokens * D;     // K or V in e4m3
  // Rings of tiles and of codes, by half steps: 2 step (keys), 2 step + 1
  // (values); 208 KB with Q at D = 128.
  // (With three tiles beside one of rows, keys would wait for the P V two steps
  // back, and S could not go ahead.)
  static constexpr int kSlots = R == 1 ? 4 : 3, kStages = 3;
  static __device__ __forceinline__ uint32_t slot(uint32_t h) {
    return h % kSlots;
  }
  static __device__ __forceinline__ uint32_t slot_use(uint32_t h) {
    return h / kSlots;
  }
  static __device__ __forceinline__ uint32_t stage(uint32_t h) {
    return h % kStages;
  }
  static __device__ __forceinline__ uint32_t stage_use(uint32_t h) {
    return h / kStages;
  }
  // threads that share a row: with one tile the two score warpgroups take half
  // of its columns each
  static constexpr int kRowThreads = R == 1 ? 2 : 1;
  static constexpr int kOffKv = R * kTile;
  static constexpr int kOffCodes = kOffKv + kSlots * kTile;
  static constexpr int kOffCtl = kOffCodes + kStages * kCodes;
};

// Up to 128 tokens of a run, newest step first.
struct alignas(16) TcStep {  // (its arrays are read 16 bytes at a time)
  int32_t groups;    // 1 .. 8 groups of 16 tokens from tok0 on; 0: the end
  int32_t tok0;
  int32_t first, last;  // of its run
  int32_t plain;     // 8 groups, and every row sees every token
  float v_ref;       // O is in units of this scale
  // of the run
  int32_t b, hkv, row0, part;  // part: -1 whole, else its slot in the workspace
  int32_t len, lo, n;          // tokens, first visible one, drafts
  int32_t pad[3];
  float k_scale[kTcGroups];
  float v_log2[kTcGroups];     // log2(scale / v_ref)
  float v_inv[kTcGroups];      // v_ref / scale
  int64_t off[kTcGroups];      // of the group's codes; -1: page out of range
};

static_assert(offsetof(TcStep, k_scale) % 16 == 0 && sizeof(TcStep) % 16 == 0,
              "alignment");

struct TcCtl {
  uint64_t step_full[kTcSteps], step_empty[kTcSteps];
  uint64_t code_full[3], code_empty[3];
  uint64_t kv_full[4], kv_empty[4];
  uint64_t q_full[2], s_full[2], p_full[2], pv_done[2], o_free[2], mma_done[2];
  uint32_t tmem;
  int abort;
  TcStep steps[kTcSteps];
  // of steps that are not plain, by step modulo 2: columns' positions, and the
  // NaN codes of V (16 dims per entry), with the step's number + 1 where there
  // are any.  They are written with V's tile, whose slot comes free when the
  // tensor core has taken P of the step before the last: the rows are done with
  // that one's.
  int32_t pos[2][kTcTokens];
  uint16_t nan[2][kTcTokens][8];
  uint32_t nan_step[2];
  // one tile of rows: what a row's two threads tell each other, [half][row]
  uint64_t meet[4];  // by TMEM lane quarter
  float pair[2][2][kTcRows];
  uint32_t pair_nan[2][4][kTcRows];
};

struct TcParams {
  PagedParams p;
  uint64_t timeout_ns;
  int32_t no_plan;  // self test: nothing is dealt out, and the other roles give up
};

__device__ __forceinline__ void tc_record(int code, int a, int b, int c) {
  int* rec = g_tree_error[code - 1];
  if (atomicCAS(&rec[0], 0, code) == 0) {
    rec[1] = a;
    rec[2] = b;
    rec[3] = c;
  }
}

// Bounded wait of a whole warp, alike in every lane: as mbar_wait, with the
// clock looked at after every 256 tries that ran out.  One copy, called, as it
// stands in every role's loop.
__device__ __noinline__ bool tc_wait_at(uint32_t bar, uint32_t parity,
                                        volatile int* abort, uint64_t limit,
                                        int where) {
  uint64_t t0 = 0;
  uint32_t ok;
#pragma unroll 1
  for (uint32_t it = 1;; ++it) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) break;
    if ((it & 255u) == 0u) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (*abort != 0) break;
      if (now - t0 > limit || it > (1u << 30)) {
        *abort = 1;
        if (threadIdx.x % 32 == 0)
          tc_record(1, blockIdx.x, where >> 4, where & 15);
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool tc_wait(const TcParams& t, TcCtl* c,
                                        uint64_t* bar, uint32_t parity,
                                        int role, int phase) {
  // (a call costs some 150 cycles: most phases are over already)
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  if (__all_sync(0xffffffffu, ok)) return true;
  return tc_wait_at(smem_u32(bar), parity, &c->abort, t.timeout_ns,
                    role * 16 + phase);
}

__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if (threadIdx.x % 32 == 0) mbar_arrive(bar);
}

__device__ __forceinline__ float pow2(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// (Loads and stores of TMEM and the MMAs' elections are a whole warp's at once: a
// __syncwarp stands between them and what lanes do apart.)

// ----------------------------------------------------------------- planner

// Value scales go along with P: its column is multiplied by scale / v_ref, at
// most 1 and no less than 2^-6, which its f16 stands (see kTcUpLog2), and the
// row sums are of P over that factor.  Pages further apart go in steps of their
// own, between which O moves to the other unit.  A unit leaves room for scales
// that are four times that of the first page.  (All in log2: of a scale of 0,
// which no page that holds tokens has, -inf, as a unit 2^-126.)
__device__ __forceinline__ bool near_scale(float log2_scale, float log2_ref) {
  const float r = log2_scale - log2_ref;
  return r >= -6.f && r <= 0.f;
}

// One run: groups [g0, g1) of its sequence's plan.
template <int D, int R>
__device__ __forceinline__ bool plan_run(const TcParams& t, TcCtl* c,
                                         int b, const PaPlan& plan, int hkv,
                                         int row0, int g0, int g1, int part,
                                         uint32_t& step) {
  const PagedParams& p = t.p;
  const int lane = threadIdx.x % 32;
  const int* table = p.table + static_cast<int64_t>(b) * p.table_stride;
  const int base = plan.len - plan.drafts;
  // lane i has group top - 1 - i of the 32 in hand; the pages of the 32 behind
  // them are looked up meanwhile
  auto page_of = [&](int top) {
    const int g = top - 1 - lane;
    return g >= g0 ? table[(plan.first_group + g) >> (p.page_shift - 4)] : -1;
  };
  int next_pid = page_of(g1);
  // the run's query into L2, for the rows that will load it at its start
  for (int i = lane; i < R * kTcRows; i += 32)
    if (row0 + i < p.H / p.H_kv * p.T) {
      const uint16_t* q = p.q + b * p.q_sb +
                          (hkv * (p.H / p.H_kv) + (row0 + i) / p.T) * p.q_sh +
                          (row0 + i) % p.T * p.q_ss;
#pragma unroll
      for (int j = 0; j < D; j += 64)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(q + j));
    }
  float ref = 0.f, log2_ref = 0.f;  // 0: none yet
#pragma unroll 1
  for (int top = g1; top > g0; top -= 32) {
    const int g = top - 1 - lane, pid = next_pid;
    const int tok = (plan.first_group + g) * kPaGroup;
    float ks = 0.f, vs = 1.f;
    int64_t off = -1;
    if (g >= g0) {
      if (static_cast<uint32_t>(pid) < static_cast<uint32_t>(p.num_pages)) {
        const int64_t block = static_cast<int64_t>(pid) * p.H_kv + hkv;
        ks = p.k_scale[block];
        vs = p.v_scale[block];
        off = ((block << p.page_shift) + (tok & (p.page_size - 1))) * D;
      } else {
        tc_record(2, b, tok >> p.page_shift, pid);
      }
    }
    next_pid = page_of(top - 32);
    const float lv = log2f(vs), rv = 1.f / vs;
    const int here = min(32, top - g0);
#pragma unroll 1
    for (int at = 0; at < here;) {
      int n = min(kTcGroups, here - at);
      const bool mine = lane >= at && lane < at + n && off >= 0;
      const unsigned some = __ballot_sync(0xffffffffu, mine);
      unsigned far = __ballot_sync(
          0xffffffffu, mine && (ref == 0.f || !near_scale(lv, log2_ref)));
      if (far & (1u << at) || (ref == 0.f && some != 0)) {
        const int one = __ffs(some) - 1;
        ref = fmaxf(4.f * __shfl_sync(0xffffffffu, vs, one), 0x1p-126f);
        log2_ref = log2f(ref);
        far = __ballot_sync(0xffffffffu, mine && !near_scale(lv, log2_ref));
        // (a scale that is near nothing, itself included, goes alone)
        far &= ~(1u << one);
      }
      if (far != 0) n = __ffs(far) - 1 - at;
      const bool ours = lane >= at && lane < at + n;
      const uint32_t slot = step % kTcSteps;
      if (!tc_wait(t, c, &c->step_empty[slot], ((step / kTcSteps) & 1) ^ 1,
                   kRolePlan, 0))
        return false;
      TcStep& s = c->steps[slot];
      const int i = at + n - 1 - lane;  // ascending tokens
      if (ours) {
        s.k_scale[i] = ks;
        s.v_log2[i] = off >= 0 ? lv - log2_ref : 0.f;
        s.v_inv[i] = off >= 0 ? rv * ref : 1.f;
        s.off[i] = off;
      }
      if (lane >= n && lane < kTcGroups) {  // their columns weigh 0
        s.k_scale[lane] = s.v_log2[lane] = 0.f;
        s.v_inv[lane] = 1.f;
      }
      const int tok0 = (plan.first_group + top - at - n) * kPaGroup;
      const unsigned there = __ballot_sync(0xffffffffu, ours && off >= 0);
      if (lane == 0) {
        s.groups = n;
        s.tok0 = tok0;
        s.first = top == g1 && at == 0;
        s.last = top - at - n == g0;
        s.plain = n == kTcGroups && tok0 + kTcTokens <= base &&
                  tok0 >= plan.lo && __popc(there) == kTcGroups &&
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
  const uint32_t slot = step % kTcSteps;  // the end
  if (!ok || !tc_wait(t, c, &c->step_empty[slot], ((step / kTcSteps) & 1) ^ 1,
                      kRolePlan, 2))
    return;
  if (lane == 0) c->steps[slot].groups = 0;
  warp_arrive(&c->step_full[slot]);
}

// ------------------------------------------------------------------- loader

__device__ __forceinline__ bool wait_step(const TcParams& t, TcCtl* c,
                                          uint32_t step, int role) {
  return tc_wait(t, c, &c->step_full[step % kTcSteps], (step / kTcSteps) & 1,
                 role, 9);
}

// Copies the codes of every step's keys and then its values: one bulk copy for
// groups that follow each other in a page.
template <int D, int R>
__device__ __forceinline__ void load_role(const TcParams& t, TcCtl* c,
                                          uint32_t codes) {
  using C = TcCfg<D, R>;
  constexpr int kBytes = kPaGroup * D;
  const int lane = threadIdx.x % 32;
  uint32_t h = 0;  // half steps copied
  int64_t off = -1;
  bool ok = true;
#pragma unroll 1
  for (;; ++h) {
    if (h % 2 == 0) {
      const uint32_t step = h / 2;
      ok = wait_step(t, c, step, kRoleLoad);
      if (!ok) break;
      const TcStep& s = c->steps[step % kTcSteps];
      const int groups = s.groups;
      if (groups == 0) break;
      off = lane < groups ? s.off[lane] : -1;
      warp_arrive(&c->step_empty[step % kTcSteps]);
    }
    const int64_t before = __shfl_up_sync(0xffffffffu, off, 1);
    const unsigned there = __ballot_sync(0xffffffffu, off >= 0);
    const unsigned starts = __ballot_sync(
        0xffffffffu,
        off >= 0 && (lane == 0 || before < 0 || before + kBytes != off));
    const uint32_t st = C::stage(h);
    ok = tc_wait(t, c, &c->code_empty[st], (C::stage_use(h) & 1) ^ 1, kRoleLoad,
                 0);
    if (!ok) break;
    if (lane == 0)
      mbar_arrive_expect_tx(&c->code_full[st], __popc(there) * kBytes);
    __syncwarp();
    if (starts >> lane & 1u) {
      // up to the next start or the next page that is not there
      const unsigned ends = (starts | ~there) >> lane >> 1;
      const int n = ends != 0 ? __ffs(ends) : 32;
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
          "[%0], [%1], %2, [%3];" ::"r"(codes + st * C::kCodes + lane * kBytes),
          "l"((h % 2 ? t.p.v : t.p.k) + off), "r"(n * kBytes),
          "r"(smem_u32(&c->code_full[st]))
          : "memory");
    }
    __syncwarp();
  }
  // Given up: the copies under way still land in this CTA's shared memory.  (At
  // the end the converters have waited for every copy.)
  if (!ok && lane == 0)
    for (uint32_t i = 1; i <= C::kStages && i <= h; ++i)
      mbar_wait_drain(&c->code_full[C::stage(h - i)],
                      C::stage_use(h - i) & 1, t.timeout_ns);
  __syncwarp();
}

// -------------------------------------------------------------- converters

// Which token's row, and which 16-byte piece of it, a thread has in 16 tokens (D
// = 128) or 32 (64).  Eight lanes that load or store together have pieces of
// two neighbouring tokens, one half of a row from each at D = 128: loads touch
// 128 different bytes, and the swizzle puts their two f16 halves into eight
// different 16-byte columns.
template <int D>
__device__ __forceinline__ int piece_of(int i) {
  return D == 128 ? (i & 3) | ((i ^ (i >> 1)) & 4) : i & 3;
}
template <int D>
__device__ __forceinline__ int token_of(int i) {
  return D == 128 ? (i >> 2 & 1) | (i >> 4 << 1) : i >> 2;
}

// What a step that is not plain needs before 16 codes of token tr are
// converted: tokens that are no sequence's become zeros, and so do NaN codes of
// values, which are noted, as a row that does not see them must not meet 0 *
// NaN.
__device__ __forceinline__ void clean_codes(TcCtl* c, const TcStep& s,
                                            uint32_t step, bool values, int tr,
                                            int piece, uint32_t* w) {
  const int tok = s.tok0 + tr;
  const bool there = tok >= s.lo && tok < s.len && s.off[tr / kPaGroup] >= 0;
  uint32_t found = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (!there) w[j] = 0u;
    const uint32_t n = nan_codes(w[j]) >> 7;  // one bit per byte
    if (values) w[j] &= ~(n * 0xffu);
    // the four bits 0, 8, 16, 24 next to each other
    found |= ((n * 0x00204081u >> 21) & 0xfu) << (4 * j);
  }
  if (!values) return;
  c->nan[step % 2][tr][piece] = static_cast<uint16_t>(found);
  if (found != 0) c->nan_step[step % 2] = step + 1;
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y,
                                       uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x),
               "r"(y), "r"(z), "r"(w)
               : "memory");
}

__device__ __forceinline__ void lds128(uint32_t w[4], uint32_t a) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(a));
}
// 16 codes as f16, the first eight at a, the others at b.
__device__ __forceinline__ void store_codes(const uint32_t w[4], uint32_t a,
                                            uint32_t b) {
  sts128(a, e4m3x2_to_f16x2(w[0]), e4m3x2_to_f16x2_hi(w[0]),
         e4m3x2_to_f16x2(w[1]), e4m3x2_to_f16x2_hi(w[1]));
  sts128(b, e4m3x2_to_f16x2(w[2]), e4m3x2_to_f16x2_hi(w[2]),
         e4m3x2_to_f16x2(w[3]), e4m3x2_to_f16x2_hi(w[3]));
}

// The converter warpgroup: every step's keys, then its values.  Tiles are rows of
// 64 elements (128 bytes) per token, two such blocks at D = 128, in the 128-byte
// swizzle.
template <int D, int R>
__device__ __forceinline__ void convert_role(const TcParams& t, TcCtl* c,
                                             uint32_t kv, uint32_t codes) {
  using C = TcCfg<D, R>;
  const PagedParams& p = t.p;
  const int i = threadIdx.x % 128, piece = piece_of<D>(i);
  const uint32_t row = token_of<D>(i), chunk = (2 * piece) & 7;
  const uint32_t line = kv + (piece >> 2) * (kTcTokens * 128) + row * 128;
  const uint32_t at_a = line + ((chunk ^ (row & 7)) << 4);
  const uint32_t at_b = line + ((chunk ^ 1u ^ (row & 7)) << 4);
  const uint32_t from = codes + row * D + piece * 16;
  constexpr int kRows = 2048 / D;  // tokens of the warpgroup at a time
#pragma unroll 1
  for (uint32_t h = 0;; ++h) {
    const uint32_t step = h / 2;
    const bool values = h % 2 != 0;
    if (!wait_step(t, c, step, kRoleConvert)) return;
    const TcStep& s = c->steps[step % kTcSteps];
    const int tokens = s.groups * kPaGroup;
    if (tokens == 0) return;
    const uint32_t st = C::stage(h), slot = C::slot(h);
    if (!tc_wait(t, c, &c->code_full[st], C::stage_use(h) & 1, kRoleConvert,
                 0) ||
        !tc_wait(t, c, &c->kv_empty[slot], (C::slot_use(h) & 1) ^ 1,
                 kRoleConvert, 1))
      return;
    const bool plain = s.plain != 0;
    const uint32_t src = from + st * C::kCodes;
    const uint32_t dst_a = at_a + slot * C::kTile,
                   dst_b = at_b + slot * C::kTile;
    constexpr int kPieces = D / 16;
    uint32_t w[kPieces][4];
    if (plain) {
#pragma unroll
      for (int k = 0; k < kPieces; ++k) lds128(w[k], src + k * 2048);
#pragma unroll
      for (int k = 0; k < kPieces; ++k)
        store_codes(w[k], dst_a + k * (kRows * 128), dst_b + k * (kRows * 128));
    } else {
#pragma unroll 1
      for (int k = 0; k * kRows < tokens; ++k) {
        const int tr = k * kRows + static_cast<int>(row);
        if (tr >= tokens) break;  // (D = 64, half of the warpgroup)
        lds128(w[0], src + k * 2048);
        clean_codes(c, s, step, values, tr, piece, w[0]);
        store_codes(w[0], dst_a + k * (kRows * 128), dst_b + k * (kRows * 128));
      }
    }
    if (!plain && values && (p.window > 0 || (p.mod.kind & kModBias))) {
      const int tok = s.tok0 + i, base = s.len - s.n;
      c->pos[step % 2][i] = tok >= base && tok < s.len
                                ? base + draft_depth(p, s.b, tok - base, s.n)
                                : tok;
    }
    fence_proxy_async();
    __syncwarp();
    if (threadIdx.x % 32 == 0) {
      mbar_arrive(&c->code_empty[st]);
      mbar_arrive(&c->kv_full[slot]);
      if (values) mbar_arrive(&c->step_empty[step % kTcSteps]);
    }
  }
}

// --------------------------------------------------------------------- MMA

// Instruction descriptor as idesc_bf16_f32, with f16 operands.
__device__ __forceinline__ constexpr uint32_t idesc_f16(int N, bool mn_major) {
  return (1u << 4) | ((mn_major ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(kTcRows >> 4) << 24);
}

// S (128 rows x 16 groups tokens) = Q K^T, by descriptors of the two tiles.
template <int D>
__device__ __forceinline__ void issue_s(uint32_t d, uint64_t q, uint64_t k,
                                        int groups) {
  const uint32_t idesc = idesc_f16(groups * kPaGroup, false);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const uint32_t off = (i >> 2) * (kTcTokens * 128 / 16) + (i & 3) * 2;
    mma_ss_elect(d, q + off, k + off, idesc, i > 0);
  }
}

// O (+)= P V over `groups` groups; first: O's first.
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t d, uint32_t p, uint64_t v,
                                         int groups, bool first) {
  constexpr uint32_t idesc = idesc_f16(D, true);
#pragma unroll
  for (int i = 0; i < kTcGroups; ++i)
    if (i < groups)
      mma_ts_elect(d, p + i * 8, v + i * (kPaGroup * 128 / 16), idesc,
                   i > 0 || !first);
}

// Two warps issue MMAs (one warp alone, whose waits and commits no other work
// covered, took 3300 cycles for a step's S and P V).  With one tile of rows warp
// 0 issues every S and warp 1 every P V; with two, each its tile's: S_t goes
// behind the P V that reads its columns, as MMAs of one thread run in the order
// they were issued.  A run's first S waits for its query, its first P V for O,
// until the rows of the run before are written out.
template <int D, int R>
__device__ __forceinline__ void mma_role(const TcParams& t, TcCtl* c,
                                         uint32_t smem, uint32_t tmem,
                                         const int w) {
  using C = TcCfg<D, R>;
  constexpr uint32_t kUnits = C::kTile >> 4;
  const int tile = R == 2 ? w : 0;
  const uint64_t dq = sdesc_sw128(smem, 16, 1024) + tile * kUnits;
  const uint64_t dk = sdesc_sw128(smem + C::kOffKv, 16, 1024);
  const uint64_t dv = sdesc_sw128(smem + C::kOffKv, kTcTokens * 128, 1024);
  const uint32_t o_acc = tmem + 256 + tile * 128;
  uint32_t runs = 0;  // begun
  int groups_before = 0;
  bool first_before = false;
  bool ok = true;
  auto wait_kv = [&](uint32_t h) {
    return tc_wait(t, c, &c->kv_full[C::slot(h)], C::slot_use(h) & 1, kRoleMma,
                   2);
  };
#pragma unroll 1
  for (uint32_t step = 0; ok; ++step) {
    ok = wait_step(t, c, step, kRoleMma);
    if (!ok) break;
    const TcStep& s = c->steps[step % kTcSteps];
    const int groups = s.groups;
    const bool first = s.first != 0;
    const bool more = groups != 0;
    warp_arrive(&c->step_empty[step % kTcSteps]);
    if (R == 1) {
      if (!more) break;
      const uint32_t buf = step & 1, use = step >> 1;
      const uint32_t s_acc = tmem + buf * 128;
      const uint32_t h = 2 * step + w;
      ok = wait_kv(h);
      if (w == 0) {
        // the buffer's P is used up
        if (ok && step > 1)
          ok = tc_wait(t, c, &c->pv_done[buf], (use - 1) & 1, kRoleMma, 5);
        if (ok && first) ok = tc_wait(t, c, &c->q_full[0], runs & 1, kRoleMma, 1);
      } else {
        if (ok) ok = tc_wait(t, c, &c->p_full[buf], use & 1, kRoleMma, 3);
        if (ok && first)
          ok = tc_wait(t, c, &c->o_free[0], (runs & 1) ^ 1, kRoleMma, 4);
      }
      if (!ok) break;
      runs += first;
      tc_fence_after();
      if (w == 0) {
        issue_s<D>(s_acc, dq, dk + C::slot(h) * kUnits, groups);
        mma_commit_elect(&c->s_full[buf]);
        mma_commit_elect(&c->kv_empty[C::slot(h)]);
      } else {
        issue_pv<D>(o_acc, s_acc, dv + C::slot(h) * kUnits, groups, first);
        mma_commit_elect(&c->pv_done[buf]);
        mma_commit_elect(&c->kv_empty[C::slot(h)]);
      }
    } else {
      const uint32_t s_acc = tmem + tile * 128;
      if (step > 0) {
        const uint32_t h = 2 * step - 1;
        ok = wait_kv(h) &&
             tc_wait(t, c, &c->p_full[tile], (step - 1) & 1, kRoleMma, 3);
        // run k (k = runs - 1) finds O free when k runs were written out
        if (ok && first_before)
          ok = tc_wait(t, c, &c->o_free[tile], runs & 1, kRoleMma, 4);
        if (!ok) break;
        tc_fence_after();
        issue_pv<D>(o_acc, s_acc, dv + C::slot(h) * kUnits, groups_before,
                    first_before);
        mma_commit_elect(&c->pv_done[tile]);
        mma_commit_elect(&c->kv_empty[C::slot(h)]);
      }
      if (!more) break;
      ok = wait_kv(2 * step);
      if (ok && first)
        ok = tc_wait(t, c, &c->q_full[tile], runs & 1, kRoleMma, 1);
      if (!ok) break;
      runs += first;
      tc_fence_after();
      issue_s<D>(s_acc, dq, dk + C::slot(2 * step) * kUnits, groups);
      mma_commit_elect(&c->s_full[tile]);
      mma_commit_elect(&c->kv_empty[C::slot(2 * step)]);
      groups_before = groups;
      first_before = first;
    }
  }
  // every MMA issued above has completed once this arrives
  __syncwarp();
  mma_commit_elect(&c->mma_done[w]);
  if (threadIdx.x % 32 == 0 &&
      !mbar_wait_drain(&c->mma_done[w], 0, t.timeout_ns))
    tc_record(1, blockIdx.x, kRoleMma, 8);
  __syncwarp();
}

// ------------------------------------------------------------------- score

// A row's query into its tile: f16, scaled so that the row's largest magnitude
// becomes [1, 2) (f16 then keeps bf16's 8 bits of every element above 2^-17 of
// it, and 2^-25 of it of the rest).  Returns the factor that undoes it.
// (Pieces [i0, i1) of 8 elements are stored.)
template <int D>
__device__ __forceinline__ float load_query(const uint16_t* src, bool live,
                                         bool negate, uint32_t tile, int r,
                                         int i0, int i1) {
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
    if (i < i0 || i >= i1) continue;
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

// cap * tanh(x / cap) of 32 of a row's scores S = q.k, in log2 units:
// polynomials where the warp's scores allow them (|y| <= 0.5, <= 1.2), else
// exponentials.
__device__ __forceinline__ void cap_scores(const ScoreMod& m, float* s) {
  float a0 = 0.f, a1 = 0.f;
#pragma unroll
  for (int c = 0; c < 32; c += 4) {
    a0 = fmax3_abs_nan(a0, s[c], s[c + 1]);
    a1 = fmax3_abs_nan(a1, s[c + 2], s[c + 3]);
  }
  const float top = fmax3_abs_nan(a0, a1, a1);
  if (__all_sync(0xffffffffu, top <= m.poly_max)) {
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      float h0, h1;
      poly_sq2<4>(h0, h1, s[c], s[c + 1], m.poly);
      fmul2v(s[c], s[c + 1], s[c], s[c + 1], h0, h1);
    }
  } else if (__all_sync(0xffffffffu, top <= m.wide_max)) {
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      float h0, h1;
      poly_sq2<7>(h0, h1, s[c], s[c + 1], m.wide);
      fmul2v(s[c], s[c + 1], s[c], s[c + 1], h0, h1);
    }
  } else {
    // tanh(y) = 1 - 2 / (1 + e^(2 y)), off by 2^-23 of the cap
    const float k2 = -2.f * m.cap_log2;
#pragma unroll
    for (int c = 0; c < 32; ++c) {
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

// The largest of 32 columns, the first 16 times f0, the others times f1.
__device__ __forceinline__ float max_of(const float* x, float f0, float f1) {
  float m[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float* v = x + 16 * i;
    const float a = fmax3(v[0], v[1], v[2]), b = fmax3(v[3], v[4], v[5]);
    const float d = fmax3(v[6], v[7], v[8]), e = fmax3(v[9], v[10], v[11]);
    m[i] = fmax3(fmax3(a, b, d), fmax3(e, v[12], v[13]), fmaxf(v[14], v[15]));
  }
  return fmaxf(m[0] * f0, m[1] * f1);
}

// P of 32 columns, 2^(x f + add) times their values' scales, into P's columns at
// `to`; returns the sum without the scales.  f, add, inv: of either 16 columns.
__device__ __forceinline__ float weigh(const float* x, const float* f,
                                       const float* add, const float* inv,
                                       uint32_t to) {
  uint32_t pk[16];
  float sum = 0.f;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
    for (int j = 16 * g; j < 16 * g + 16; j += 4) {
      float x0, x1, x2, x3;
      ffma2(x0, x1, x[j], x[j + 1], f[g], add[g]);
      ffma2(x2, x3, x[j + 2], x[j + 3], f[g], add[g]);
      const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
      const float p2 = ex2_approx(x2), p3 = ex2_approx(x3);
      fadd2(l0, l1, l0, l1, p0, p1);
      fadd2(l2, l3, l2, l3, p2, p3);
      pk[j / 2] = pack_f16x2(p0, p1);
      pk[j / 2 + 1] = pack_f16x2(p2, p3);
    }
    sum = fmaf((l0 + l1) + (l2 + l3), inv[g], sum);
  }
  tmem_st16(to, pk);
  return sum;
}

// The scores of a step that its scales alone do not give (32-column pieces [q0,
// q1)), written back as they are to be weighed; returns the largest.  Out of
// line, as most steps are plain and the score loop is to stay short.
template <int D>
struct NanPlaces {  // dims in which a row sees a NaN value
  uint32_t w[D / 32];
};

template <int D, bool MOD>
__device__ __noinline__ float modified_scores(const PagedParams& p, TcCtl* c,
                                              const TcStep& s, uint32_t step,
                                              uint32_t s_addr, int q0, int q1,
                                              float q_mul, float slope2,
                                              int pos, int tq,
                                              NanPlaces<D>* nans) {
  const float NEG_INF = __int_as_float(0xff800000);
  const bool plain = s.plain != 0;
  const bool capped = MOD && (p.mod.kind & kModCap);
  const bool biased = MOD && (p.mod.kind & kModBias);
  float top = NEG_INF;
#pragma unroll 1
  for (int q = q0; q < q1; ++q) {
    uint32_t keep = ~0u;
    if (!plain) {
      keep = pos >= 0 ? visible(p, s, q, tq) : 0u;
      const int* at = c->pos[step % 2] + 32 * q;
      if (p.window > 0)
#pragma unroll 1
        for (int j = 0; j < 32; ++j)
          if (pos - at[j] >= p.window) keep &= ~(1u << j);
      if (c->nan_step[step % 2] == step + 1) {
        // values that are NaN: a row that sees one has NaN in that place
#pragma unroll 1
        for (uint32_t k = keep; k != 0; k &= k - 1) {
          const uint16_t* n = c->nan[step % 2][32 * q + __ffs(k) - 1];
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            nans->w[i] |= *reinterpret_cast<const uint32_t*>(n + 2 * i);
        }
      }
      __syncwarp();  // (what the lanes did differs)
    }
    float x[32];
    tmem_ld32(s_addr + q * 32, reinterpret_cast<uint32_t*>(x));
    tmem_ld_wait();
    const float f0 = q_mul * s.k_scale[2 * q];
    const float f1 = q_mul * s.k_scale[2 * q + 1];
#pragma unroll
    for (int j = 0; j < 32; j += 2)
      fmul2(x[j], x[j + 1], x[j], x[j + 1], j < 16 ? f0 : f1);
    if (MOD) {
      // columns that are not seen may hold anything; 0 costs the cap
      // nothing
      if (!plain)
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (!(keep >> j & 1u)) x[j] = 0.f;
      if (capped) cap_scores(p.mod, x);
      if (biased && plain) {
        const float d0 = static_cast<float>(s.tok0 + 32 * q - pos);
#pragma unroll
        for (int j = 0; j < 32; ++j)
          x[j] = fmaf(slope2, d0 + static_cast<float>(j), x[j]);
      } else if (biased) {
        const int* at = c->pos[step % 2] + 32 * q;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          x[j] = fmaf(-slope2, fabsf(static_cast<float>(pos - at[j])),
                      x[j]);
      }
    }
    if (!plain)
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (!(keep >> j & 1u)) x[j] = NEG_INF;
    top = fmaxf(top, max_of(x, 1.f, 1.f));
    tmem_st32(s_addr + q * 32, reinterpret_cast<uint32_t*>(x));
  }
  tmem_st_wait();
  return top;
}

// The rows' warpgroups: one of each tile, or, with one tile, one of each half of
// a step's columns (and of O's): a row's two threads then tell each other their
// maxima.
template <int D, int R, bool MOD>
__device__ __forceinline__ void score_role(const TcParams& tp, TcCtl* c,
                                           uint32_t smem, uint32_t tmem,
                                           const int w) {
  using C = TcCfg<D, R>;
  const PagedParams& p = tp.p;
  const int tile = R == 2 ? w : 0, half = R == 1 ? w : 0;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int quarter = warp % 4;
  const int r = quarter * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  constexpr int kDims = D / C::kRowThreads;  // of O that a thread scales, writes
  const uint32_t o_addr = tmem + lane_off + 256 + tile * 128 + half * kDims;
  const float NEG_INF = __int_as_float(0xff800000);
  const int G = p.H / p.H_kv, rows = G * p.T;
  const bool capped = MOD && (p.mod.kind & kModCap);
  const bool biased = MOD && (p.mod.kind & kModBias);
  const bool negate = !capped && p.scale_x < 0.f;
  uint32_t meets = 0;
  // Tells the row's other thread x, and the NaN places if any are given, and
  // waits for its.
  auto exchange = [&](float& x, const NanPlaces<D>* nans, float* other) {
    c->pair[meets & 1][half][r] = x;
    if (nans != nullptr)
#pragma unroll
      for (int i = 0; i < D / 32; ++i) c->pair_nan[half][i][r] = nans->w[i];
    warp_arrive(&c->meet[quarter]);
    const bool ok =
        tc_wait(tp, c, &c->meet[quarter], meets & 1, kRoleScore, 6);
    *other = c->pair[meets & 1][half ^ 1][r];
    ++meets;
    return ok;
  };
  auto wait_pv = [&](uint32_t step, int phase) {  // a step's P V is done
    return R == 2
               ? tc_wait(tp, c, &c->pv_done[tile], step & 1, kRoleScore, phase)
               : tc_wait(tp, c, &c->pv_done[step & 1], step >> 1 & 1,
                         kRoleScore, phase);
  };
  // the run's query into its tile; the tile's S before must be done
  auto start_query = [&](const TcStep& s) {
    const int at = s.row0 + tile * kTcRows + r;
    const bool live = at < rows;
    const int head = s.hkv * G + (live ? at / p.T : 0);
    const float up = load_query<D>(
        p.q + s.b * p.q_sb + head * p.q_sh + (live ? at % p.T : 0) * p.q_ss,
        live, negate, smem + tile * C::kTile, r, half * (kDims / 8),
        (half + 1) * (kDims / 8));
    fence_proxy_async();
    mbar_arrive(&c->q_full[tile]);
    return up;
  };
  // of the run
  float q_mul = 0.f, slope2 = 0.f, m_used = NEG_INF, l_sum = 0.f, ref = 1.f;
  int row = 0, tq = 0, pos = -1;
  NanPlaces<D> nans;
  uint32_t run_pv = 0;
  float up = 0.f;  // of the next run's query, which is loaded ahead
#pragma unroll 1
  for (uint32_t step = 0;; ++step) {
    if (!wait_step(tp, c, step, kRoleScore)) return;
    const TcStep& s = c->steps[step % kTcSteps];
    if (s.groups == 0) return;
    if (s.first) {
      if (step == 0) up = start_query(s);
      row = s.row0 + tile * kTcRows + r;
      const bool live = row < rows;
      tq = live ? row % p.T : 0;
      const int head = s.hkv * G + (live ? row / p.T : 0);
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
      for (int i = 0; i < D / 32; ++i) nans.w[i] = 0u;
      __syncwarp();
    }
    const int buf = R == 2 ? tile : static_cast<int>(step & 1);
    const uint32_t use = R == 2 ? step : step >> 1;
    const uint32_t s_addr = tmem + lane_off + buf * 128;
    const bool plain = s.plain != 0;
    if (!plain) {  // positions and NaN codes come with the values
      const uint32_t h = 2 * step + 1;
      if (!tc_wait(tp, c, &c->kv_full[C::slot(h)], C::slot_use(h) & 1,
                   kRoleScore, 5))
        return;
    }
    if (!tc_wait(tp, c, &c->s_full[buf], use & 1, kRoleScore, 1)) return;
    tc_fence_after();
    // ---- the largest score.  Scores that the scales alone do not give are
    // written back as they are to be weighed.
    const bool scaled = MOD || !plain;
    float top = NEG_INF;
    if (scaled)
      top = modified_scores<D, MOD>(p, c, s, step, s_addr, 2 * half,
                                    R == 1 ? 2 * half + 2 : 4, q_mul, slope2,
                                    pos, tq, &nans);
    float xa[32], xb[32];
    float f[4];  // the scales of xa's and xb's groups
    auto load_scales = [&](int q) {
      const float4 ks = *reinterpret_cast<const float4*>(&s.k_scale[2 * q]);
      f[0] = scaled ? 1.f : ks.x * q_mul, f[1] = scaled ? 1.f : ks.y * q_mul;
      f[2] = scaled ? 1.f : ks.z * q_mul, f[3] = scaled ? 1.f : ks.w * q_mul;
    };
    if (R == 1) {  // this thread's columns stay in registers
      const uint32_t at = s_addr + half * 64;
      tmem_ld32(at, reinterpret_cast<uint32_t*>(xa));
      tmem_ld32(at + 32, reinterpret_cast<uint32_t*>(xb));
      load_scales(2 * half);
      tmem_ld_wait();
      if (!scaled)
        top = fmaxf(max_of(xa, f[0], f[1]), max_of(xb, f[2], f[3]));
      // (and P may now be written over all of S)
      tc_fence_before();
      float other;
      if (!exchange(top, nullptr, &other)) return;
      tc_fence_after();
      top = fmaxf(top, other);
    } else if (!scaled) {
#pragma unroll 1
      for (int q = 0; q < 4; q += 2) {
        tmem_ld32(s_addr + q * 32, reinterpret_cast<uint32_t*>(xa));
        tmem_ld32(s_addr + q * 32 + 32, reinterpret_cast<uint32_t*>(xb));
        load_scales(q);
        tmem_ld_wait();
        top = fmax3(top, max_of(xa, f[0], f[1]), max_of(xb, f[2], f[3]));
      }
    }
    // (selected, not branched on: the lanes stay together)
    const bool up_now = top > m_used + kTcRescaleLog2;
    float scale_o = up_now ? ex2_approx(m_used - top) : 1.f;  // 0 from -inf
    l_sum *= scale_o;
    m_used = up_now ? top : m_used;
    if (s.v_ref != ref) {
      scale_o *= ref / s.v_ref;
      ref = s.v_ref;
    }
    // ---- P; 2^9 goes along with it and the sums
    const float add = m_used == NEG_INF ? kTcUpLog2 : kTcUpLog2 - m_used;
    auto weigh64 = [&](int q) {  // xa, xb: pieces q, q + 1
      const float4 vl = *reinterpret_cast<const float4*>(&s.v_log2[2 * q]);
      const float4 vi = *reinterpret_cast<const float4*>(&s.v_inv[2 * q]);
      const float a[4] = {add + vl.x, add + vl.y, add + vl.z, add + vl.w};
      const float i[4] = {vi.x, vi.y, vi.z, vi.w};
      l_sum += weigh(xa, f, a, i, s_addr + q * 16);
      l_sum += weigh(xb, f + 2, a + 2, i + 2, s_addr + q * 16 + 16);
    };
    if (R == 1) {
      weigh64(2 * half);
    } else {
      // (P's columns lie before the next ones to be read)
#pragma unroll 1
      for (int q = 0; q < 4; q += 2) {
        tmem_ld32(s_addr + q * 32, reinterpret_cast<uint32_t*>(xa));
        tmem_ld32(s_addr + q * 32 + 32, reinterpret_cast<uint32_t*>(xb));
        load_scales(q);
        tmem_ld_wait();
        weigh64(q);
      }
    }
    if (__any_sync(0xffffffffu, scale_o != 1.f) && run_pv > 0) {
      if (!wait_pv(step - 1, 2)) return;
      tc_fence_after();
#pragma unroll 1
      for (int q = 0; q < kDims / 32; ++q) {
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
    ++run_pv;
    if (!s.last) {
      warp_arrive(&c->step_empty[step % kTcSteps]);
      continue;
    }
    // ---- the row's result, or its part of it; the next run's query first, as
    // its S may then go ahead
    const int b = s.b, head = s.hkv * G + (row < rows ? row : 0) / p.T;
    const int part_at = s.part;
    warp_arrive(&c->step_empty[step % kTcSteps]);
    if (!wait_step(tp, c, step + 1, kRoleScore)) return;
    if (c->steps[(step + 1) % kTcSteps].groups != 0)
      up = start_query(c->steps[(step + 1) % kTcSteps]);
    const bool there = pos >= 0;  // else an empty row, whatever it gathered
    float sum = there ? l_sum * pow2(-static_cast<int>(kTcUpLog2)) : 0.f;
    if (R == 1) {
      float other;
      if (!exchange(sum, &nans, &other)) return;
      sum += other;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) nans.w[i] |= c->pair_nan[half ^ 1][i][r];
    }
    if (!wait_pv(step, 3)) return;
    tc_fence_after();
    const float unit = ref * pow2(-static_cast<int>(kTcUpLog2));
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    constexpr int kPartRows = R * kTcRows;
    float* part = part_at < 0 ? nullptr
                              : p.parts + static_cast<int64_t>(part_at) *
                                              (kPartRows * (D + 2));
    const int in_part = tile * kTcRows + r;
#pragma unroll 1
    for (int q = 0; q < kDims / 32; ++q) {
      const int dim = half * kDims + q * 32;
      float o[32];
      tmem_ld32(o_addr + q * 32, reinterpret_cast<uint32_t*>(o));
      tmem_ld_wait();
      uint32_t nan = 0;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) nan = i * 32 == dim ? nans.w[i] : nan;
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = there ? o[j] * unit : 0.f;
      if (nan != 0)
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (nan >> j & 1u) o[j] = __int_as_float(0x7fffffff);
      if (row >= rows) {  // none
      } else if (part != nullptr) {  // [dim][row]: a warp's rows lie side by side
        float* dst = part + dim * kPartRows + in_part;
#pragma unroll
        for (int j = 0; j < 32; ++j) dst[j * kPartRows] = o[j];
      } else {
        uint16_t* dst =
            p.out + b * p.o_sb + head * p.o_sh + tq * p.o_ss + dim;
#pragma unroll
        for (int j = 0; j < 32; j += 8)
          st_global_v4(dst + j, pack_bf16x2(o[j] * inv, o[j + 1] * inv),
                       pack_bf16x2(o[j + 2] * inv, o[j + 3] * inv),
                       pack_bf16x2(o[j + 4] * inv, o[j + 5] * inv),
                       pack_bf16x2(o[j + 6] * inv, o[j + 7] * inv));
      }
      __syncwarp();  // (the next piece is the whole warp's to load)
    }
    tc_fence_before();
    mbar_arrive(&c->o_free[tile]);
    if (row < rows && half == 0) {
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
  }
}

// Joins the parts of items that were cut, and writes the rows of sequences
// without drafts: 32 rows (a lane each) and 16 dims per block, whose warps share
// the parts.  Parts lie [dim][row], so a warp reads its rows' elements of a dim
// at once; all loads of a part are on their way together.
constexpr int kJoinDims = 16, kJoinWarps = 4;

template <int D, int R>
__global__ void __launch_bounds__(32 * kJoinWarps)
    tree_join_kernel(const PagedParams p, const int grid) {
  using X = TcDeal;
  constexpr int kRows = R * kTcRows;
  __shared__ float top[kJoinWarps][32], total[kJoinWarps][32];
  __shared__ float part_x[kJoinWarps][kJoinDims][32];
  const int rows = p.H / p.H_kv * p.T;
  const int tiles = (rows + kRows - 1) / kRows;
  const int per = p.H_kv * tiles;
  const int b = blockIdx.z, item = blockIdx.y;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int dim = blockIdx.x % (D / kJoinDims) * kJoinDims;
  const int r = blockIdx.x / (D / kJoinDims) * 32 + lane;
  const int rr = item % tiles * kRows + r;
  const PaScan scan = scan_before<X>(p, b);
  const int64_t units = scan.all * per;
  const int n = plan_of<X>(p, b).n_units;
  // every block waits for the attention grid, so that work after this kernel
  // on the stream sees what that grid wrote itself
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int64_t c0 = 0, c1 = -1;
  if (n > 0) {
    const int64_t busy = busy_ctas<X>(units, grid);
    // the CTAs that hold its first and last unit
    const int64_t u0 = scan.before * per +
                       static_cast<int64_t>(item) * (n + X::kRunCost) +
                       X::kRunCost;
    auto cta_of = [&](int64_t u) {  // the last c with c * units / busy <= u
      const int64_t c = mul_div(u + 1, busy, units);
      return c - (c * units == (u + 1) * busy);
    };
    c0 = cta_of(u0), c1 = cta_of(u0 + n - 1);
    if (c0 == c1) return;  // whole in one CTA, which wrote it
  }
  const bool live = rr < rows && r < kRows;
  constexpr int64_t kPart = kRows * (D + 2);
  // the first CTA leaves its part in slot 1
  auto part_of = [&](int64_t c) {
    return p.parts + (c * 2 + (c == c0 ? 1 : 0)) * kPart + (live ? r : 0);
  };
  // a running maximum over this warp's parts
  float base = __int_as_float(0xff7fffff);  // as every part's before a key
  float sum = 0.f, x[kJoinDims];
#pragma unroll
  for (int i = 0; i < kJoinDims; ++i) x[i] = 0.f;
#pragma unroll 2
  for (int64_t c = c0 + warp; c <= c1; c += kJoinWarps) {
    const float* part = part_of(c);
    float y[kJoinDims];
#pragma unroll
    for (int i = 0; i < kJoinDims; ++i) y[i] = part[(dim + i) * kRows];
    const float m = part[kRows * D], l = part[kRows * D + kRows];
    const float to = fmaxf(base, m);
    const float f0 = ex2_approx(base - to), f1 = ex2_approx(m - to);
    base = to;
    sum = fmaf(l, f1, sum * f0);
#pragma unroll
    for (int i = 0; i < kJoinDims; ++i) x[i] = fmaf(y[i], f1, x[i] * f0);
  }
  top[warp][lane] = base;
  __syncthreads();
  float all = base;
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) all = fmaxf(all, top[i][lane]);
  const float f = ex2_approx(base - all);
  total[warp][lane] = sum * f;
#pragma unroll
  for (int i = 0; i < kJoinDims; ++i) part_x[warp][i][lane] = x[i] * f;
  __syncthreads();
  if (warp > 0 || !live) return;
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) sum += total[i][lane];
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int i = 0; i < kJoinDims; ++i) {
    x[i] = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) x[i] += part_x[w][i][lane];
    x[i] *= inv;
  }
  const int head = item / tiles * (p.H / p.H_kv) + rr / p.T, t = rr % p.T;
  uint16_t* dst = p.out + b * p.o_sb + head * p.o_sh + t * p.o_ss + dim;
#pragma unroll
  for (int i = 0; i < kJoinDims; i += 8)
    st_global_v4(dst + i, pack_bf16x2(x[i], x[i + 1]),
                 pack_bf16x2(x[i + 2], x[i + 3]),
                 pack_bf16x2(x[i + 4], x[i + 5]),
                 pack_bf16x2(x[i + 6], x[i + 7]));
  if (dim == 0 && p.lse != nullptr)
    p.lse[(static_cast<int64_t>(b) * p.H + head) * p.T + t] =
        sum != 0.f ? (all + log2f(sum)) * 0.6931471805599453f
                   : __int_as_float(0xff800000);
}

template <int D, int R, bool MOD>
__global__ void __launch_bounds__(kTcThreads, 1)
    paged_tree_kernel(const __grid_constant__ TcParams t) {
  using C = TcCfg<D, R>;
  extern __shared__ uint8_t smem_raw[];
  // (by an offset, so that the compiler knows it for shared memory)
  uint8_t* smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  TcCtl* c = reinterpret_cast<TcCtl*>(smem + C::kOffCtl);
  const int warp = threadIdx.x / 32, wg = threadIdx.x / 128;
  // the join kernel may be scheduled once every CTA here runs; it waits for
  // this grid's end before it reads the parts
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kConvertWarps = 4, kScoreWarps = 8;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kTcSteps; ++i) {
      mbar_init(&c->step_full[i], 1);
      mbar_init(&c->step_empty[i], 3 + kConvertWarps + kScoreWarps);
    }
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&c->code_full[i], 1);
      mbar_init(&c->code_empty[i], 4);
    }
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&c->kv_full[i], 4);
      mbar_init(&c->kv_empty[i], R);  // MMAs that read a tile
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c->q_full[i], kTcRows * C::kRowThreads);
      mbar_init(&c->s_full[i], 1);
      mbar_init(&c->p_full[i], kTcRows * C::kRowThreads);
      mbar_init(&c->pv_done[i], 1);
      mbar_init(&c->o_free[i], kTcRows * C::kRowThreads);
      mbar_init(&c->mma_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&c->meet[i], 2);
    c->abort = 0;
    c->nan_step[0] = c->nan_step[1] = 0;
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
    if (warp == 3) {
      load_role<D, R>(t, c, base + C::kOffCodes);
    } else if (warp > 0) {
      mma_role<D, R>(t, c, base, tmem, warp - 1);
    } else if (!t.no_plan) {
      plan_role<D, R>(t, c);
    }
  } else if (wg == 1) {
    convert_role<D, R>(t, c, base + C::kOffKv, base + C::kOffCodes);
  } else {
    score_role<D, R, MOD>(t, c, base, tmem, wg - 2);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTcTmem);
}

template <int D, int R, bool MOD>
cudaError_t launch_attend(const TcParams& t, int grid, cudaStream_t stream) {
  using C = TcCfg<D, R>;
  auto kern = paged_tree_kernel<D, R, MOD>;
  constexpr int smem = C::kOffCtl + static_cast<int>(sizeof(TcCtl)) + 1024;
  static_assert(smem <= 232448, "shared memory budget");
  cudaError_t e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           smem);
  if (e != cudaSuccess) return e;
  kern<<<grid, kTcThreads, smem, stream>>>(t);
  return cudaGetLastError();
}

template <int D, int R, bool MOD>
cudaError_t launch_tc(const TcParams& t, int num_sms, cudaStream_t stream) {
  const cudaError_t e = launch_attend<D, R, MOD>(t, num_sms, stream);
  if (e != cudaSuccess) return e;
  const int rows = t.p.H / t.p.H_kv * t.p.T;
  const int tiles = (rows + R * kTcRows - 1) / (R * kTcRows);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((min(rows, R * kTcRows) + 31) / 32 * (D / kJoinDims),
                     t.p.H_kv * tiles, t.p.B);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_join_kernel<D, R>, t.p, num_sms);
}

template <int D, int R>
cudaError_t launch_mod(const TcParams& t, int num_sms, cudaStream_t stream) {
  return t.p.mod.kind != 0 ? launch_tc<D, R, true>(t, num_sms, stream)
                           : launch_tc<D, R, false>(t, num_sms, stream);
}

}  // namespace

// Tiles of rows that a CTA works on: what does not fit one takes two at a time,
// for which each code is copied and converted once.
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
  t.no_plan = 0;
  const int tiles = tree_tiles(static_cast<int64_t>(p.H / p.H_kv) * p.T);
  if (p.D == 128)
    return tiles == 1 ? launch_mod<128, 1>(t, num_sms, stream)
                      : launch_mod<128, 2>(t, num_sms, stream);
  return tiles == 1 ? launch_mod<64, 1>(t, num_sms, stream)
                    : launch_mod<64, 2>(t, num_sms, stream);
}

cudaError_t launch_tree_selftest(uint64_t timeout_ns, cudaStream_t stream) {
  TcParams t = {};  // (no role gets to a pointer: each waits for its first step)
  t.p.H = t.p.H_kv = t.p.T = 1;
  t.p.D = 64;
  t.timeout_ns = timeout_ns;
  t.no_plan = 1;
  return launch_attend<64, 1, false>(t, 1, stream);
}

cudaError_t read_tree_error(int code, int32_t out[4]) {
  const size_t bytes = 4 * sizeof(int32_t), at = (code - 1) * bytes;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_tree_error, bytes, at);
  if (e != cudaSuccess) return e;
  const int32_t zero[4] = {0, 0, 0, 0};
  return cudaMemcpyToSymbol(g_tree_error, zero, bytes, at);
}

}  // namespace bsm
