// Block-sparse masked attention forward for sm_103a (GB300).  Two kernels:
// the lockstep one described here, and a variant whose two query tiles run as
// independent pipelines (see "Decoupled query tiles" below): at head dim 128
// for packed sequences (segment ids) and for any mask below 4096 keys, and for
// modified softmax scores (tanh cap, distance bias; see modify_tile) at both
// head dims, all but those with an arbitrary mask.
//
// One persistent CTA per SM takes work units of (batch, head, 256 query
// rows) from a counter in the caller's workspace, longest units first.  A
// unit is two 128-row query tiles that share one stream of
// 128-key KV tiles: the union of the nonzero blocks of both tiles, read from
// the mask-info block classes (hstu_ops `_next_nonzero`: 0 empty, 1
// partial, 2 full).  Empty KV tiles are never loaded (splash notes section
// 21); the element mask is evaluated on partial tiles only.
//
// Warp roles (384 threads, three warpgroups; the first gives registers to
// the other two with setmaxnreg):
//   warp 3      takes work units from the counter and builds each unit's
//               KV-tile list, up to two units ahead (three list buffers).
//   warp 0      issues TMA loads: Q per query tile, K and V tiles through a
//               ring of shared-memory slots (128-byte swizzle).
//   warps 1,2   one MMA issuer per query tile (warp 1 also allocates the 512
//               TMEM columns): the whole warp waits and issues, each
//               tcgen05 MMA going out from the lane elect.sync picks:
//               S_t = Q_t K^T (both operands in shared memory) and
//               O_t += P_t V (P_t read from TMEM, V from shared memory).
//   warps 4-7   score warpgroup of query tile 0, warps 8-11 of tile 1: one
//               thread per query row (its TMEM lane).  Softmax: online
//               max/sum with the correction of the splash notes section 15
//               (O is rescaled in TMEM only when the running max grew by more
//               than 2^8, which leaves the final O / l exact).  Pointwise:
//               x * sigmoid(x) / Sq with x = scale * q.k, masked -> 0
//               (hstu_ops fwd kernel).  P goes back to TMEM as bf16 over S.
//               In the instance used for long units without segment ids
//               the two score warps of each SM sub-partition take their
//               softmax turns alternately (see score_role).
// TMEM: S0/P0 cols [0,128), S1/P1 [128,256), O0 [256,256+D), O1 [384,384+D).
//
// Element mask of a partial tile (hstu_ops `_apply_mask`): each row's visible
// keys under causal / local / band masks -- and under segment ids when the kv
// ids are sorted, via the mask-info's per-row segment ranges -- are one
// interval, so the mask is a column-range test; unsorted segment ids are
// compared element by element and an arbitrary mask contributes its bits
// (both as per-column keep bits).  Key indices are the tile's true KV
// position.
#include <climits>
#include <cmath>
#include <cstdint>

#include "bsm_internal.h"
#include "bsm_ptx.cuh"

namespace bsm {

// Error record: [0] code (1 = wait timed out), [1] block, [2] role, [3] phase.
__device__ int g_fwd_error[4];

namespace {

constexpr int kThreads = 384;
// Register split: warpgroup 0 (load, MMA, list) drops to kRegsLight per
// thread, the two score warpgroups rise to kRegsScore.  Their sum must stay
// within what the CTA was launched with (kThreads x the kernel's register
// count), which the launcher checks.
constexpr uint32_t kRegsLight = 80, kRegsScore = 208;
constexpr int kRegsNeeded = 128 * kRegsLight + 256 * kRegsScore;
constexpr float kRescaleLog2 = 8.0f;
constexpr int kPingPongMin = 12;  // see score_role
// K/V ring slots at head dim 128, each holding one 128 x 128 K or V tile.
// Five (224 KB of shared memory with the two Q tiles) keep the long units'
// loads ahead of the alternating softmax turns; three were as fast on
// packed sequences but 9-12 % slower on long causal and local-window units.
constexpr int kSlots128 = 5;
constexpr uint32_t kTmemCols = 512;
constexpr int kRoleLoad = 1, kRoleMma = 2, kRoleScore = 3, kRoleList = 4;

template <int D>
struct Cfg {
  static constexpr int kKBlocks = D / 64;            // 128-byte k-blocks
  static constexpr int kTileBytes = kTileM * D * 2;  // Q, K or V tile
  static constexpr int kSlots = (D == 128) ? kSlots128 : 8;
  static constexpr int kOffQ = 0;
  static constexpr int kOffKV = 2 * kTileBytes;
  static constexpr int kOffBar = kOffKV + kSlots * kTileBytes;
  static constexpr int kSmemBytes = kOffBar + 512 + 1024;
};
static_assert(Cfg<128>::kSmemBytes <= 232448, "shared memory budget");

struct ListMeta {
  int n;          // entries (KV tiles) of the unit
  int n_t[2];     // entries used by query tile t
  int last_t[2];  // index of the last entry used by query tile t (-1: none)
  int unit;
  int b, h, st;   // the unit's batch row, head and 256-row super-tile
};

struct Bars {
  uint64_t list_full[kListBufs], list_free[kListBufs];
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[8], kv_empty[8];  // up to 8 ring slots
  uint64_t s_full[2], p_full[2], pv_done[2], o_free[2];
  // softmax turn of each score warp: [query tile][TMEM lane quarter]
  uint64_t sm_turn[2][4];
  uint64_t mma_done[2];
  uint32_t tmem_base;
  int abort;
  uint32_t trace_n[6];
  ListMeta meta[kListBufs];
};
static_assert(sizeof(Bars) <= 512, "barrier block");

__device__ __forceinline__ void record_timeout(int role, int phase) {
  if (atomicCAS(&g_fwd_error[0], 0, 1) == 0) {
    g_fwd_error[1] = blockIdx.x;
    g_fwd_error[2] = role;
    g_fwd_error[3] = phase;
  }
}

// Optional event trace.  CTA c owns records [c*(cap+2), (c+1)*(cap+2)):
// records 0-1 hold the event counts of the six recording threads (uint32
// each: load, MMA tile 0, score tile 0, score tile 1, list, MMA tile 1), then
// come six equal regions, each written by one thread with a plain counter.  A record is
// {globaltimer ns, role<<28 | event<<24 | tile<<20 | entry, unit}.
struct TraceRec {
  uint64_t t;
  uint32_t a, b;
};
enum : uint32_t {
  kEvListBuilt = 1, kEvQIssued = 2, kEvMmaUnit = 3, kEvMmaLastPv = 4,
  kEvSFull = 5, kEvPFull = 6, kEvEpiBegin = 7, kEvEpiEnd = 8, kEvRescale = 9,
  kEvEpiPvLanded = 10, kEvSIssued = 11, kEvPReady = 12, kEvPVIssued = 13,
  kEvEpiOLoaded = 14, kEvTmaIssued = 15
};

__device__ __forceinline__ void trace(const FwdParams& p, Bars* bars,
                                      uint32_t role, uint32_t ev, uint32_t tile,
                                      uint32_t entry, uint32_t unit) {
  if (p.trace == nullptr) return;
  const uint32_t slot = role == kRoleScore ? 2 + tile
                        : role == kRoleMma   ? (tile == 0 ? 1 : 5)
                        : role == kRoleList  ? 4
                                             : 0;
  const uint32_t per = p.trace_cap / 6;
  const uint32_t i = bars->trace_n[slot]++;
  if (i < per) {
    TraceRec* r = reinterpret_cast<TraceRec*>(p.trace) +
                  static_cast<size_t>(blockIdx.x) * (p.trace_cap + 2) + 2 +
                  slot * per + i;
    r->t = globaltimer_ns();
    r->a = (role << 28) | (ev << 24) | (tile << 20) | (entry & 0xFFFFFu);
    r->b = unit;
  }
}

// Warp-wide bounded wait: every lane polls, and the outcome is made uniform
// so that no lane runs a .sync.aligned instruction its siblings skip.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity,
                                          volatile int* abort_flag,
                                          uint64_t timeout_ns) {
  const bool ok = mbar_wait(bar, parity, abort_flag, timeout_ns);
  return __all_sync(0xffffffffu, ok);
}

struct UnitCoord {
  int b, h, st;
};

// Work unit u -> (batch, head, super-tile).  Units come in groups that
// share one (mask table, super-tile) pair: all heads of that batch row with
// one table per batch row, else all batch rows and heads.  The pairs are
// taken longest first when the mask info carries that order; otherwise the
// last super-tiles go first (under a causal mask the last rows see the most
// keys).
__device__ __forceinline__ UnitCoord decode_unit(const FwdParams& p, int u) {
  const int per = p.tables == 1 ? p.B * p.H : p.H;
  const int rank = u / per, r = u % per;
  int table, st;
  if (p.super_order != nullptr) {
    const int pr = p.super_order[rank];
    table = pr / p.n_super;
    st = pr % p.n_super;
  } else {
    table = rank % p.tables;
    st = p.n_super - 1 - rank / p.tables;
  }
  UnitCoord c;
  c.st = st;
  c.b = p.tables == 1 ? r / p.H : table;
  c.h = p.tables == 1 ? r % p.H : r;
  return c;
}

// Class of (128-row query tile starting at row R0) x (KV tile jt), combined
// from the mask-info blocks that cover it: 2 if all are full, 0 if all are
// empty, else 1.  A KV tile cut by the end of the keys is never full.
__device__ __forceinline__ int tile_class(const FwdParams& p, int table,
                                          int R0, int jt) {
  if (R0 >= p.Sq) return 0;
  const int R1 = min(p.Sq, R0 + kTileM) - 1;
  const int C0 = jt * kTileN;
  const int C1 = min(p.Skv, C0 + kTileN) - 1;
  const int i0 = R0 / p.bq, i1 = R1 / p.bq;
  const int j0 = C0 / p.bkv, j1 = C1 / p.bkv;
  const int8_t* bm =
      p.block_mask + static_cast<int64_t>(table) * p.mi_nq * p.mi_nk;
  bool all_full = true, any = false;
  for (int i = i0; i <= i1; ++i)
    for (int j = j0; j <= j1; ++j) {
      const int c = bm[static_cast<int64_t>(i) * p.mi_nk + j];
      all_full = all_full && (c == 2);
      any = any || (c != 0);
    }
  if (!any) return 0;
  if (all_full && C0 + kTileN <= p.Skv) return 2;
  return 1;
}

// Takes the next work unit from the launch's counter and builds its list
// into buffer ui % 3 (whole warp).  Entries are uint16: kv tile << 4 | class
// of query tile 0 << 2 | class of tile 1.  When no unit is left the buffer
// carries unit = -1, which ends every role's loop.
__device__ __forceinline__ bool build_list(const FwdParams& p, Bars* bars,
                                           uint16_t* lists, int ui) {
  const int lane = threadIdx.x % 32;
  const int buf = ui % kListBufs;
  if (!warp_wait(&bars->list_free[buf], ((ui / kListBufs) & 1) ^ 1,
                 &bars->abort, p.timeout_ns)) {
    if (lane == 0) record_timeout(kRoleList, 0);
    return false;
  }
  int unit = 0;
  if (lane == 0) unit = atomicAdd(p.unit_counter, 1);
  unit = __shfl_sync(0xffffffffu, unit, 0);
  if (unit >= p.num_units) {
    if (lane == 0) {
      bars->meta[buf].unit = -1;
      bars->meta[buf].n = 0;
      mbar_arrive(&bars->list_full[buf]);
    }
    __syncwarp();
    return true;
  }
  const UnitCoord uc = decode_unit(p, unit);
  const int table = (p.flags & BSM_MASK_SEGMENT) ? uc.b : 0;
  const int row0 = uc.st * kUnitRows;
  uint16_t* list = lists + buf * kMaxKvTiles;
  int n = 0, n0 = 0, n1 = 0, last0 = -1, last1 = -1;
  for (int base = 0; base < p.n_kvtiles; base += 64) {
    // two chunks of 32 tiles per pass so that their loads overlap
    int c[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int jt = base + 32 * h + lane;
      c[h][0] = c[h][1] = 0;
      if (jt < p.n_kvtiles) {
        c[h][0] = tile_class(p, table, row0, jt);
        c[h][1] = tile_class(p, table, row0 + kTileM, jt);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int jt = base + 32 * h + lane;
      const int c0 = c[h][0], c1 = c[h][1];
      const unsigned m = __ballot_sync(0xffffffffu, (c0 | c1) != 0);
      const int pos = n + __popc(m & ((1u << lane) - 1u));
      if (c0 | c1)
        list[pos] = static_cast<uint16_t>((jt << 4) | (c0 << 2) | c1);
      n0 += __popc(__ballot_sync(0xffffffffu, c0 != 0));
      n1 += __popc(__ballot_sync(0xffffffffu, c1 != 0));
      last0 = max(last0, __reduce_max_sync(0xffffffffu, c0 ? pos : -1));
      last1 = max(last1, __reduce_max_sync(0xffffffffu, c1 ? pos : -1));
      n += __popc(m);
    }
  }
  __syncwarp();
  if (lane == 0) {
    ListMeta& mt = bars->meta[buf];
    mt.n = n;
    mt.n_t[0] = n0;
    mt.n_t[1] = n1;
    mt.last_t[0] = last0;
    mt.last_t[1] = last1;
    mt.unit = unit;
    mt.b = uc.b;
    mt.h = uc.h;
    mt.st = uc.st;
    trace(p, bars, kRoleList, kEvListBuilt, 0, n, unit);
    mbar_arrive(&bars->list_full[buf]);
  }
  __syncwarp();
  return true;
}

// List-builder warp: stays up to two units ahead of the consumers.
__device__ __forceinline__ void list_role(const FwdParams& p, Bars* bars,
                                         uint16_t* lists) {
  for (int ui = 0;; ++ui) {
    if (!build_list(p, bars, lists, ui)) break;
    if (bars->meta[ui % kListBufs].unit < 0) break;  // sentinel written
  }
}

template <int D>
__device__ __forceinline__ void load_role(const FwdParams& p,
                                          const CUtensorMap* tq,
                                          const CUtensorMap* tk,
                                          const CUtensorMap* tv, uint8_t* smem,
                                          Bars* bars, uint16_t* lists) {
  using C = Cfg<D>;
  const int lane = threadIdx.x % 32;
  volatile int* abort_flag = &bars->abort;
  const uint64_t pol_q = l2_policy_evict_first();
  const uint64_t pol_kv = l2_policy_evict_last();
  uint32_t kv_it = 0;
  uint32_t q_it[2] = {0, 0};
  bool ok = true;
  for (int ui = 0; ok; ++ui) {
    const int buf = ui % kListBufs;
    ok = warp_wait(&bars->list_full[buf], (ui / kListBufs) & 1, abort_flag,
                   p.timeout_ns);
    if (!ok) {
      if (lane == 0) record_timeout(kRoleLoad, 0);
      break;
    }
    const ListMeta mt = bars->meta[buf];
    if (mt.unit < 0) break;
    const int unit = mt.unit;
    const uint16_t* list = lists + buf * kMaxKvTiles;
    const UnitCoord uc{mt.b, mt.h, mt.st};
    const int row0 = uc.st * kUnitRows;
    // Q, per query tile that has work in this unit
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (!ok || mt.n_t[t] == 0) continue;
      ok = warp_wait(&bars->q_empty[t], (q_it[t] & 1) ^ 1, abort_flag,
                     p.timeout_ns);
      if (!ok) {
        if (lane == 0) record_timeout(kRoleLoad, 1);
        break;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars->q_full[t], C::kTileBytes);
        for (int kb = 0; kb < C::kKBlocks; ++kb)
          tma_load_4d(tq, &bars->q_full[t],
                      smem + C::kOffQ + t * C::kTileBytes + kb * kTileM * 128,
                      kb * 64, row0 + t * kTileM, uc.h, uc.b, pol_q);
        trace(p, bars, kRoleLoad, kEvQIssued, t, 0, unit);
      }
      ++q_it[t];
    }
    const int hkv = uc.h / (p.H / p.Hkv);
    for (int e = 0; ok && e < mt.n; ++e) {
      const int jt = static_cast<int>(list[e] >> 4);
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        if (!ok) break;
        const int slot = kv_it % C::kSlots;
        const uint32_t ph = (kv_it / C::kSlots) & 1;
        ok = warp_wait(&bars->kv_empty[slot], ph ^ 1, abort_flag,
                       p.timeout_ns);
        if (!ok) {
          if (lane == 0) record_timeout(kRoleLoad, 2);
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars->kv_full[slot], C::kTileBytes);
          uint8_t* dst = smem + C::kOffKV + slot * C::kTileBytes;
          for (int kb = 0; kb < C::kKBlocks; ++kb)
            tma_load_4d(which == 0 ? tk : tv, &bars->kv_full[slot],
                        dst + kb * kTileN * 128, kb * 64, jt * kTileN, hkv,
                        uc.b, pol_kv);
          trace(p, bars, kRoleLoad, kEvTmaIssued, which, e, unit);
        }
        ++kv_it;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->list_free[buf]);
  }
  // Drain: wait for the loads already issued (after an abort some may still
  // be landing in shared memory); the last load into each barrier completes
  // the phase of parity (loads issued into it - 1) & 1.
  if (lane == 0) {
    for (int s = 0; s < C::kSlots; ++s) {
      const uint32_t n = kv_it > static_cast<uint32_t>(s)
                             ? (kv_it - 1 - s) / C::kSlots + 1 : 0;
      if (n > 0 && !mbar_wait_drain(&bars->kv_full[s], (n - 1) & 1,
                                    p.timeout_ns) && ok)
        record_timeout(kRoleLoad, 3);
    }
    for (int t = 0; t < 2; ++t)
      if (q_it[t] > 0 && !mbar_wait_drain(&bars->q_full[t], (q_it[t] - 1) & 1,
                                          p.timeout_ns) && ok)
        record_timeout(kRoleLoad, 4);
  }
  __syncwarp();
}

// MMA issuer of query tile t: warp 1 (tile 0) or warp 11 (tile 1).  The
// whole warp runs the loop, waits and issues together: each MMA and commit
// goes out from the lane elect.sync picks, the same lane every time (a
// commit tracks the MMAs of the thread that issues it).  The
// two issuers share the K/V ring: every slot is released by both (kv_empty
// counts two arrivals), and an issuer whose tile skips an entry still waits
// for that slot to be filled before releasing it, so the two never drift
// more than one ring cycle apart.
template <int D, int SCORE>
__device__ __forceinline__ void mma_role(const FwdParams& p, uint8_t* smem,
                                         Bars* bars, const uint16_t* lists,
                                         uint32_t tmem, const int t) {
  using C = Cfg<D>;
  const bool leader = (threadIdx.x % 32) == 0;
  volatile int* abort_flag = &bars->abort;
  constexpr uint32_t idesc_s = idesc_bf16_f32(kTileM, kTileN, false);
  constexpr uint32_t idesc_o = idesc_bf16_f32(kTileM, D, true);
  constexpr uint32_t kTileUnits = C::kTileBytes >> 4;
  // Descriptors of the tile bases; a K-step only adds to the start-address
  // field (16-byte units), which never carries into the upper fields.
  const uint64_t dq =
      sdesc_sw128(smem_u32(smem + C::kOffQ), 16, 1024) + t * kTileUnits;
  const uint64_t dkv0 = sdesc_sw128(smem_u32(smem + C::kOffKV), 16, 1024);
  const uint64_t dv0 =
      sdesc_sw128(smem_u32(smem + C::kOffKV), kTileN * 128, 1024);
  const uint32_t s_acc = tmem + t * 128;        // S_t, and P_t over it
  const uint32_t o_acc = tmem + 256 + t * 128;  // O_t
  uint32_t kv_it = 0, q_it = 0, s_cnt = 0;
  bool ok = true;

  auto wait_slot = [&](int& slot) -> bool {
    slot = kv_it % C::kSlots;
    const bool r = warp_wait(&bars->kv_full[slot], (kv_it / C::kSlots) & 1,
                             abort_flag, p.timeout_ns);
    ++kv_it;
    return r;
  };
  // S_t = Q_t K^T for the K tile in `kslot` (the whole warp; one lane
  // issues).
  auto issue_s = [&](int kslot) {
    const uint64_t b = dkv0 + kslot * kTileUnits;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint32_t off = (k >> 2) * (kTileM * 128 / 16) + (k & 3) * 2;
      mma_ss_elect(s_acc, dq + off, b + off, idesc_s, k > 0 ? 1u : 0u);
    }
    mma_commit_elect(&bars->s_full[t]);
  };
  auto fail = [&](int where) {
    if (leader) record_timeout(kRoleMma, where);
  };

  for (int ui = 0; ok; ++ui) {
    const int buf = ui % kListBufs;
    ok = warp_wait(&bars->list_full[buf], (ui / kListBufs) & 1, abort_flag,
                   p.timeout_ns);
    if (!ok) {
      fail(0);
      break;
    }
    const ListMeta mt = bars->meta[buf];
    if (mt.unit < 0) break;
    const int unit = mt.unit;
    const uint16_t* list = lists + buf * kMaxKvTiles;
    const int shift = t == 0 ? 2 : 0;
    if (leader) trace(p, bars, kRoleMma, kEvMmaUnit, t, mt.n, unit);
    bool q_ready = false, first_pv = true;
    bool s_ahead = false;  // S_t of the current entry already issued
    int kslot_ahead = -1;  // K slot of the current entry if waited ahead
    uint32_t nxt = mt.n > 0 ? list[0] : 0u;  // list entries are read one ahead
    for (int e = 0; e < mt.n && ok; ++e) {
      const bool use = ((nxt >> shift) & 3u) != 0;
      nxt = (e + 1 < mt.n) ? list[e + 1] : 0u;
      const bool use_next = (e + 1 < mt.n) && ((nxt >> shift) & 3u) != 0;
      // ---- K of this entry
      int kslot = kslot_ahead;
      if (kslot < 0 && !(ok = wait_slot(kslot))) {
        fail(2);
        break;
      }
      kslot_ahead = -1;
      if (use && !s_ahead) {
        if (!q_ready) {
          q_ready = true;
          if (!(ok = warp_wait(&bars->q_full[t], q_it & 1, abort_flag,
                               p.timeout_ns))) {
            fail(1);
            break;
          }
        }
        tc_fence_after();
        issue_s(kslot);
        if (leader) trace(p, bars, kRoleMma, kEvSIssued, t, e, unit);
        ++s_cnt;
      }
      if (use && e == mt.last_t[t])  // Q_t of this unit no longer needed
        mma_commit_elect(&bars->q_empty[t]);
      // release the K slot once the S MMA that read it has completed
      if (use)
        mma_commit_elect(&bars->kv_empty[kslot]);
      else if (leader)
        mbar_arrive(&bars->kv_empty[kslot]);
      if (use && e == mt.last_t[t]) ++q_it;
      __syncwarp();
      // ---- V of this entry: O_t += P_t V, then S_t of the next entry
      int vslot;
      if (!(ok = wait_slot(vslot))) {
        fail(4);
        break;
      }
      s_ahead = false;
      if (!use) {
        if (leader) mbar_arrive(&bars->kv_empty[vslot]);
        __syncwarp();
        continue;
      }
      ok = warp_wait(&bars->p_full[t], (s_cnt - 1) & 1, abort_flag,
                     p.timeout_ns);
      if (ok && first_pv)
        ok = warp_wait(&bars->o_free[t], (ui & 1) ^ 1, abort_flag,
                       p.timeout_ns);
      if (!ok) {
        fail(5);
        break;
      }
      {
        if (leader) trace(p, bars, kRoleMma, kEvPReady, t, e, unit);
        tc_fence_after();
        const uint64_t b = dv0 + vslot * kTileUnits;
        if (SCORE == BSM_SCORE_SOFTMAX) {
          // P: key 16kk..16kk+15 in TMEM columns 8kk..8kk+7
#pragma unroll
          for (int kk = 0; kk < kTileN / 16; ++kk)
            mma_ts_elect(o_acc, s_acc + kk * 8, b + kk * (16 * 128 / 16),
                         idesc_o, (kk > 0 || !first_pv) ? 1u : 0u);
        } else {
          // P = hi + lo, per 64-key half h: hi in columns 64h..64h+31, lo in
          // 64h+32..64h+63
#pragma unroll 2
          for (int kk = 0; kk < kTileN / 16; ++kk) {
            const uint32_t col = (kk >> 2) * 64 + (kk & 3) * 8;
            mma_ts_elect(o_acc, s_acc + col, b + kk * (16 * 128 / 16),
                         idesc_o, (kk > 0 || !first_pv) ? 1u : 0u);
            mma_ts_elect(o_acc, s_acc + col + 32, b + kk * (16 * 128 / 16),
                         idesc_o, 1u);
          }
        }
        mma_commit_elect(&bars->pv_done[t]);
        if (leader) trace(p, bars, kRoleMma, kEvPVIssued, t, e, unit);
      }
      first_pv = false;
      // S_t of the next entry goes right behind this P.V.  It overwrites the
      // TMEM columns the P.V just read: tcgen05.mma instructions of one
      // thread run in the order they were issued.
      if (use_next) {
        if (!(ok = wait_slot(kslot_ahead))) {
          fail(2);
          break;
        }
        tc_fence_after();
        issue_s(kslot_ahead);
        if (leader) trace(p, bars, kRoleMma, kEvSIssued, t, e + 1, unit);
        ++s_cnt;
        s_ahead = true;
      }
      mma_commit_elect(&bars->kv_empty[vslot]);
      __syncwarp();
    }
    if (!ok) break;
    if (leader) {
      trace(p, bars, kRoleMma, kEvMmaLastPv, t, mt.n, unit);
      mbar_arrive(&bars->list_free[buf]);
    }
    __syncwarp();
  }
  // Drain: every MMA issued above has completed once this arrives (waited
  // for also after an abort, before the CTA frees TMEM).
  __syncwarp();
  mma_commit_elect(&bars->mma_done[t]);
  if (leader && !mbar_wait_drain(&bars->mma_done[t], 0, p.timeout_ns) && ok)
    record_timeout(kRoleMma, 6);
  __syncwarp();
}

// "Same segment" bits of the 128 keys of a tile for one row (unsorted
// segment ids), one 32-bit word per 32 keys.  Computed before S is loaded
// from TMEM, so the loads never compete with S for registers.
template <int NC = kTileN>
__device__ __forceinline__ void segment_bits(uint32_t keep[4],
                                             const int32_t* segk, int nvalid,
                                             int segq) {
  const bool vec =
      nvalid == NC && (reinterpret_cast<uintptr_t>(segk) & 15u) == 0;
#pragma unroll 1
  for (int w = 0; w < NC / 32; ++w) {
    uint32_t bits = 0;
    if (vec) {
      const int4* s4 = reinterpret_cast<const int4*>(segk + 32 * w);
#pragma unroll
      for (int c4 = 0; c4 < 8; ++c4) {
        const int4 v = __ldg(s4 + c4);
        bits |= (v.x == segq ? 1u : 0u) << (4 * c4);
        bits |= (v.y == segq ? 1u : 0u) << (4 * c4 + 1);
        bits |= (v.z == segq ? 1u : 0u) << (4 * c4 + 2);
        bits |= (v.w == segq ? 1u : 0u) << (4 * c4 + 3);
      }
    } else {
#pragma unroll 8
      for (int c = 0; c < 32; ++c) {
        const int k = 32 * w + c;
        if (k < nvalid && __ldg(segk + k) == segq) bits |= 1u << c;
      }
    }
    keep[0] = w == 0 ? bits : keep[0];
    keep[1] = w == 1 ? bits : keep[1];
    keep[2] = w == 2 ? bits : keep[2];
    keep[3] = w == 3 ? bits : keep[3];
  }
}

// Masks S of a partial tile in place: columns outside [lo_c, hi_c] (and,
// with use_keep, columns whose keep bit is clear) become -inf.  Each thread
// holds one row.  Per 32-column chunk the row's visible columns are built as
// one bit word from the two bounds; a chunk that all 32 rows of the warp see
// whole (a warp-uniform test) is left alone, the others cost one bit test
// and one select per column.  Under causal and packed-segment masks most
// chunks of a partial tile are whole for the warp.  (fill: instead of -inf.)
template <int NC = kTileN>
__device__ __forceinline__ void mask_tile(
    float* s, int lo_c, int hi_c, const uint32_t* keep, bool use_keep,
    float fill = -INFINITY) {
#pragma unroll
  for (int q = 0; q < NC / 32; ++q) {
    const int c0 = 32 * q;
    // visible columns of this chunk as bits: [lo_c, hi_c] cut to the chunk
    const int lb = min(max(lo_c - c0, 0), 32), hb = min(max(hi_c - c0 + 1, 0), 32);
    const uint32_t below_hi = hb >= 32 ? 0xffffffffu : (1u << hb) - 1u;
    const uint32_t below_lo = lb >= 32 ? 0xffffffffu : (1u << lb) - 1u;
    uint32_t vm = below_hi & ~below_lo;
    if (use_keep) vm &= keep[q];
    if (!__all_sync(0xffffffffu, vm == 0xffffffffu)) {
#pragma unroll
      for (int c = 0; c < 32; ++c)
        s[c0 + c] = (vm & (1u << c)) ? s[c0 + c] : fill;
    }
  }
}

// s = s * (c[0] + c[1] s^2 + ...), with kModBias + the bias of the column's
// place among eight.
template <int MOD, int NC, int N>
__device__ __forceinline__ void cap_tile(float* s, const float* c,
                                         const float* pc) {
#pragma unroll
  for (int j = 0; j < NC; j += 2) {
    float h0, h1;
    poly_sq2<N>(h0, h1, s[j], s[j + 1], c);
    if (MOD & kModBias)
      ffma2v(s[j], s[j + 1], s[j], s[j + 1], h0, h1, pc[j & 7],
             pc[(j & 7) + 1]);
    else
      fmul2v(s[j], s[j + 1], s[j], s[j + 1], h0, h1);
  }
}

// Modified scores of one row's NC columns, in place and in log2 units: from
// S = q.k to cap * tanh(scale S / cap) (kModCap) or scale S, minus slope *
// |q - k| (kModBias; slope2 = slope * log2(e)).
//
// tanh.  Where every |S| of the warp's rows lies within poly_max (|y| <= 0.5),
// an odd polynomial of degree 7 on the paired f32 pipe, off by 5.5e-7 of its
// value; no MUFU operation.  (The backward's second polynomial, of degree 13,
// was no faster here than the exponential.)  Else 1 - 2 / (1 + e^(2 y)), one reciprocal for two
// columns, to a few 2^-23 of the cap; e^(2 y) is cut at 2^60, where tanh is 1
// in f32, so that the product of two stays in range.  NaN stays NaN in both, and
// would reach the neighbour through the reciprocal they share: where the warp
// holds a NaN, the columns that a row of a partial tile does not see, whose
// score may be anything, are set to 0 before (a NaN that a row sees makes the
// whole row NaN in any case).
// (tanh.approx is off by up to 2^-11 of its value, which the logsumexp would
// show.)  What bounds it: the f32 pipe and the latency of the softmax, which
// the tensor core waits for.  Measured on packed S=8192, 2 x 16 heads, against
// 120 us unmodified: cap 50 183 us with an exponential and a reciprocal per
// column, 145 us with the polynomial.
//
// Bias (where the tensor core does not add it, see kDtOffBias).  All columns of
// a tile that lie on one side of the row have bias
// sl (kbase - qrow + c), sl = +-slope2: column c gets sl (c % 8) here, in the
// same paired operation that scales S, and *base = sl (kbase - qrow); the
// caller adds sl 8 (c / 8) + *base per 8 columns.  A tile with columns on both
// sides that no causal mask cuts takes the bias whole, column by column.
//
// partial, lo_c, hi_c, keep, use_keep: the row's visible columns, as mask_tile
// takes them, if the tile is partial.
template <int MOD, int NC>
__device__ __forceinline__ void modify_tile(float* s, const FwdParams& p,
                                            int kbase, int qrow, bool partial,
                                            int lo_c, int hi_c,
                                            const uint32_t* keep, bool use_keep,
                                            float slope2, float* sl_out,
                                            float* base_out) {
  float pc[8];  // bias of columns 0-7 of a chunk
  bool split = false;
  if (MOD & kModBias) {
    const int lane = threadIdx.x % 32;
    const int first = qrow - lane;  // the warp's rows: first .. first + 31
    const bool left =
        (p.flags & BSM_MASK_CAUSAL) != 0 || kbase + NC - 1 <= first;
    split = !left && kbase < first + 31;  // warp-uniform
    const float sl = split ? 0.f : left ? slope2 : -slope2;
#pragma unroll
    for (int c = 0; c < 8; ++c) pc[c] = sl * static_cast<float>(c);
    *sl_out = 8.f * sl;
    *base_out = sl * static_cast<float>(kbase - qrow);
  }
  if (MOD & kModCap) {
    float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
    for (int c = 0; c < NC; c += 8) {
      a0 = fmax3_abs_nan(a0, s[c], s[c + 1]);
      a1 = fmax3_abs_nan(a1, s[c + 2], s[c + 3]);
      a2 = fmax3_abs_nan(a2, s[c + 4], s[c + 5]);
      a3 = fmax3_abs_nan(a3, s[c + 6], s[c + 7]);
    }
    float top = fmax3_abs_nan(fmax3_abs_nan(a0, a1, a2), a3, a3);
    bool near = __all_sync(0xffffffffu, top <= p.mod.poly_max);
    if (near) {
      cap_tile<MOD, NC, 4>(s, p.mod.poly, pc);
    } else if (__any_sync(0xffffffffu, top != top)) {
      if (partial) mask_tile<NC>(s, lo_c, hi_c, keep, use_keep, 0.f);
      top = 0.f;  // of what is no NaN
#pragma unroll
      for (int c = 0; c < NC; c += 2) top = fmax3_abs(top, s[c], s[c + 1]);
      near = __all_sync(0xffffffffu, top <= p.mod.poly_max);
      if (near) cap_tile<MOD, NC, 4>(s, p.mod.poly, pc);
    }
    if (!near) {
      const float k2 = -2.f * p.mod.cap_log2, k0 = p.mod.cap_log2;
#pragma unroll
      for (int c = 0; c < NC; c += 2) {
        float e0, e1;
        fmul2(e0, e1, s[c], s[c + 1], p.mod.cap_e);
        e0 = ex2_approx(fmin_nan(e0, 60.f));
        e1 = ex2_approx(fmin_nan(e1, 60.f));
        fadd2(e0, e1, e0, e1, 1.f, 1.f);
        const float r = rcp_approx(e0 * e1) * k2;
        if (MOD & kModBias)
          ffma2v(s[c], s[c + 1], e1, e0, r, r, k0 + pc[c & 7],
                 k0 + pc[(c & 7) + 1]);
        else
          ffma2v(s[c], s[c + 1], e1, e0, r, r, k0, k0);
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < NC; c += 2)
      ffma2v(s[c], s[c + 1], s[c], s[c + 1], p.scale_log2, p.scale_log2,
             pc[c & 7], pc[(c & 7) + 1]);
  }
  if ((MOD & kModBias) && split) {
    const float d0 = static_cast<float>(kbase - qrow);
#pragma unroll
    for (int c = 0; c < NC; ++c)
      s[c] = fmaf(-slope2, fabsf(d0 + c), s[c]);
  }
}

// Row maximum of a tile whose bias per 8 columns is sl8 (c / 8) + base, to be
// added to s.
template <int NC>
__device__ __forceinline__ float biased_max(const float* s, float sl8,
                                            float base) {
  float mx[2];
#pragma unroll
  for (int i = 0; i < NC / 8; ++i) {
    const float* t = s + 8 * i;
    const float m = fmax3(fmax3(t[0], t[1], t[2]), fmax3(t[3], t[4], t[5]),
                          fmaxf(t[6], t[7])) +
                    fmaf(sl8, static_cast<float>(i), base);
    mx[i & 1] = i < 2 ? m : fmaxf(mx[i & 1], m);
  }
  return fmaxf(mx[0], mx[1]);
}

// Floor of log2(x) for a positive normal x.
__device__ __forceinline__ float exponent_of(float x) {
  return static_cast<float>(static_cast<int>(__float_as_uint(x) >> 23) - 127);
}

// Whether a row saw a key.  With modified scores a sum of NaN counts (and the
// logsumexp becomes NaN); without, such rows have always had -inf.
template <int MOD>
__device__ __forceinline__ bool has_sum(float l_sum) {
  return MOD != 0 ? l_sum != 0.f : l_sum > 0.f;
}

// KEEP: partial tiles also carry per-element "keep" bits -- from segment ids
// compared element by element (some key-id row is not sorted) and/or from
// an arbitrary bit-packed mask; otherwise every mask is a key range per row.
template <int D, int SCORE, int MOD, bool KEEP, bool PINGPONG>
__device__ __forceinline__ void score_role(const FwdParams& p, Bars* bars,
                                           const uint16_t* lists,
                                           uint32_t tmem) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int t = (warp - 4) / 4;  // query tile of this warpgroup
  const int quarter = warp % 4;  // TMEM lane quarter this warp may access
  const int r = quarter * 32 + lane;
  const bool tracer = (r == 0);
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t s_addr = tmem + lane_off + t * 128;
  const uint32_t o_addr = tmem + lane_off + 256 + t * 128;
  volatile int* abort_flag = &bars->abort;
  const float NEG_INF = __int_as_float(0xff800000);
  const bool seg = (p.flags & BSM_MASK_SEGMENT) != 0;
  const bool seg_elem = KEEP && seg && (*p.seg_flags & 1) != 0;
  const bool dense = KEEP && p.dense != nullptr;
  uint32_t s_cnt = 0, pv_cnt = 0, turns = 0;
  auto pass_turn = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->sm_turn[1 - t][quarter]);
  };
  for (int ui = 0;; ++ui) {
    const int buf = ui % kListBufs;
    if (!warp_wait(&bars->list_full[buf], (ui / kListBufs) & 1, abort_flag,
                   p.timeout_ns)) {
      record_timeout(kRoleScore, 0);
      break;
    }
    const int unit = bars->meta[buf].unit;
    if (unit < 0) break;
    const int n_ent = bars->meta[buf].n;
    const UnitCoord uc{bars->meta[buf].b, bars->meta[buf].h,
                       bars->meta[buf].st};
    const uint16_t* list = lists + buf * kMaxKvTiles;
    const int qrow = uc.st * kUnitRows + t * kTileM + r;
    const bool row_ok = qrow < p.Sq;
    // visible keys of this row form [rlo, rhi] (plus the element compare of
    // unsorted segment ids)
    int rlo = 0, rhi = p.Skv - 1;
    if (p.flags & BSM_MASK_CAUSAL) rhi = min(rhi, qrow);
    if (p.flags & BSM_MASK_LOCAL) rlo = max(rlo, qrow - p.window + 1);
    if (p.flags & BSM_MASK_BAND) rhi = min(rhi, qrow + p.window - 1);
    int segq = 0;
    if (seg && row_ok) {
      const int64_t qi = static_cast<int64_t>(uc.b) * p.Sq + qrow;
      if (seg_elem) {
        segq = p.q_seg[qi];
      } else {
        const int2 sr = reinterpret_cast<const int2*>(p.seg_range)[qi];
        rlo = max(rlo, sr.x);
        rhi = min(rhi, sr.y);
      }
    }
    const int32_t* segk_b =
        seg_elem ? p.kv_seg + static_cast<int64_t>(uc.b) * p.Skv : nullptr;
    float m_used = NEG_INF, l_sum = 0.f;
    const float slope2 = (MOD & kModBias) && p.mod.slopes != nullptr
                             ? p.mod.slopes[uc.h] * 1.4426950408889634f
                             : 0.f;
    uint32_t unit_pv = 0;
    bool ok = true;
    for (int e = 0; e < n_ent; ++e) {
      const uint32_t ent = list[e];
      const int cls = t == 0 ? static_cast<int>((ent >> 2) & 3u)
                             : static_cast<int>(ent & 3u);
      if (!cls) continue;
      // On entries both tiles use, softmax turns alternate between the two
      // score warps that share an SM sub-partition (same lane quarter,
      // tiles 0 and 1; tile 0 first): one works while the tensor core runs
      // the other tile's P.V and next S, instead of both competing for the
      // same issue slots and MUFU at once.
      // (only in units of at least kPingPongMin entries: in a short unit
      // the two tiles would spend a softmax setting up the alternation)
      const bool shared = PINGPONG && n_ent >= kPingPongMin &&
                          ((ent >> 2) & 3u) != 0 && (ent & 3u) != 0;
      if (shared) {
        ok = warp_wait(&bars->sm_turn[t][quarter],
                       (turns & 1) ^ (t == 0 ? 1u : 0u), abort_flag,
                       p.timeout_ns);
        if (!ok) {
          record_timeout(kRoleScore, 6);
          break;
        }
        ++turns;
      }
      const int jt = static_cast<int>(ent >> 4);
      const int kbase = jt * kTileN;
      uint32_t keep[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
      if (KEEP && cls == 1) {
        if (seg_elem)
          segment_bits(keep, segk_b + kbase, min(kTileN, p.Skv - kbase), segq);
        if (dense) {  // the row's mask words for these 128 keys
          const int64_t w0 = kbase >> 5;
          const uint32_t* dw =
              p.dense + static_cast<int64_t>(row_ok ? qrow : 0) * p.dense_words;
#pragma unroll
          for (int w = 0; w < 4; ++w)
            keep[w] &= (row_ok && w0 + w < p.dense_words) ? __ldg(dw + w0 + w)
                                                          : 0u;
        }
      }
      ok = warp_wait(&bars->s_full[t], s_cnt & 1, abort_flag, p.timeout_ns);
      if (!ok) {
        record_timeout(kRoleScore, 1);
        break;
      }
      ++s_cnt;
      if (tracer) trace(p, bars, kRoleScore, kEvSFull, t, e, unit);
      tc_fence_after();
      uint32_t sraw[kTileN];
#pragma unroll
      for (int q = 0; q < kTileN / 32; ++q)
        tmem_ld32(s_addr + q * 32, sraw + q * 32);
      tmem_ld_wait();
      float* s = reinterpret_cast<float*>(sraw);
      float sl8 = 0.f, cbase = 0.f;  // bias of each 8 columns (kModBias)
      if (MOD != 0)
        modify_tile<MOD, kTileN>(s, p, kbase, qrow, cls == 1, rlo - kbase,
                                 rhi - kbase, keep, KEEP, slope2, &sl8, &cbase);
      if (cls == 1) mask_tile(s, rlo - kbase, rhi - kbase, keep, KEEP);

      uint32_t pk[16];
      if (SCORE == BSM_SCORE_SOFTMAX) {
        float m_blk;
        if (MOD == 0) {
          // row max: three-input max, four independent chains
          float mx0 = fmaxf(s[0], s[1]), mx1 = fmaxf(s[2], s[3]);
          float mx2 = fmaxf(s[4], s[5]), mx3 = fmaxf(s[6], s[7]);
#pragma unroll
          for (int c = 8; c < kTileN; c += 8) {
            mx0 = fmax3(mx0, s[c], s[c + 1]);
            mx1 = fmax3(mx1, s[c + 2], s[c + 3]);
            mx2 = fmax3(mx2, s[c + 4], s[c + 5]);
            mx3 = fmax3(mx3, s[c + 6], s[c + 7]);
          }
          const float mx = fmax3(mx0, mx1, fmaxf(mx2, mx3));
          m_blk = mx * p.scale_log2;
        } else {
          m_blk = biased_max<kTileN>(s, sl8, cbase);
        }
        bool rescale = false;
        float alpha = 1.f;
        if (m_blk > m_used + kRescaleLog2) {
          if (m_used != NEG_INF) {
            alpha = ex2_approx(m_used - m_blk);
            rescale = true;
          }
          l_sum *= alpha;
          m_used = m_blk;
        }
        const float neg_m = (m_used == NEG_INF) ? 0.f : -m_used;
        float ls0 = 0.f, ls1 = 0.f, ls2 = 0.f, ls3 = 0.f;
#pragma unroll
        for (int q = 0; q < kTileN / 32; ++q) {  // 32 columns at a time
#pragma unroll
          for (int c = 32 * q; c < 32 * q + 32; c += 4) {
            // paired f32 FMA/add: the same roundings as one element at a time
            float x0, x1, x2, x3;
            if (MOD == 0) {
              ffma2(x0, x1, s[c], s[c + 1], p.scale_log2, neg_m);
              ffma2(x2, x3, s[c + 2], s[c + 3], p.scale_log2, neg_m);
            } else {
              const float add =
                  fmaf(sl8, static_cast<float>(c / 8), cbase + neg_m);
              fadd2(x0, x1, s[c], s[c + 1], add, add);
              fadd2(x2, x3, s[c + 2], s[c + 3], add, add);
            }
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            const float p2 = ex2_approx(x2), p3 = ex2_approx(x3);
            fadd2(ls0, ls1, ls0, ls1, p0, p1);
            fadd2(ls2, ls3, ls2, ls3, p2, p3);
            pk[(c & 31) / 2] = pack_bf16x2(p0, p1);
            pk[(c & 31) / 2 + 1] = pack_bf16x2(p2, p3);
          }
          tmem_st16(s_addr + q * 16, pk);
        }
        l_sum += (ls0 + ls1) + (ls2 + ls3);
        // Rescale O_t (needs the previous PV of this tile to have landed).
        if (__any_sync(0xffffffffu, rescale) && unit_pv > 0) {
          ok = warp_wait(&bars->pv_done[t], (pv_cnt - 1) & 1, abort_flag,
                         p.timeout_ns);
          if (!ok) {
            record_timeout(kRoleScore, 2);
            break;
          }
          if (tracer) trace(p, bars, kRoleScore, kEvRescale, t, e, unit);
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(o_addr + q * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 32; ++c)
              o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
            tmem_st32(o_addr + q * 32, o);
          }
        }
      } else {
        // pointwise: x = scale*qk; p = x*sigmoid(x)/Sq; masked (-inf) -> 0.
        // With sigmoid(x) = (1 + tanh(x/2)) / 2 this is g + g*tanh(x/2),
        // g = x / (2 Sq): one tanh per element, the rest on paired f32.
        // hstu_ops multiplies the f32 scores by f32 v, so p is kept to about
        // 16 bits: p = hi + lo, both bf16 (lo = p - hi is exact in f32).
        // Each 64-key half's hi and lo (32 columns each) go back over that
        // half's own 64 columns of S; the MMA warp adds both products into O.
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t pl[16];
#pragma unroll
            for (int c = 64 * hf + 32 * q; c < 64 * hf + 32 * q + 32; c += 2) {
              float h0, h1, g0, g1, p0, p1;
              fmul2(h0, h1, s[c], s[c + 1], p.pw_half);
              fmul2(g0, g1, s[c], s[c + 1], p.pw_g);
              ffma2v(p0, p1, g0, g1, tanh_approx(h0), tanh_approx(h1), g0,
                     g1);
              p0 = s[c] != NEG_INF ? p0 : 0.f;
              p1 = s[c + 1] != NEG_INF ? p1 : 0.f;
              const uint32_t hi = pack_bf16x2(p0, p1);
              pk[(c & 31) / 2] = hi;
              pl[(c & 31) / 2] =
                  pack_bf16x2(p0 - __uint_as_float(hi << 16),
                              p1 - __uint_as_float(hi & 0xffff0000u));
            }
            tmem_st16(s_addr + hf * 64 + q * 16, pk);
            tmem_st16(s_addr + hf * 64 + 32 + q * 16, pl);
          }
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bars->p_full[t]);
      if (shared) pass_turn();
      if (tracer) trace(p, bars, kRoleScore, kEvPFull, t, e, unit);
      ++pv_cnt;
      ++unit_pv;
    }
    if (!ok) break;

    // ---- epilogue: out = O / l (softmax) or O (pointwise), bf16
    if (tracer) trace(p, bars, kRoleScore, kEvEpiBegin, t, 0, unit);
    uint16_t* orow = p.out + static_cast<int64_t>(uc.b) * p.o_sb +
                     static_cast<int64_t>(uc.h) * p.o_sh +
                     static_cast<int64_t>(qrow) * p.o_ss;
    if (unit_pv > 0) {
      if (!warp_wait(&bars->pv_done[t], (pv_cnt - 1) & 1, abort_flag,
                     p.timeout_ns)) {
        record_timeout(kRoleScore, 3);
        break;
      }
      if (tracer) trace(p, bars, kRoleScore, kEvEpiPvLanded, t, 0, unit);
      tc_fence_after();
      // all of O_t into registers with one wait; the next unit's first P.V
      // may then overwrite it while the stores go out
      uint32_t o[D];
#pragma unroll
      for (int q = 0; q < D / 32; ++q) tmem_ld32(o_addr + q * 32, o + q * 32);
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(&bars->o_free[t]);
      if (tracer) trace(p, bars, kRoleScore, kEvEpiOLoaded, t, 0, unit);
      float inv = 1.f;
      if (SCORE == BSM_SCORE_SOFTMAX) inv = has_sum<MOD>(l_sum) ? 1.f / l_sum : 0.f;
      if (row_ok) {
        // 32 bytes per store where the row alignment allows: each warp
        // store touches 32 rows, so fewer, wider stores cost fewer requests
        const bool v8 = p.o_vec8 != 0;
#pragma unroll
        for (int v = 0; v < D / 16; ++v) {
          uint32_t w[8];
#pragma unroll
          for (int c = 0; c < 8; ++c)
            w[c] = pack_bf16x2(__uint_as_float(o[16 * v + 2 * c]) * inv,
                               __uint_as_float(o[16 * v + 2 * c + 1]) * inv);
          if (v8) {
            st_global_v8(orow + v * 16, w);
          } else {
            st_global_v4(orow + v * 16, w[0], w[1], w[2], w[3]);
            st_global_v4(orow + v * 16 + 8, w[4], w[5], w[6], w[7]);
          }
        }
      }
    } else {
      if (row_ok) {
#pragma unroll
        for (int v = 0; v < D / 8; ++v)
          st_global_v4(orow + v * 8, 0u, 0u, 0u, 0u);
      }
      tc_fence_before();
      mbar_arrive(&bars->o_free[t]);
    }
    if (SCORE == BSM_SCORE_SOFTMAX && p.lse != nullptr && row_ok) {
      const float lse = has_sum<MOD>(l_sum)
                            ? (m_used + log2f(l_sum)) * 0.6931471805599453f
                            : NEG_INF;
      p.lse[(static_cast<int64_t>(uc.b) * p.H + uc.h) * p.Sq + qrow] = lse;
    }
    mbar_arrive(&bars->list_free[buf]);
    if (tracer) trace(p, bars, kRoleScore, kEvEpiEnd, t, 0, unit);
  }
}

template <int D, int SCORE, int MOD, bool PINGPONG>
__global__ void __launch_bounds__(kThreads, 1)
    splash_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v,
                      const FwdParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kOffBar);
  uint16_t* lists = p.lists + static_cast<size_t>(blockIdx.x) * kListBufs *
                                  kMaxKvTiles;
  const int warp = threadIdx.x / 32;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kListBufs; ++i) {
      mbar_init(&bars->list_full[i], 1);
      mbar_init(&bars->list_free[i], 3 + 2 * kTileM);  // load, 2 MMA, score
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->q_empty[i], 1);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i], kTileM);
      mbar_init(&bars->pv_done[i], 1);
      mbar_init(&bars->o_free[i], kTileM);
      for (int q = 0; q < 4; ++q) mbar_init(&bars->sm_turn[i][q], 1);
    }
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&bars->kv_full[i], 1);
      mbar_init(&bars->kv_empty[i], 2);  // both MMA issuers
    }
    mbar_init(&bars->mma_done[0], 1);
    mbar_init(&bars->mma_done[1], 1);
    bars->abort = 0;
    for (int i = 0; i < 6; ++i) bars->trace_n[i] = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp < 4) {
    setmaxnreg_dec<kRegsLight>();
    if (warp == 0)
      load_role<D>(p, &tm_q, &tm_k, &tm_v, smem, bars, lists);
    else if (warp == 3)
      list_role(p, bars, lists);
    else
      mma_role<D, SCORE>(p, smem, bars, lists, tmem, warp - 1);
  } else {
    setmaxnreg_inc<kRegsScore>();
    // one path per launch: per-element keep bits only when segment ids are
    // unsorted or an arbitrary mask is given (read once; the same for every
    // thread).  The alternating-turn instance is never launched for either.
    if (!PINGPONG && (((p.flags & BSM_MASK_SEGMENT) && (*p.seg_flags & 1) != 0) ||
                      p.dense != nullptr))
      score_role<D, SCORE, MOD, !PINGPONG, PINGPONG>(p, bars, lists, tmem);
    else
      score_role<D, SCORE, MOD, false, PINGPONG>(p, bars, lists, tmem);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
  if (p.trace != nullptr && threadIdx.x == 0) {
    uint32_t* hdr = reinterpret_cast<uint32_t*>(
        reinterpret_cast<TraceRec*>(p.trace) +
        static_cast<size_t>(blockIdx.x) * (p.trace_cap + 2));
    const uint32_t per = p.trace_cap / 6;
    for (int i = 0; i < 8; ++i) hdr[i] = i < 6 ? min(bars->trace_n[i], per) : 0;
  }
}

// ---------------------------------------------------------------------------
// Decoupled query tiles, made for packed sequences (segment ids).  There the
// units are short and the two query tiles of a unit often need different KV
// tiles, so the lockstep pipeline above spends much of its time at unit
// boundaries and on entries one tile skips.  Here the two 128-row query
// tiles of an SM are two independent pipelines: each takes its own work
// units (one query tile of one (batch, head)), builds its own KV-tile list,
// and has its own Q buffer and two-slot K/V ring, so one pipeline's unit
// boundary overlaps the other's work on the tensor core.  K/V tiles are not
// shared between the tiles (L2 carries the reuse).  Masks without segment
// ids take this kernel too below 4096 keys, where units are short as well,
// and modified scores at any length (see launch_score).
//
// Warp roles (384 threads, three warpgroups, registers split as above):
// warps 0/1 take pipeline 0/1's units, build their lists and load their
// tiles; warps 2/3 issue its MMAs (warp 2 also owns the TMEM); warps 4-7
// and 8-11 are the score warpgroups of pipeline 0 and 1.  With a cap each
// pipeline has two score warpgroups in most cases (640 threads without a
// register split; see dt_score_cap_role).  TMEM as above: S_t/P_t at [128 t, +128),
// O_t at [256 + 128 t, +D).  Head dim 128, softmax or pointwise; head dim 64
// with modified scores only.
constexpr int kDtThreads = 384;
constexpr int kDtTile = kTileM * 128 * 2;  // one 128 x 128 bf16 tile
constexpr int kDtOffQ = 0;                 // Q of pipeline t at t tiles
constexpr int kDtOffKV = 2 * kDtTile;      // ring slot s of pipeline t
constexpr int kDtOffBar = kDtOffKV + 4 * kDtTile;
constexpr int kDtSmemBytes = kDtOffBar + 1024 + 1024;
static_assert(kDtSmemBytes <= 232448, "shared memory budget");

struct DtMeta {
  int n;     // entries (KV tiles) of the unit
  int unit;  // -1: no unit left
  int b, h;  // batch row and head
  int qt;    // 128-row query tile
};

struct DtBars {
  uint64_t list_full[2][kListBufs], list_free[2][kListBufs];
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[2][2], kv_empty[2][2];  // [pipeline][slot]: K, V
  uint64_t s_full[2], p_full[2], pv_done[2], o_free[2], mma_done[2];
  // two threads per row: the two score warps of a pipeline and lane quarter,
  // on every entry and at a unit's end
  uint64_t meet[2][4], meet_sum[2][4];
  uint64_t merge;  // pipelines sharing a tile: pipeline 1's part is there
  uint32_t tmem_base;
  int abort;
  uint32_t trace_n[6];
  DtMeta meta[2][kListBufs];
};
static_assert(sizeof(DtBars) <= 1024, "barrier block");

// Two threads per row: their sums by pipeline and half.  A unit's sums
// alternate between two places: a thread writes the next unit's while its
// partner may still read this one's, but the one after that only once the
// partner has arrived with the next.
// Pipelines sharing a tile: pipeline 1's reference and sum of each row.
struct DtPair {
  float sum[2][2][2][kTileM];
  float ref[kTileM], total[kTileM];
};
// Pipelines sharing a tile: pipeline 1 leaves its O, [D][128] f32, in its own
// K and V slots, which nothing reads or writes any more.
constexpr int kDtOffMerge = kDtOffKV + 2 * kDtTile;
static_assert(kTileM * 128 * 4 <= 2 * kDtTile, "merge area");
constexpr int kDtOffPair = kDtOffBar + 1024;
static_assert(kDtSmemBytes + sizeof(DtPair) <= 232448, "shared memory budget");

// A distance bias alone (kModBias) is added by the tensor core: the bias of a
// tile's columns on one side of the row, in units of S, is +-slope / scale *
// (c - 64) for column c plus a term per row, so S gets one more step of 16 with
// A = [1 1 1 0 ..] (negated right of the row) in every row and B row c = the
// three bf16 parts of slope / scale * (c - 64), whose sum is the f32 value.
// What is left of the bias is one number per row and tile, which goes into the
// softmax's reference.  (With the bias added by the score warps, one paired
// addition per two scores more, causal S=8192, 32/8 heads took 527 us; so 466,
// key tiles in rising order both times; see dt_order_list.)  One 128 x 64 tile
// (128-byte swizzle) holds it all: columns [0, 16) and [16, 32) B of the
// pipelines, [32, 48) and [48, 64) A and -A.
constexpr int kDtOffBias = kDtOffPair + sizeof(DtPair);
constexpr int kDtBiasBytes = kTileM * 128;
static_assert(kDtOffBias % 1024 == 0, "swizzle atom");
static_assert(kDtOffBias + kDtBiasBytes + 1024 <= 232448,
              "shared memory budget");
constexpr int kBiasMid = kTileN / 2;

// 16-byte piece `piece` of row `row` of that tile.
__device__ __forceinline__ uint4* bias_piece(uint8_t* smem, int row, int piece) {
  return reinterpret_cast<uint4*>(smem + kDtOffBias + row * 128 +
                                  ((piece ^ (row & 7)) << 4));
}

// B of pipeline t for a head (whole warp).
__device__ __forceinline__ void write_bias(uint8_t* smem, int t, float ratio) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int i = 0; i < kTileN / 32; ++i) {
    const int c = i * 32 + lane;
    const float v = ratio * static_cast<float>(c - kBiasMid);
    const uint32_t h = pack_bf16x2(v, 0.f);  // the lower half
    const float v1 = v - __uint_as_float(h << 16);
    const uint32_t m = pack_bf16x2(v1, 0.f);
    const float v2 = v1 - __uint_as_float(m << 16);
    *bias_piece(smem, c, 2 * t) =
        make_uint4(h | m << 16, pack_bf16x2(v2, 0.f), 0u, 0u);
  }
  fence_proxy_async();
  __syncwarp();
}

// Score threads of one pipeline, and threads of the kernel.
// (kModFixed: cap and bias with a fixed reference, see dt_score_cap_role.)
constexpr int kModFixed = kModCap | kModBias | 4;
constexpr bool dt_two_per_row(int mod) {
  return mod == kModCap || mod == kModFixed;
}
constexpr int dt_score_threads(int mod) {
  return dt_two_per_row(mod) ? 256 : 128;
}
constexpr int dt_threads(int mod) { return 128 + 2 * dt_score_threads(mod); }

// Optional event trace, in the layout of `trace` above; the six recording
// threads are: loader 0, MMA 0, score 0, score 1, loader 1, MMA 1.
template <bool TRACE>
__device__ __forceinline__ void dt_trace(const FwdParams& p, DtBars* bars,
                                         uint32_t role, uint32_t ev,
                                         uint32_t tile, uint32_t entry,
                                         uint32_t unit) {
  if (!TRACE) return;
  const uint32_t slot = role == kRoleScore ? 2 + tile
                        : role == kRoleMma   ? (tile == 0 ? 1 : 5)
                                             : (tile == 0 ? 0 : 4);
  const uint32_t per = p.trace_cap / 6;
  const uint32_t i = bars->trace_n[slot]++;
  if (i < per) {
    TraceRec* r = reinterpret_cast<TraceRec*>(p.trace) +
                  static_cast<size_t>(blockIdx.x) * (p.trace_cap + 2) + 2 +
                  slot * per + i;
    r->t = globaltimer_ns();
    r->a = (role << 28) | (ev << 24) | (tile << 20) | (entry & 0xFFFFFu);
    r->b = unit;
  }
}

// SHARED (modified scores, at most half as many query tiles as SMs): the two
// pipelines of a CTA share its tile, each takes every other KV tile and
// pipeline 0 joins the two results.  (us, one tile per pipeline, one per CTA
// with an idle pipeline, and shared: S=1280, 12/4 heads, no mask, cap 50: 35.7,
// 26.4, 24.7; causal S=2048, 4/2 heads, D=64, cap 50: 43.8, 32.3, 26.8.)

// The order of a unit's KV tiles under a bias that falls with the distance: the
// query tile's own, those left of it from near to far, those right of it from
// near to far.  The first then sets the softmax's reference for good; in
// rising order a steep head's moves, and O is rescaled, on every entry (us,
// rising order and this one: causal S=8192, 32/8 heads: 466 and 425, with a cap
// and a running maximum 630 and 560).  Whole warp.
template <int MOD>
__device__ __forceinline__ void dt_order_list(const FwdParams& p,
                                              uint16_t* list, int n, int qt,
                                              int head) {
  if (p.mod.slopes == nullptr || !(p.mod.slopes[head] > 0.f)) return;
  const int lane = threadIdx.x % 32;
  int m = 0;  // entries up to the query tile's own
  if (p.flags & BSM_MASK_CAUSAL) {
    m = n;
  } else {
    for (int i = 0; i < n; i += 32)
      m += __popc(__ballot_sync(0xffffffffu, i + lane < n &&
                                                 (list[i + lane] >> 2) <= qt));
  }
  for (int i = lane; 2 * i < m - 1; i += 32) {
    const uint16_t a = list[i];
    list[i] = list[m - 1 - i];
    list[m - 1 - i] = a;
  }
  __syncwarp();
}

// Takes pipeline t's next unit from the counter and writes its KV-tile
// list (uint16: tile << 2 | class) into buffer ui % kListBufs (whole warp);
// unit -1 when none is left.  Units are numbered two per 256-row unit of
// the lockstep kernel's order (its two query tiles), longest first.
template <int MOD, bool TRACE, bool SHARED>
__device__ __forceinline__ bool dt_build_list(const FwdParams& p, DtBars* bars,
                                              uint16_t* lists, const int t,
                                              const int ui) {
  const int lane = threadIdx.x % 32;
  volatile int* abort_flag = &bars->abort;
  const int n_units = 2 * p.num_units;
  {
    const int buf = ui % kListBufs;
    if (!warp_wait(&bars->list_free[t][buf], ((ui / kListBufs) & 1) ^ 1,
                   abort_flag, p.timeout_ns)) {
      if (lane == 0) record_timeout(kRoleList, 0);
      return false;
    }
    int unit = 0;
    if (p.unit_counter == nullptr) {  // nothing to count
      unit = ui > 0 ? n_units
             : SHARED ? static_cast<int>(blockIdx.x)
                      : static_cast<int>(blockIdx.x) * 2 + t;
    } else {
      if (lane == 0) unit = atomicAdd(p.unit_counter, 1);
      unit = __shfl_sync(0xffffffffu, unit, 0);
    }
    DtMeta& mt = bars->meta[t][buf];
    if (unit >= n_units) {
      if (lane == 0) {
        mt.unit = -1;
        mt.n = 0;
        mbar_arrive(&bars->list_full[t][buf]);
      }
      __syncwarp();
      return true;
    }
    const UnitCoord uc = decode_unit(p, unit >> 1);
    const int qt = uc.st * 2 + (unit & 1);
    const int table = (p.flags & BSM_MASK_SEGMENT) ? uc.b : 0;
    uint16_t* list = lists + buf * kMaxKvTiles;
    int n = 0;
    for (int base = 0; base < p.n_kvtiles; base += 64) {
      int c[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int jt = base + 32 * h + lane;
        c[h] = jt < p.n_kvtiles ? tile_class(p, table, qt * kTileM, jt) : 0;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int jt = base + 32 * h + lane;
        const unsigned m = __ballot_sync(0xffffffffu, c[h] != 0);
        const int at = n + __popc(m & ((1u << lane) - 1u));
        if (c[h] && (!SHARED || (at & 1) == t))
          list[SHARED ? at >> 1 : at] =
              static_cast<uint16_t>((jt << 2) | c[h]);
        n += __popc(m);
      }
    }
    if (SHARED) n = (n + 1 - t) >> 1;  // every other entry
    __syncwarp();
    if (MOD & kModBias) dt_order_list<MOD>(p, list, n, qt, uc.h);
    if (lane == 0) {
      mt.n = n;
      mt.unit = unit;
      mt.b = uc.b;
      mt.h = uc.h;
      mt.qt = qt;
      dt_trace<TRACE>(p, bars, kRoleList, kEvListBuilt, t, n, unit);
      mbar_arrive(&bars->list_full[t][buf]);
    }
    __syncwarp();
  }
  return true;
}

// Pipeline t's loader: builds the next unit's list, then loads its Q and
// the K and V of every entry through the pipeline's two slots (K in slot
// 0, V in slot 1).  The next list is built once this unit's last loads are
// issued, i.e. while the unit's last entries still run (building it after
// the first entry's loads measured slower).
template <int D, int MOD, bool TRACE, bool SHARED>
__device__ __forceinline__ void dt_load_role(const FwdParams& p,
                                             const CUtensorMap* tq,
                                             const CUtensorMap* tk,
                                             const CUtensorMap* tv,
                                             uint8_t* smem, DtBars* bars,
                                             uint16_t* lists, const int t) {
  const int lane = threadIdx.x % 32;
  volatile int* abort_flag = &bars->abort;
  const uint64_t pol_q = l2_policy_evict_first();
  const uint64_t pol_kv = l2_policy_evict_last();
  uint32_t kv_it = 0, q_it = 0;
  bool ok = true;
  for (int ui = 0; ok; ++ui) {
    const int buf = ui % kListBufs;
    ok = dt_build_list<MOD, TRACE, SHARED>(p, bars, lists, t, ui);
    if (!ok) break;
    const DtMeta mt = bars->meta[t][buf];
    if (mt.unit < 0) break;
    const uint16_t* list = lists + buf * kMaxKvTiles;
    if (mt.n > 0) {
      ok = warp_wait(&bars->q_empty[t], (q_it & 1) ^ 1, abort_flag,
                     p.timeout_ns);
      if (!ok) {
        if (lane == 0) record_timeout(kRoleLoad, 1);
        break;
      }
      if (MOD == kModBias)  // (the last unit's S, which read it, is complete)
        write_bias(smem, t, p.mod.slopes[mt.h] / p.scale);
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars->q_full[t], kTileM * D * 2);
        for (int kb = 0; kb < D / 64; ++kb)
          tma_load_4d(tq, &bars->q_full[t],
                      smem + kDtOffQ + t * kDtTile + kb * kTileM * 128,
                      kb * 64, mt.qt * kTileM, mt.h, mt.b, pol_q);
        dt_trace<TRACE>(p, bars, kRoleLoad, kEvQIssued, t, 0, mt.unit);
      }
      ++q_it;
    }
    const int hkv = mt.h / (p.H / p.Hkv);
    for (int e = 0; ok && e < mt.n; ++e) {
      const int jt = static_cast<int>(list[e] >> 2);
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        if (!ok) break;
        const uint32_t ph = (kv_it >> 1) & 1;
        ok = warp_wait(&bars->kv_empty[t][which], ph ^ 1, abort_flag,
                       p.timeout_ns);
        if (!ok) {
          if (lane == 0) record_timeout(kRoleLoad, 2);
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars->kv_full[t][which], kTileN * D * 2);
          uint8_t* dst = smem + kDtOffKV + (2 * t + which) * kDtTile;
          for (int kb = 0; kb < D / 64; ++kb)
            tma_load_4d(which == 0 ? tk : tv, &bars->kv_full[t][which],
                        dst + kb * kTileN * 128, kb * 64, jt * kTileN, hkv,
                        mt.b, pol_kv);
          dt_trace<TRACE>(p, bars, kRoleLoad, kEvTmaIssued, t, e * 2 + which, mt.unit);
        }
        ++kv_it;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->list_free[t][buf]);
  }
  // Drain the loads already issued (each slot received kv_it / 2 loads).
  if (lane == 0) {
    for (int s = 0; s < 2; ++s) {
      const uint32_t n = (kv_it + 1 - s) >> 1;  // loads slot s received
      if (n > 0 && !mbar_wait_drain(&bars->kv_full[t][s], (n - 1) & 1,
                                    p.timeout_ns) && ok)
        record_timeout(kRoleLoad, 3);
    }
    if (q_it > 0 && !mbar_wait_drain(&bars->q_full[t], (q_it - 1) & 1,
                                     p.timeout_ns) && ok)
      record_timeout(kRoleLoad, 4);
  }
  __syncwarp();
}

// Pipeline t's MMA warp: S(e) = Q K(e)^T, then O += P(e) V(e) and S(e + 1)
// right behind it (tcgen05 MMAs of one thread run in issue order, so
// S(e + 1) overwrites the columns P(e) V read only after that product).
// The K slot is released once the S that read it completed, the V slot
// once the P.V did.  The whole warp runs the issuing code and each MMA and
// commit goes out from the lane elect.sync picks (the same lane every
// time: the warp is converged there); issued that way the pipeline's MMAs
// measured ~5 % faster than from a branch lane 0 takes alone.
template <int D, int SCORE, int MOD, bool TRACE>
__device__ __forceinline__ void dt_mma_role(const FwdParams& p, uint8_t* smem,
                                            DtBars* bars,
                                            const uint16_t* lists,
                                            uint32_t tmem, const int t) {
  const bool leader = (threadIdx.x % 32) == 0;
  volatile int* abort_flag = &bars->abort;
  constexpr uint32_t idesc_s = idesc_bf16_f32(kTileM, kTileN, false);
  constexpr uint32_t idesc_o = idesc_bf16_f32(kTileM, D, true);
  const uint64_t dq =
      sdesc_sw128(smem_u32(smem + kDtOffQ + t * kDtTile), 16, 1024);
  const uint64_t dk =
      sdesc_sw128(smem_u32(smem + kDtOffKV + (2 * t) * kDtTile), 16, 1024);
  const uint64_t dv = sdesc_sw128(
      smem_u32(smem + kDtOffKV + (2 * t + 1) * kDtTile), kTileN * 128, 1024);
  const uint32_t s_acc = tmem + t * 128;
  const uint32_t o_acc = tmem + 256 + t * 128;
  uint32_t k_it = 0, v_it = 0, q_it = 0, s_cnt = 0;
  bool ok = true;
  auto fail = [&](int where) {
    if (leader) record_timeout(kRoleMma, where);
  };
  const uint64_t dbias = sdesc_sw128(smem_u32(smem + kDtOffBias), 16, 1024);
  auto issue_s = [&](bool right) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint32_t off = (k >> 2) * (kTileM * 128 / 16) + (k & 3) * 2;
      mma_ss_elect(s_acc, dq + off, dk + off, idesc_s, k > 0 ? 1u : 0u);
    }
    if (MOD == kModBias)
      mma_ss_elect(s_acc, dbias + (right ? 6 : 4), dbias + 2 * t, idesc_s, 1u);
    mma_commit_elect(&bars->s_full[t]);
  };
  for (int ui = 0; ok; ++ui) {
    const int buf = ui % kListBufs;
    ok = warp_wait(&bars->list_full[t][buf], (ui / kListBufs) & 1, abort_flag,
                   p.timeout_ns);
    if (!ok) {
      fail(0);
      break;
    }
    const DtMeta mt = bars->meta[t][buf];
    if (mt.unit < 0) break;
    const uint16_t* list = lists + buf * kMaxKvTiles;
    // whether entry e's keys lie right of the query tile
    auto right = [&](int e) {
      return MOD == kModBias && static_cast<int>(list[e] >> 2) > mt.qt;
    };
    const int n = mt.n;
    if (n > 0) {
      ok = warp_wait(&bars->q_full[t], q_it & 1, abort_flag, p.timeout_ns) &&
           warp_wait(&bars->kv_full[t][0], k_it & 1, abort_flag, p.timeout_ns);
      if (!ok) {
        fail(1);
        break;
      }
      ++q_it;
      ++k_it;
      tc_fence_after();
      issue_s(right(0));
      if (leader) dt_trace<TRACE>(p, bars, kRoleMma, kEvSIssued, t, 0, mt.unit);
      if (n == 1) mma_commit_elect(&bars->q_empty[t]);
      mma_commit_elect(&bars->kv_empty[t][0]);
      ++s_cnt;
    }
    for (int e = 0; ok && e < n; ++e) {
      ok = warp_wait(&bars->kv_full[t][1], v_it & 1, abort_flag,
                     p.timeout_ns) &&
           warp_wait(&bars->p_full[t], (s_cnt - 1) & 1, abort_flag,
                     p.timeout_ns);
      if (ok && e == 0)
        ok = warp_wait(&bars->o_free[t], (ui & 1) ^ 1, abort_flag,
                       p.timeout_ns);
      if (!ok) {
        fail(5);
        break;
      }
      ++v_it;
      if (leader) dt_trace<TRACE>(p, bars, kRoleMma, kEvPReady, t, e, mt.unit);
      tc_fence_after();
      if (SCORE == BSM_SCORE_SOFTMAX) {
#pragma unroll
        for (int kk = 0; kk < kTileN / 16; ++kk)
          mma_ts_elect(o_acc, s_acc + kk * 8, dv + kk * (16 * 128 / 16),
                       idesc_o, (kk > 0 || e > 0) ? 1u : 0u);
      } else {
#pragma unroll 2
        for (int kk = 0; kk < kTileN / 16; ++kk) {
          const uint32_t col = (kk >> 2) * 64 + (kk & 3) * 8;
          mma_ts_elect(o_acc, s_acc + col, dv + kk * (16 * 128 / 16), idesc_o,
                       (kk > 0 || e > 0) ? 1u : 0u);
          mma_ts_elect(o_acc, s_acc + col + 32, dv + kk * (16 * 128 / 16),
                       idesc_o, 1u);
        }
      }
      mma_commit_elect(&bars->pv_done[t]);
      mma_commit_elect(&bars->kv_empty[t][1]);
      if (leader)
        dt_trace<TRACE>(p, bars, kRoleMma, kEvPVIssued, t, e, mt.unit);
      if (e + 1 < n) {
        ok = warp_wait(&bars->kv_full[t][0], k_it & 1, abort_flag,
                       p.timeout_ns);
        if (!ok) {
          fail(2);
          break;
        }
        ++k_it;
        tc_fence_after();
        issue_s(right(e + 1));
        if (leader)
          dt_trace<TRACE>(p, bars, kRoleMma, kEvSIssued, t, e + 1, mt.unit);
        if (e + 1 == n - 1) mma_commit_elect(&bars->q_empty[t]);
        mma_commit_elect(&bars->kv_empty[t][0]);
        ++s_cnt;
      }
    }
    if (!ok) break;
    if (leader) mbar_arrive(&bars->list_free[t][buf]);
    __syncwarp();
  }
  __syncwarp();
  mma_commit_elect(&bars->mma_done[t]);
  if (leader && !mbar_wait_drain(&bars->mma_done[t], 0, p.timeout_ns) && ok)
    record_timeout(kRoleMma, 6);
  __syncwarp();
}

template <int D, int SCORE, int MOD, bool KEEP, bool TRACE, bool SHARED>
__device__ __forceinline__ void dt_score_role(const FwdParams& p, DtBars* bars,
                                              DtPair* pair, float* merge,
                                              const uint16_t* lists,
                                              uint32_t tmem, const int t) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int quarter = warp % 4;  // TMEM lane quarter this warp may access
  const int r = quarter * 32 + lane;
  const bool tracer = (r == 0);
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t s_addr = tmem + lane_off + t * 128;
  const uint32_t o_addr = tmem + lane_off + 256 + t * 128;
  volatile int* abort_flag = &bars->abort;
  const float NEG_INF = __int_as_float(0xff800000);
  const bool seg = (p.flags & BSM_MASK_SEGMENT) != 0;
  const bool seg_elem = KEEP && seg && (*p.seg_flags & 1) != 0;
  const bool dense = KEEP && p.dense != nullptr;
  uint32_t s_cnt = 0, pv_cnt = 0;
  for (int ui = 0;; ++ui) {
    const int buf = ui % kListBufs;
    if (!warp_wait(&bars->list_full[t][buf], (ui / kListBufs) & 1, abort_flag,
                   p.timeout_ns)) {
      record_timeout(kRoleScore, 0);
      break;
    }
    const int unit = bars->meta[t][buf].unit;
    if (unit < 0) break;
    const int n_ent = bars->meta[t][buf].n;
    const UnitCoord uc{bars->meta[t][buf].b, bars->meta[t][buf].h, 0};
    const uint16_t* list = lists + buf * kMaxKvTiles;
    const int qt = bars->meta[t][buf].qt;
    const int qrow = qt * kTileM + r;
    const bool row_ok = qrow < p.Sq;
    // visible keys of this row form [rlo, rhi] (plus the element compare of
    // unsorted segment ids)
    int rlo = 0, rhi = p.Skv - 1;
    if (p.flags & BSM_MASK_CAUSAL) rhi = min(rhi, qrow);
    if (p.flags & BSM_MASK_LOCAL) rlo = max(rlo, qrow - p.window + 1);
    if (p.flags & BSM_MASK_BAND) rhi = min(rhi, qrow + p.window - 1);
    int segq = 0;
    if (seg && row_ok) {
      const int64_t qi = static_cast<int64_t>(uc.b) * p.Sq + qrow;
      if (seg_elem) {
        segq = p.q_seg[qi];
      } else {
        const int2 sr = reinterpret_cast<const int2*>(p.seg_range)[qi];
        rlo = max(rlo, sr.x);
        rhi = min(rhi, sr.y);
      }
    }
    const int32_t* segk_b =
        seg_elem ? p.kv_seg + static_cast<int64_t>(uc.b) * p.Skv : nullptr;
    float m_used = NEG_INF, l_sum = 0.f;
    const float slope2 = (MOD & kModBias) && p.mod.slopes != nullptr
                             ? p.mod.slopes[uc.h] * 1.4426950408889634f
                             : 0.f;
    uint32_t unit_pv = 0;
    bool ok = true;
    for (int e = 0; e < n_ent; ++e) {
      const uint32_t ent = list[e];
      const int cls = static_cast<int>(ent & 3u);
      if (!cls) continue;
      const int jt = static_cast<int>(ent >> 2);
      const int kbase = jt * kTileN;
      uint32_t keep[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
      if (KEEP && cls == 1) {
        if (seg_elem)
          segment_bits(keep, segk_b + kbase, min(kTileN, p.Skv - kbase), segq);
        if (dense) {  // the row's mask words for these 128 keys
          const int64_t w0 = kbase >> 5;
          const uint32_t* dw =
              p.dense + static_cast<int64_t>(row_ok ? qrow : 0) * p.dense_words;
#pragma unroll
          for (int w = 0; w < 4; ++w)
            keep[w] &= (row_ok && w0 + w < p.dense_words) ? __ldg(dw + w0 + w)
                                                          : 0u;
        }
      }
      ok = warp_wait(&bars->s_full[t], s_cnt & 1, abort_flag, p.timeout_ns);
      if (!ok) {
        record_timeout(kRoleScore, 1);
        break;
      }
      ++s_cnt;
      if (tracer) dt_trace<TRACE>(p, bars, kRoleScore, kEvSFull, t, e, unit);
      tc_fence_after();
      if (MOD == kModBias && jt == qt && !(p.flags & BSM_MASK_CAUSAL)) {
        // Keys on both sides of the row: S has the left side's bias, which is
        // taken twice off the keys on the right.  In TMEM, 32 columns at a
        // time: code for it over all of the row's registers cost every tile 8 %.
        const float twice = -2.f * (slope2 / p.scale_log2);
#pragma unroll 1
        for (int q = 0; q < kTileN / 32; ++q) {
          uint32_t x[32];
          tmem_ld32(s_addr + q * 32, x);
          tmem_ld_wait();
          const int d0 = kbase + q * 32 - qrow;
#pragma unroll
          for (int c = 0; c < 32; ++c)
            x[c] = __float_as_uint(fmaf(twice,
                                        static_cast<float>(max(d0 + c, 0)),
                                        __uint_as_float(x[c])));
          tmem_st32(s_addr + q * 32, x);
        }
        tmem_st_wait();
      }
      uint32_t sraw[kTileN];
#pragma unroll
      for (int q = 0; q < kTileN / 32; ++q)
        tmem_ld32(s_addr + q * 32, sraw + q * 32);
      tmem_ld_wait();
      float* s = reinterpret_cast<float*>(sraw);
      float sl8 = 0.f, cbase = 0.f;  // bias of each 8 columns (cap and bias)
      float base = 0.f;              // of the row (bias alone)
      if (MOD == kModBias) {
        // S has the tile's part already
        base = (jt > qt ? -slope2 : slope2) *
               static_cast<float>(kbase + kBiasMid - qrow);
      } else if (MOD != 0) {
        modify_tile<MOD, kTileN>(s, p, kbase, qrow, cls == 1, rlo - kbase,
                                 rhi - kbase, keep, KEEP, slope2, &sl8, &cbase);
      }
      if (cls == 1) mask_tile(s, rlo - kbase, rhi - kbase, keep, KEEP);

      uint32_t pk[16];
      if (SCORE == BSM_SCORE_SOFTMAX) {
        float m_blk;
        if (MOD == 0 || MOD == kModBias) {
          // row max: three-input max, four independent chains
          float mx0 = fmaxf(s[0], s[1]), mx1 = fmaxf(s[2], s[3]);
          float mx2 = fmaxf(s[4], s[5]), mx3 = fmaxf(s[6], s[7]);
#pragma unroll
          for (int c = 8; c < kTileN; c += 8) {
            mx0 = fmax3(mx0, s[c], s[c + 1]);
            mx1 = fmax3(mx1, s[c + 2], s[c + 3]);
            mx2 = fmax3(mx2, s[c + 4], s[c + 5]);
            mx3 = fmax3(mx3, s[c + 6], s[c + 7]);
          }
          const float mx = fmax3(mx0, mx1, fmaxf(mx2, mx3));
          m_blk = MOD == 0 ? mx * p.scale_log2 : fmaf(mx, p.scale_log2, base);
        } else {
          m_blk = biased_max<kTileN>(s, sl8, cbase);
        }
        bool rescale = false;
        float alpha = 1.f;
        if (m_blk > m_used + kRescaleLog2) {
          if (m_used != NEG_INF) {
            alpha = ex2_approx(m_used - m_blk);
            rescale = true;
          }
          l_sum *= alpha;
          m_used = m_blk;
        }
        float neg_m = (m_used == NEG_INF) ? 0.f : -m_used;
        if (MOD == kModBias) neg_m += base;
        float ls0 = 0.f, ls1 = 0.f, ls2 = 0.f, ls3 = 0.f;
#pragma unroll
        for (int q = 0; q < kTileN / 32; ++q) {  // 32 columns at a time
#pragma unroll
          for (int c = 32 * q; c < 32 * q + 32; c += 4) {
            // paired f32 FMA/add: the same roundings as one element at a time
            float x0, x1, x2, x3;
            if (MOD == 0 || MOD == kModBias) {
              ffma2(x0, x1, s[c], s[c + 1], p.scale_log2, neg_m);
              ffma2(x2, x3, s[c + 2], s[c + 3], p.scale_log2, neg_m);
            } else {
              const float add =
                  fmaf(sl8, static_cast<float>(c / 8), cbase + neg_m);
              fadd2(x0, x1, s[c], s[c + 1], add, add);
              fadd2(x2, x3, s[c + 2], s[c + 3], add, add);
            }
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            const float p2 = ex2_approx(x2), p3 = ex2_approx(x3);
            fadd2(ls0, ls1, ls0, ls1, p0, p1);
            fadd2(ls2, ls3, ls2, ls3, p2, p3);
            pk[(c & 31) / 2] = pack_bf16x2(p0, p1);
            pk[(c & 31) / 2 + 1] = pack_bf16x2(p2, p3);
          }
          tmem_st16(s_addr + q * 16, pk);
        }
        l_sum += (ls0 + ls1) + (ls2 + ls3);
        // Rescale O_t (needs the previous PV of this tile to have landed).
        if (__any_sync(0xffffffffu, rescale) && unit_pv > 0) {
          ok = warp_wait(&bars->pv_done[t], (pv_cnt - 1) & 1, abort_flag,
                         p.timeout_ns);
          if (!ok) {
            record_timeout(kRoleScore, 2);
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(o_addr + q * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 32; ++c)
              o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
            tmem_st32(o_addr + q * 32, o);
          }
        }
      } else {
        // pointwise: x = scale*qk; p = x*sigmoid(x)/Sq; masked (-inf) -> 0.
        // With sigmoid(x) = (1 + tanh(x/2)) / 2 this is g + g*tanh(x/2),
        // g = x / (2 Sq): one tanh per element, the rest on paired f32.
        // hstu_ops multiplies the f32 scores by f32 v, so p is kept to about
        // 16 bits: p = hi + lo, both bf16 (lo = p - hi is exact in f32).
        // Each 64-key half's hi and lo (32 columns each) go back over that
        // half's own 64 columns of S; the MMA warp adds both products into O.
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t pl[16];
#pragma unroll
            for (int c = 64 * hf + 32 * q; c < 64 * hf + 32 * q + 32; c += 2) {
              float h0, h1, g0, g1, p0, p1;
              fmul2(h0, h1, s[c], s[c + 1], p.pw_half);
              fmul2(g0, g1, s[c], s[c + 1], p.pw_g);
              ffma2v(p0, p1, g0, g1, tanh_approx(h0), tanh_approx(h1), g0,
                     g1);
              p0 = s[c] != NEG_INF ? p0 : 0.f;
              p1 = s[c + 1] != NEG_INF ? p1 : 0.f;
              const uint32_t hi = pack_bf16x2(p0, p1);
              pk[(c & 31) / 2] = hi;
              pl[(c & 31) / 2] =
                  pack_bf16x2(p0 - __uint_as_float(hi << 16),
                              p1 - __uint_as_float(hi & 0xffff0000u));
            }
            tmem_st16(s_addr + hf * 64 + q * 16, pk);
            tmem_st16(s_addr + hf * 64 + 32 + q * 16, pl);
          }
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bars->p_full[t]);
      if (tracer) dt_trace<TRACE>(p, bars, kRoleScore, kEvPFull, t, e, unit);
      ++pv_cnt;
      ++unit_pv;
    }
    if (!ok) break;

    // ---- epilogue: out = O / l (softmax) or O (pointwise), bf16
    if (tracer) dt_trace<TRACE>(p, bars, kRoleScore, kEvEpiBegin, t, 0, unit);
    uint16_t* orow = p.out + static_cast<int64_t>(uc.b) * p.o_sb +
                     static_cast<int64_t>(uc.h) * p.o_sh +
                     static_cast<int64_t>(qrow) * p.o_ss;
    if (unit_pv > 0) {
      if (!warp_wait(&bars->pv_done[t], (pv_cnt - 1) & 1, abort_flag,
                     p.timeout_ns)) {
        record_timeout(kRoleScore, 3);
        break;
      }
      tc_fence_after();
      // all of O_t into registers with one wait; the next unit's first P.V
      // may then overwrite it while the stores go out
      uint32_t o[D];
#pragma unroll
      for (int q = 0; q < D / 32; ++q) tmem_ld32(o_addr + q * 32, o + q * 32);
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(&bars->o_free[t]);
      if (SHARED) {
        if (t == 1) {  // O, reference and sum for pipeline 0
#pragma unroll
          for (int c = 0; c < D; ++c)
            merge[c * kTileM + r] = __uint_as_float(o[c]);
          pair->ref[r] = m_used;
          pair->total[r] = l_sum;
          mbar_arrive(&bars->merge);
          mbar_arrive(&bars->list_free[t][buf]);
          continue;
        }
        if (!warp_wait(&bars->merge, 0, abort_flag, p.timeout_ns)) {
          record_timeout(kRoleScore, 8);
          break;
        }
        const float l1 = pair->total[r], m1 = pair->ref[r];
        const float mm = fmaxf(m_used, m1);
        const float w0 = m_used == NEG_INF ? 0.f : ex2_approx(m_used - mm);
        const float w1 = m1 == NEG_INF ? 0.f : ex2_approx(m1 - mm);
        if (!(l1 == 0.f)) {  // (0: it saw nothing, or had no entry)
#pragma unroll
          for (int c = 0; c < D; ++c)
            o[c] = __float_as_uint(fmaf(merge[c * kTileM + r], w1,
                                        __uint_as_float(o[c]) * w0));
          l_sum = fmaf(l1, w1, l_sum * w0);
          m_used = mm;
        }
      }
      float inv = 1.f;
      if (SCORE == BSM_SCORE_SOFTMAX) inv = has_sum<MOD>(l_sum) ? 1.f / l_sum : 0.f;
      if (row_ok) {
        // 32 bytes per store where the row alignment allows: each warp
        // store touches 32 rows, so fewer, wider stores cost fewer requests
        const bool v8 = p.o_vec8 != 0;
#pragma unroll
        for (int v = 0; v < D / 16; ++v) {
          uint32_t w[8];
#pragma unroll
          for (int c = 0; c < 8; ++c)
            w[c] = pack_bf16x2(__uint_as_float(o[16 * v + 2 * c]) * inv,
                               __uint_as_float(o[16 * v + 2 * c + 1]) * inv);
          if (v8) {
            st_global_v8(orow + v * 16, w);
          } else {
            st_global_v4(orow + v * 16, w[0], w[1], w[2], w[3]);
            st_global_v4(orow + v * 16 + 8, w[4], w[5], w[6], w[7]);
          }
        }
      }
    } else if (SHARED && t == 1) {
      pair->ref[r] = NEG_INF;
      pair->total[r] = 0.f;
      tc_fence_before();
      mbar_arrive(&bars->o_free[t]);
      mbar_arrive(&bars->merge);
      mbar_arrive(&bars->list_free[t][buf]);
      continue;
    } else {
      if (row_ok) {
#pragma unroll
        for (int v = 0; v < D / 8; ++v)
          st_global_v4(orow + v * 8, 0u, 0u, 0u, 0u);
      }
      tc_fence_before();
      mbar_arrive(&bars->o_free[t]);
    }
    if (SCORE == BSM_SCORE_SOFTMAX && p.lse != nullptr && row_ok) {
      const float lse = has_sum<MOD>(l_sum)
                            ? (m_used + log2f(l_sum)) * 0.6931471805599453f
                            : NEG_INF;
      p.lse[(static_cast<int64_t>(uc.b) * p.H + uc.h) * p.Sq + qrow] = lse;
    }
    mbar_arrive(&bars->list_free[t][buf]);
    if (tracer) dt_trace<TRACE>(p, bars, kRoleScore, kEvEpiEnd, t, 0, unit);
  }
}

// Distance from a row to the nearest (or farthest) key that it sees in a unit's
// KV tiles under unsorted segment ids, 0 if there is none.  All lanes of a warp.
// It compares the ids of a tile as the scores do, the best placed tiles first
// and only while a row of the warp may find a better key there.  (Forward at
// S=16384, 4 heads, D=64, no other mask, random ids of four: 856 us, a cap alone
// 815; where half of the rows have an id that no key has 1448, and 4136 with a
// walk from the row key by key.)
__device__ __forceinline__ int segment_distance(const FwdParams& p,
                                                const uint16_t* list, int n_ent,
                                                const int32_t* segk, int segq,
                                                int qrow, bool row_ok, int rlo,
                                                int rhi, bool nearest) {
  const int lane = threadIdx.x % 32;
  const int first = qrow - lane, last = first + 31;  // the warp's rows
  int d = -1;
  for (int e0 = 0; e0 < n_ent; e0 += 32) {
    const uint32_t ent = e0 + lane < n_ent ? list[e0 + lane] : 0u;
    const int tile = static_cast<int>(ent >> 2) * kTileN;
    // the best that this lane's tile has for a row of the warp
    const int may = nearest ? max(max(tile - last, first - (tile + kTileN - 1)), 0)
                            : max(last - tile, tile + kTileN - 1 - first);
    bool open = e0 + lane < n_ent;
    for (;;) {
      // the worst that a row of the warp has so far
      const int worst =
          nearest ? __reduce_max_sync(0xffffffffu,
                                      !row_ok ? -1 : d < 0 ? 1 << 30 : d)
                  : __reduce_min_sync(0xffffffffu, !row_ok ? 1 << 30 : d);
      open = open && (nearest ? may < worst : may > worst);
      if (!__any_sync(0xffffffffu, open)) break;
      const int pick =
          nearest ? __reduce_min_sync(0xffffffffu,
                                      open ? may * 32 + lane : INT_MAX)
                  : __reduce_max_sync(0xffffffffu, open ? may * 32 + lane : -1);
      if (pick % 32 == lane) open = false;
      const uint32_t x = __shfl_sync(0xffffffffu, ent, pick % 32);
      const int kbase = static_cast<int>(x >> 2) * kTileN;
      uint32_t keep[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
      if ((x & 3u) == 1u)
        segment_bits(keep, segk + kbase, min(p.Skv - kbase, kTileN), segq);
#pragma unroll
      for (int w = 0; w < kTileN / 32; ++w) {
        const int c0 = kbase + 32 * w;
        const int lb = min(max(rlo - c0, 0), 32);
        const int hb = min(max(rhi - c0 + 1, 0), 32);
        const uint32_t below_hi = hb >= 32 ? 0xffffffffu : (1u << hb) - 1u;
        const uint32_t below_lo = lb >= 32 ? 0xffffffffu : (1u << lb) - 1u;
        const uint32_t seen = keep[w] & below_hi & ~below_lo;
        // the keys up to the row, and those after it
        const int at = qrow - c0;
        const uint32_t upto =
            at < 0 ? 0u : at >= 31 ? 0xffffffffu : (2u << at) - 1u;
        const uint32_t l = seen & upto, r = seen & ~upto;
        if (l != 0) {
          const int x = at - (nearest ? 31 - __clz(l) : __ffs(l) - 1);
          d = d < 0 ? x : nearest ? min(d, x) : max(d, x);
        }
        if (r != 0) {
          const int x = (nearest ? __ffs(r) - 1 : 31 - __clz(r)) - at;
          d = d < 0 ? x : nearest ? min(d, x) : max(d, x);
        }
      }
    }
  }
  return max(d, 0);
}

// Score warps of pipeline t for softmax scores that a cap bounds (kModCap, and
// kModFixed with a bias too): eight instead of four, two threads per query row,
// each with one 64-key half of the tile.  The arithmetic per score is about
// twice the unmodified one's and the tensor core waits for it on every entry,
// so a row's latency is halved.  No running maximum is kept, so the threads of a
// row share only the maximum of the unit's first tile and, in the epilogue,
// their sums; and half 1, whose P goes over columns
// [32, 64) of S (half 0's scores), writes after half 0 has read.  Measured
// (us): packed S=8192, 2 x 16 heads: cap 50 148, cap 20 171, with a bias 153 and
// 178 (one thread per row and a running maximum: 172 and 211); causal S=8192,
// 32/8 heads: cap 50 504, with a bias 518 (560).  A constant reference would be
// 6 to 12 % faster with a cap alone, but see ref.  What bounds cap 20 is the
// MUFU pipe (2.5 operations per score: about 540 us at 16 a clock and SM).
template <int D, int MOD, bool KEEP, bool TRACE, bool SHARED>
__device__ __forceinline__ void dt_score_cap_role(const FwdParams& p,
                                                  DtBars* bars, DtPair* pair,
                                                  float* merge,
                                                  const uint16_t* lists,
                                                  uint32_t tmem, const int t,
                                                  const int hf) {
  constexpr int NC = kTileN / 2;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int quarter = warp % 4;  // TMEM lane quarter this warp may access
  const int r = quarter * 32 + lane;
  const bool tracer = r == 0 && hf == 0;
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t s_addr = tmem + lane_off + t * 128;
  const uint32_t o_addr = tmem + lane_off + 256 + t * 128 + hf * (D / 2);
  volatile int* abort_flag = &bars->abort;
  const float NEG_INF = __int_as_float(0xff800000);
  const bool seg = (p.flags & BSM_MASK_SEGMENT) != 0;
  const bool seg_elem = KEEP && seg;
  uint64_t* meet = &bars->meet[t][quarter];
  uint32_t s_cnt = 0, pv_cnt = 0, meets = 0, sums = 0;
  for (int ui = 0;; ++ui) {
    const int buf = ui % kListBufs;
    if (!warp_wait(&bars->list_full[t][buf], (ui / kListBufs) & 1, abort_flag,
                   p.timeout_ns)) {
      record_timeout(kRoleScore, 0);
      break;
    }
    const int unit = bars->meta[t][buf].unit;
    if (unit < 0) break;
    const int n_ent = bars->meta[t][buf].n;
    const UnitCoord uc{bars->meta[t][buf].b, bars->meta[t][buf].h, 0};
    const uint16_t* list = lists + buf * kMaxKvTiles;
    const int qrow = bars->meta[t][buf].qt * kTileM + r;
    const bool row_ok = qrow < p.Sq;
    // visible keys of this row form [rlo, rhi] (plus the element compare of
    // unsorted segment ids)
    int rlo = 0, rhi = p.Skv - 1;
    if (p.flags & BSM_MASK_CAUSAL) rhi = min(rhi, qrow);
    if (p.flags & BSM_MASK_LOCAL) rlo = max(rlo, qrow - p.window + 1);
    if (p.flags & BSM_MASK_BAND) rhi = min(rhi, qrow + p.window - 1);
    int segq = 0;
    if (seg && row_ok) {
      const int64_t qi = static_cast<int64_t>(uc.b) * p.Sq + qrow;
      if (seg_elem) {
        segq = p.q_seg[qi];
      } else {
        const int2 sr = reinterpret_cast<const int2*>(p.seg_range)[qi];
        rlo = max(rlo, sr.x);
        rhi = min(rhi, sr.y);
      }
    }
    const int32_t* segk_b =
        seg_elem ? p.kv_seg + static_cast<int64_t>(uc.b) * p.Skv : nullptr;
    // No running maximum: the cap bounds the logits to +-cap_log2, with a bias
    // around the row's largest bias, that of its nearest key (farthest, for a
    // negative slope).  The reference is the maximum of the unit's first tile
    // (with a bias the one next to the row), so that a key that outweighs all
    // others there has p = 1 as with a running maximum; with a constant its
    // rounding to bf16 reached the gradients (4.4e-3 in norm instead of 3.3e-3
    // on short rows).  A key that outweighs the others in a later tile has a
    // rounded p all the same (with a cap alone the first tile is the farthest,
    // and packed it may hold few of the row's keys: output 2.2e-3 in norm at
    // S=8192).  The reference is at most 90 below the upper bound, so p lies
    // below 2^90, where 2^18 of them stay inside f32, and the row's largest
    // above 2^-84 (cap_log2 <= 87; 75 with a bias): what is flushed to 0, below
    // 2^-126, weighs 2^-42 of it.
    float ref = p.mod.cap_log2 - 90.f, l_sum = 0.f;
    float slope2 = 0.f;
    if (MOD == kModFixed) {
      slope2 = p.mod.slopes[uc.h] * 1.4426950408889634f;
      const int near = max(max(qrow - rhi, rlo - qrow), 0);
      const int far = max(qrow - rlo, rhi - qrow);
      int d = slope2 >= 0.f ? near : far;
      if (KEEP && slope2 != 0.f)
        d = segment_distance(p, list, n_ent, segk_b, segq, qrow, row_ok, rlo,
                             rhi, slope2 >= 0.f);
      ref -= slope2 * static_cast<float>(d);
    }
    uint32_t unit_pv = 0;
    bool ok = true;
    for (int e = 0; e < n_ent; ++e) {
      const uint32_t ent = list[e];
      const int cls = static_cast<int>(ent & 3u);
      const int jt = static_cast<int>(ent >> 2);
      const int kbase = jt * kTileN + hf * NC;
      uint32_t keep[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
      if (KEEP && cls == 1)
        segment_bits<NC>(keep, segk_b + kbase,
                         min(max(p.Skv - kbase, 0), NC), segq);
      ok = warp_wait(&bars->s_full[t], s_cnt & 1, abort_flag, p.timeout_ns);
      if (!ok) {
        record_timeout(kRoleScore, 1);
        break;
      }
      ++s_cnt;
      if (tracer) dt_trace<TRACE>(p, bars, kRoleScore, kEvSFull, t, e, unit);
      tc_fence_after();
      uint32_t sraw[NC];
#pragma unroll
      for (int q = 0; q < NC / 32; ++q)
        tmem_ld32(s_addr + hf * NC + q * 32, sraw + q * 32);
      tmem_ld_wait();
      float* s = reinterpret_cast<float*>(sraw);
      if (hf == 0) {  // half 1 may write over S
        tc_fence_before();
        mbar_arrive(meet);
      }
      float sl8, cbase;  // bias of each 8 columns
      modify_tile<MOD, NC>(s, p, kbase, qrow, cls == 1, rlo - kbase,
                           rhi - kbase, keep, KEEP, slope2, &sl8, &cbase);
      if (MOD == kModCap) sl8 = cbase = 0.f;
      if (cls == 1) mask_tile<NC>(s, rlo - kbase, rhi - kbase, keep, KEEP);

      if (unit_pv == 0) {  // the two halves' maxima
        pair->sum[sums & 1][t][hf][r] = biased_max<NC>(s, sl8, cbase);
        mbar_arrive(&bars->meet_sum[t][quarter]);
        ok = warp_wait(&bars->meet_sum[t][quarter], sums & 1, abort_flag,
                       p.timeout_ns);
        if (!ok) {
          record_timeout(kRoleScore, 9);
          break;
        }
        ref = fmax3(ref, pair->sum[sums & 1][t][0][r],
                    pair->sum[sums & 1][t][1][r]);
        ++sums;
      }
      float ls0 = 0.f, ls1 = 0.f, ls2 = 0.f, ls3 = 0.f;
#pragma unroll
      for (int q = 0; q < NC / 32; ++q) {  // 32 columns at a time
        uint32_t pk[16];
#pragma unroll
        for (int c = 32 * q; c < 32 * q + 32; c += 4) {
          const float add = fmaf(sl8, static_cast<float>(c / 8), cbase - ref);
          fadd2(s[c], s[c + 1], s[c], s[c + 1], add, add);
          fadd2(s[c + 2], s[c + 3], s[c + 2], s[c + 3], add, add);
          const float p0 = ex2_approx(s[c]), p1 = ex2_approx(s[c + 1]);
          const float p2 = ex2_approx(s[c + 2]), p3 = ex2_approx(s[c + 3]);
          fadd2(ls0, ls1, ls0, ls1, p0, p1);
          fadd2(ls2, ls3, ls2, ls3, p2, p3);
          pk[(c & 31) / 2] = pack_bf16x2(p0, p1);
          pk[(c & 31) / 2 + 1] = pack_bf16x2(p2, p3);
        }
        if (hf == 1 && q == 0) {
          ok = warp_wait(meet, meets & 1, abort_flag, p.timeout_ns);
          tc_fence_after();
        }
        tmem_st16(s_addr + hf * 32 + q * 16, pk);
      }
      ++meets;
      if (!ok) {
        record_timeout(kRoleScore, 6);
        break;
      }
      l_sum += (ls0 + ls1) + (ls2 + ls3);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bars->p_full[t]);
      if (tracer) dt_trace<TRACE>(p, bars, kRoleScore, kEvPFull, t, e, unit);
      ++pv_cnt;
      ++unit_pv;
    }
    if (!ok) break;

    // ---- epilogue: out = O / l, bf16; each thread half of the row
    if (tracer) dt_trace<TRACE>(p, bars, kRoleScore, kEvEpiBegin, t, 0, unit);
    uint16_t* orow = p.out + static_cast<int64_t>(uc.b) * p.o_sb +
                     static_cast<int64_t>(uc.h) * p.o_sh +
                     static_cast<int64_t>(qrow) * p.o_ss + hf * (D / 2);
    if (unit_pv > 0) {
      // the two halves' sums
      pair->sum[sums & 1][t][hf][r] = l_sum;
      mbar_arrive(&bars->meet_sum[t][quarter]);
      if (!warp_wait(&bars->meet_sum[t][quarter], sums & 1, abort_flag,
                     p.timeout_ns)) {
        record_timeout(kRoleScore, 7);
        break;
      }
      l_sum = pair->sum[sums & 1][t][0][r] + pair->sum[sums & 1][t][1][r];
      ++sums;
      if (!warp_wait(&bars->pv_done[t], (pv_cnt - 1) & 1, abort_flag,
                     p.timeout_ns)) {
        record_timeout(kRoleScore, 3);
        break;
      }
      tc_fence_after();
      uint32_t o[D / 2];
#pragma unroll
      for (int q = 0; q < D / 64; ++q) tmem_ld32(o_addr + q * 32, o + q * 32);
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(&bars->o_free[t]);
      if (SHARED) {
        float* at = merge + hf * (D / 2) * kTileM + r;
        if (t == 1) {  // O, sum and reference for pipeline 0
#pragma unroll
          for (int c = 0; c < D / 2; ++c)
            at[c * kTileM] = __uint_as_float(o[c]);
          if (hf == 0) pair->total[r] = l_sum;
          if (hf == 0) pair->ref[r] = ref;
          mbar_arrive(&bars->merge);
          mbar_arrive(&bars->list_free[t][buf]);
          continue;
        }
        if (!warp_wait(&bars->merge, 0, abort_flag, p.timeout_ns)) {
          record_timeout(kRoleScore, 8);
          break;
        }
        const float l1 = pair->total[r];
        if (!(l1 == 0.f)) {  // (0: it saw nothing, or had no entry)
          // by the size of the sums, as the references may lie anywhere below
          // them (unsorted ids: each pipeline's by the keys of its own tiles)
          const float r1 = pair->ref[r];
          const float m0 = l_sum == 0.f ? NEG_INF : ref + exponent_of(l_sum);
          const float mm = fmaxf(m0, r1 + exponent_of(l1));
          const float w0 = l_sum == 0.f ? 0.f : ex2_approx(ref - mm);
          const float w1 = ex2_approx(r1 - mm);
          ref = mm;
#pragma unroll
          for (int c = 0; c < D / 2; ++c)
            o[c] = __float_as_uint(
                fmaf(at[c * kTileM], w1, __uint_as_float(o[c]) * w0));
          l_sum = fmaf(l1, w1, l_sum * w0);
        }
      }
      const float inv = has_sum<MOD>(l_sum) ? 1.f / l_sum : 0.f;
      if (row_ok) {
        const bool v8 = p.o_vec8 != 0;
#pragma unroll
        for (int v = 0; v < D / 32; ++v) {
          uint32_t w[8];
#pragma unroll
          for (int c = 0; c < 8; ++c)
            w[c] = pack_bf16x2(__uint_as_float(o[16 * v + 2 * c]) * inv,
                               __uint_as_float(o[16 * v + 2 * c + 1]) * inv);
          if (v8) {
            st_global_v8(orow + v * 16, w);
          } else {
            st_global_v4(orow + v * 16, w[0], w[1], w[2], w[3]);
            st_global_v4(orow + v * 16 + 8, w[4], w[5], w[6], w[7]);
          }
        }
      }
    } else if (SHARED && t == 1) {
      if (hf == 0) pair->total[r] = 0.f;
      tc_fence_before();
      mbar_arrive(&bars->o_free[t]);
      mbar_arrive(&bars->merge);
      mbar_arrive(&bars->list_free[t][buf]);
      continue;
    } else {
      if (row_ok) {
#pragma unroll
        for (int v = 0; v < D / 16; ++v)
          st_global_v4(orow + v * 8, 0u, 0u, 0u, 0u);
      }
      tc_fence_before();
      mbar_arrive(&bars->o_free[t]);
    }
    if (hf == 0 && p.lse != nullptr && row_ok) {
      const float lse = has_sum<MOD>(l_sum)
                            ? (ref + log2f(l_sum)) * 0.6931471805599453f
                            : NEG_INF;
      p.lse[(static_cast<int64_t>(uc.b) * p.H + uc.h) * p.Sq + qrow] = lse;
    }
    mbar_arrive(&bars->list_free[t][buf]);
    if (tracer) dt_trace<TRACE>(p, bars, kRoleScore, kEvEpiEnd, t, 0, unit);
  }
}

template <int D, int SCORE, int MOD, bool TRACE, bool SHARED>
__global__ void __launch_bounds__(dt_threads(MOD), 1)
    splash_fwd_dt_kernel(const __grid_constant__ CUtensorMap tm_q,
                         const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v,
                         const FwdParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  DtBars* bars = reinterpret_cast<DtBars*>(smem + kDtOffBar);
  // the CTA's lists: kListBufs per pipeline
  uint16_t* lists = p.lists + static_cast<size_t>(blockIdx.x) * 2 * kListBufs *
                                  kMaxKvTiles;
  const int warp = threadIdx.x / 32;

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      for (int i = 0; i < kListBufs; ++i) {
        mbar_init(&bars->list_full[t][i], 1);
        // load, MMA, score
        mbar_init(&bars->list_free[t][i], 2 + dt_score_threads(MOD));
      }
      mbar_init(&bars->q_full[t], 1);
      mbar_init(&bars->q_empty[t], 1);
      for (int s = 0; s < 2; ++s) {
        mbar_init(&bars->kv_full[t][s], 1);
        mbar_init(&bars->kv_empty[t][s], 1);
      }
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t], dt_score_threads(MOD));
      mbar_init(&bars->pv_done[t], 1);
      mbar_init(&bars->o_free[t], dt_score_threads(MOD));
      mbar_init(&bars->mma_done[t], 1);
      for (int q = 0; q < 4; ++q) {
        mbar_init(&bars->meet[t][q], 32);  // half 0 tells half 1
        mbar_init(&bars->meet_sum[t][q], 64);
      }
      mbar_init(&bars->merge, dt_score_threads(MOD));
    }
    bars->abort = 0;
    for (int i = 0; i < 6; ++i) bars->trace_n[i] = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (MOD == kModBias) {  // A, -A and zeros (B comes with each unit)
    for (int i = threadIdx.x; i < kTileM * 8; i += dt_threads(MOD)) {
      const uint32_t one = i % 8 == 4 ? 0x3f80u : i % 8 == 6 ? 0xbf80u : 0u;
      *bias_piece(smem, i / 8, i % 8) = make_uint4(one | one << 16, one, 0u, 0u);
    }
    fence_proxy_async();
  }
  if (warp == 2) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp < 4) {
    if (!dt_two_per_row(MOD)) setmaxnreg_dec<kRegsLight>();
    const int t = warp & 1;
    uint16_t* lt = lists + t * kListBufs * kMaxKvTiles;
    if (warp < 2)
      dt_load_role<D, MOD, TRACE, SHARED>(p, &tm_q, &tm_k, &tm_v, smem, bars, lt, t);
    else
      dt_mma_role<D, SCORE, MOD, TRACE>(p, smem, bars, lt, tmem, t);
  } else {
    // per-element keep bits only when segment ids are unsorted or an
    // arbitrary mask is given (read once; the same for every thread)
    DtPair* pair = reinterpret_cast<DtPair*>(smem + kDtOffPair);
    float* merge = reinterpret_cast<float*>(smem + kDtOffMerge);
    if constexpr (!dt_two_per_row(MOD)) {
      setmaxnreg_inc<kRegsScore>();
      const int t = (warp - 4) / 4;
      const uint16_t* lt = lists + t * kListBufs * kMaxKvTiles;
      if (((p.flags & BSM_MASK_SEGMENT) && (*p.seg_flags & 1) != 0) ||
          p.dense != nullptr)
        dt_score_role<D, SCORE, MOD, true, TRACE, SHARED>(p, bars, pair, merge,
                                                          lt, tmem, t);
      else
        dt_score_role<D, SCORE, MOD, false, TRACE, SHARED>(p, bars, pair, merge,
                                                           lt, tmem, t);
    } else {
      const int t = (warp - 4) / 8, hf = (warp - 4) / 4 & 1;
      const uint16_t* lt = lists + t * kListBufs * kMaxKvTiles;
      // (an arbitrary mask with modified scores takes the lockstep kernel)
      if ((p.flags & BSM_MASK_SEGMENT) && (*p.seg_flags & 1) != 0)
        dt_score_cap_role<D, MOD, true, TRACE, SHARED>(p, bars, pair, merge,
                                                       lt, tmem, t, hf);
      else
        dt_score_cap_role<D, MOD, false, TRACE, SHARED>(p, bars, pair, merge,
                                                        lt, tmem, t, hf);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, kTmemCols);
  if (TRACE && threadIdx.x == 0) {
    uint32_t* hdr = reinterpret_cast<uint32_t*>(
        reinterpret_cast<TraceRec*>(p.trace) +
        static_cast<size_t>(blockIdx.x) * (p.trace_cap + 2));
    const uint32_t per = p.trace_cap / 6;
    for (int i = 0; i < 8; ++i) hdr[i] = i < 6 ? min(bars->trace_n[i], per) : 0;
  }
}

template <int D, int SCORE, int MOD>
cudaError_t launch_dt(const FwdParams& p, const CUtensorMap& tq,
                      const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                      int num_sms, cudaStream_t stream) {
  // the instance that records the event trace is launched only with one
  auto kern = p.trace != nullptr
                  ? splash_fwd_dt_kernel<D, SCORE, MOD, true, false>
                  : splash_fwd_dt_kernel<D, SCORE, MOD, false, false>;
  if constexpr (MOD != 0) {
    // a CTA for every query tile, where there are SMs enough
    if (p.trace == nullptr && p.unit_counter == nullptr &&
        2 * p.num_units <= num_sms) {
      kern = splash_fwd_dt_kernel<D, SCORE, MOD, false, true>;
      grid = 2 * p.num_units;
    }
  }
  cudaFuncAttributes attr;
  cudaError_t e = cudaFuncGetAttributes(&attr, kern);
  if (e != cudaSuccess) return e;
  if (!dt_two_per_row(MOD) && attr.numRegs * kDtThreads < kRegsNeeded)
    return cudaErrorInvalidConfiguration;
  constexpr int kSmem = kDtSmemBytes + (MOD != 0 ? sizeof(DtPair) : 0) +
                        (MOD == kModBias ? kDtBiasBytes : 0);
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSmem);
  if (e != cudaSuccess) return e;
  kern<<<grid, dt_threads(MOD), kSmem, stream>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

template <int D, int SCORE, int MOD, bool PINGPONG>
cudaError_t launch_one(const FwdParams& p, const CUtensorMap& tq,
                       const CUtensorMap& tk, const CUtensorMap& tv,
                       int grid, cudaStream_t stream) {
  using C = Cfg<D>;
  auto kern = splash_fwd_kernel<D, SCORE, MOD, PINGPONG>;
  cudaFuncAttributes attr;
  cudaError_t e = cudaFuncGetAttributes(&attr, kern);
  if (e != cudaSuccess) return e;
  // the setmaxnreg split must fit the registers the CTA is launched with,
  // else the score warps would wait for registers forever
  if (attr.numRegs * kThreads < kRegsNeeded) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           C::kSmemBytes);
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, C::kSmemBytes, stream>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

// The instances of one score path (SCORE and, for the softmax, the kind of
// modified scores MOD).
template <int SCORE, int MOD>
cudaError_t launch_score(const FwdParams& p, const CUtensorMap& tq,
                         const CUtensorMap& tk, const CUtensorMap& tv,
                         int grid, int num_sms, cudaStream_t stream) {
  // Softmax turns alternate between the tiles only where work units are
  // long: no segment ids and at least 4096 keys.  Packed sequences and
  // short sequences give short units, where the alternation costs more
  // than it saves.  Arbitrary masks take the other instance too, which
  // keeps the alternating one free of per-element keep bits; head dim 64
  // is built without it.
  const bool pp = (p.flags & BSM_MASK_SEGMENT) == 0 && p.Skv >= 4096 &&
                  p.dense == nullptr && p.D == 128;
  // Packed sequences (segment ids, no arbitrary mask) at head dim 128 take
  // the kernel with decoupled query tiles, and so do the other masks below
  // 4096 keys (causal S=2048: 11 % faster there; from 4096 keys on, the
  // lockstep kernel's shared K/V stream is 2-6 % faster).
  // Modified scores take it at every length: their softmax, not the tensor
  // core, sets the pace, and its turns in the lockstep kernel leave half the
  // score warps waiting (causal S=8192, 32/8 heads, in one form of the scores:
  // cap 50 672 us there, 623 here; bias 618 and 524; both 1049 and 757).
  // (Caps with a fixed reference, which only that kernel has, do not come here.)
  const bool dt = MOD != 0 ? p.D == 128 && fwd_mod_dt(p)
                           : p.dense == nullptr && p.D == 128 &&
                                 ((p.flags & BSM_MASK_SEGMENT) != 0 ||
                                  p.Skv < 4096);
  if (dt) return launch_dt<128, SCORE, MOD>(p, tq, tk, tv, grid, num_sms, stream);
  if constexpr (MOD != 0) {  // and at head dim 64 too
    if (p.D == 64 && fwd_mod_dt(p))
      return launch_dt<64, SCORE, MOD>(p, tq, tk, tv, grid, num_sms, stream);
  }
  if constexpr (MOD == 0) {
    if (p.D == 128 && pp)
      return launch_one<128, SCORE, MOD, true>(p, tq, tk, tv, grid, stream);
  }
  if (p.D == 128)
    return launch_one<128, SCORE, MOD, false>(p, tq, tk, tv, grid, stream);
  if (p.D == 64)  // head dim 64 uses the instance without alternation
    return launch_one<64, SCORE, MOD, false>(p, tq, tk, tv, grid, stream);
  return cudaErrorInvalidValue;
}

// Self test of the bounded wait: nothing ever arrives on this barrier.
__global__ void wait_selftest_kernel(uint64_t timeout_ns) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    if (!mbar_wait(&bar, 0, &abort_flag, timeout_ns)) record_timeout(0, 7);
  }
  __syncthreads();
}

}  // namespace

int fwd_grid_size(const FwdParams& p, int num_sms) {
  return p.num_units < num_sms ? p.num_units : num_sms;
}

cudaError_t launch_splash_fwd(const FwdParams& p, const CUtensorMap& tq,
                              const CUtensorMap& tk, const CUtensorMap& tv,
                              int num_sms, cudaStream_t stream) {
  const int grid = fwd_grid_size(p, num_sms);
  if (p.score == BSM_SCORE_POINTWISE)
    return launch_score<BSM_SCORE_POINTWISE, 0>(p, tq, tk, tv, grid, num_sms, stream);
  // a cap with a fixed reference (see dt_score_cap_role), alone or with a bias
  const int kind = p.mod.kind;
  if (kind == kModCap && p.mod.cap_log2 <= 87.f && fwd_mod_dt(p))
    return p.D == 128 ? launch_dt<128, BSM_SCORE_SOFTMAX, kModCap>(
                            p, tq, tk, tv, grid, num_sms, stream)
                      : launch_dt<64, BSM_SCORE_SOFTMAX, kModCap>(
                            p, tq, tk, tv, grid, num_sms, stream);
  if (kind == (kModCap | kModBias) && p.mod.cap_log2 <= 75.f && fwd_mod_dt(p))
    return p.D == 128 ? launch_dt<128, BSM_SCORE_SOFTMAX, kModFixed>(
                            p, tq, tk, tv, grid, num_sms, stream)
                      : launch_dt<64, BSM_SCORE_SOFTMAX, kModFixed>(
                            p, tq, tk, tv, grid, num_sms, stream);
  switch (kind) {
    case 0:
      return launch_score<BSM_SCORE_SOFTMAX, 0>(p, tq, tk, tv, grid, num_sms, stream);
    case kModBias:
      return launch_score<BSM_SCORE_SOFTMAX, kModBias>(p, tq, tk, tv, grid, num_sms, stream);
    // larger caps and arbitrary masks: a running maximum (and, for a cap
    // alone, slopes of zero)
    case kModCap:
    case kModCap | kModBias:
      return launch_score<BSM_SCORE_SOFTMAX, kModCap | kModBias>(
          p, tq, tk, tv, grid, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_wait_selftest(uint64_t timeout_ns, cudaStream_t stream) {
  wait_selftest_kernel<<<1, 32, 0, stream>>>(timeout_ns);
  return cudaGetLastError();
}

cudaError_t read_device_error(int32_t out[4], cudaStream_t stream) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return e;
  e = cudaMemcpyFromSymbol(out, g_fwd_error, 4 * sizeof(int32_t));
  if (e != cudaSuccess) return e;
  const int32_t zero[4] = {0, 0, 0, 0};
  return cudaMemcpyToSymbol(g_fwd_error, zero, 4 * sizeof(int32_t));
}

}  // namespace bsm
