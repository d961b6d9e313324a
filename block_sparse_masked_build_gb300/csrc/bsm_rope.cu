// Norm and rotation of query and key rows for sm_103a (GB300), forward and
// backward.
//
// A row x [D] is normalised, n = x r with r = 1 / sqrt(mean(x^2) + eps), y =
// w n, and its first `dim` elements turn pair by pair by the angles of its
// token's position.  Backward, with g' = the gradient turned back:
//     dx = r (w g' - n mean(w g' n)),   dw = sum over rows of g' n.
//
// D / 16 neighbouring lanes hold one row, 16 elements each, chosen so that the
// two elements of a pair lie in one lane: the only exchange between lanes is
// the norm's sum.  Such a group of lanes takes `per` heads of one token, so
// that cosines, sines and weights are computed or read once for them, and has
// the next three heads' rows on their way while it works on one.
//
// Bound by memory: 4 bytes per element forward, 6 backward.  Measured, norm and
// rotation: a prompt of 8192 tokens, 32/8 heads of 128, 30.5 us (5.5 TB/s of a
// copy's 6.8); 2 x 16 heads of 8192 tokens, queries and keys, forward and
// backward 117 us (5.7 TB/s); one token for 8 sequences 7.5-11 us, the launch and
// a round trip.  Instructions issue in two thirds of the cycles, the most of what
// is left between these and the copy's rate.
// With few key heads lanes idle: a token's groups of queries and of keys share a
// warp and run the longer of their counts, and the backward's key blocks have a
// job's angles for one head each.  8192 tokens, 4 x 8/1 heads: forward 64 % of the
// copy's rate, backward 58 %; 2 x 16/2: 77 and 71 %; 32/8: 84 and 86 %.  Rotation
// alone: 80-90 % forward, 59 (8/1) to 84 % (16/16) backward.
#include <algorithm>
#include <cstdint>

#include "bsm_internal.h"
#include "bsm_ptx.cuh"
#include "bsm_rope.cuh"

namespace bsm {
namespace {

constexpr int kFwdThreads = 128, kBwdThreads = 256;
// MODE: how elements are paired
enum { kPlain = 0, kHalves = 1, kPairs = 2 };

// Pair i of a lane's 16 elements, turned by +angle (or -angle).
template <int MODE, bool BACK>
__device__ __forceinline__ void turn(float* v, const float* c, const float* s) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& a = MODE == kHalves ? v[i] : v[2 * i];
    float& b = MODE == kHalves ? v[8 + i] : v[2 * i + 1];
    const float sn = BACK ? -s[i] : s[i];
    const float x = a * c[i] - b * sn;
    b = b * c[i] + a * sn;
    a = x;
  }
}

// Sum over the D / 16 lanes of a row.
template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int d = 1; d < D / 16; d *= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

// What a group of lanes works on: heads [head, head + n) of one token.
struct Job {
  int which;  // 0 queries, 1 keys
  int b, s, head, n;
};

__device__ __forceinline__ Job job_of(const NormRopeParams& p, int which,
                                      uint32_t token, int chunk) {
  Job j;
  j.which = which;
  j.b = token / static_cast<uint32_t>(p.S);
  j.s = token - static_cast<uint32_t>(j.b) * p.S;
  j.head = chunk * p.per[which];
  j.n = min(p.per[which], p.heads[which] - j.head);
  return j;
}

__device__ __forceinline__ uint16_t* row_at(const RowView& v, const Job& j) {
  return v.data + j.b * v.sb + j.head * v.sh + j.s * v.ss;
}

// Rows on their way: a thread's 16 elements of kAhead rows to come, copied to
// its own places in shared memory, so that they take no registers (loads of the
// next row alone into registers left the forward pass at 67 % of the copy
// bandwidth, the backward one at 71 %).  One place more than rows on their way:
// a place is filled when the row read from it has been used.
constexpr int kAhead = 3, kPlaces = kAhead + 1;

__device__ __forceinline__ void fetch8(uint4* place, const uint16_t* p) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   smem_u32(place)),
               "l"(p)
               : "memory");
}
__device__ __forceinline__ void fetch_end() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void fetch_wait() {  // for the oldest of kAhead
  asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
}

__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                 pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

template <int MODE>
__device__ __forceinline__ void load_steps(const TurnParams& t,
                                           uint64_t* steps) {
  if (MODE != kPlain) {
    if (threadIdx.x < 64) steps[threadIdx.x] = t.rope.step[threadIdx.x];
    __syncthreads();
  }
}

template <int MODE>
__device__ __forceinline__ void job_turns(const TurnParams& t,
                                          const uint64_t* steps,
                                          const LanePart& part, const Job& j,
                                          float* c, float* s) {
  if (MODE != kPlain && part.freq >= 0)
    turns_of<8>(t.rope, steps + part.freq, part.freq,
                t.pos == nullptr ? nullptr
                                 : t.pos + j.b * t.pos_sb + j.s * t.pos_ss,
                t.pos_sa, j.s, c, s);
}

template <int D, int MODE, bool NORM>
__global__ void __launch_bounds__(kFwdThreads)
    norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int L = D / 16, kGroups = kFwdThreads / L;
  __shared__ uint64_t steps[64];
  load_steps<MODE>(p.turn, steps);
  const uint32_t tokens = static_cast<uint32_t>(p.B) * p.S;
  const uint32_t chunks = p.chunks[0] + p.chunks[1];
  const uint32_t job = blockIdx.x * kGroups + threadIdx.x / L;
  const uint32_t token = job / chunks;
  const bool live = token < tokens;  // (every lane stays for the row sums)
  int chunk = job - token * chunks;
  const int which = chunk >= p.chunks[0];
  if (which) chunk -= p.chunks[0];
  Job j = job_of(p, which, live ? token : 0, chunk);
  if (!live) j.n = 0;
  const LanePart part =
      lane_part(threadIdx.x % L, p.turn.rope.dim, MODE == kHalves);
  const uint16_t* src = row_at(p.x[which], j);
  uint16_t* dst = row_at(p.out[which], j);
  const int64_t src_sh = p.x[which].sh, dst_sh = p.out[which].sh;
  __shared__ uint4 rows[kPlaces][2][kFwdThreads];
  auto fetch = [&](int i) {  // (a row that is not there leaves its place as is)
    if (i < j.n) {
      fetch8(&rows[i % kPlaces][0][threadIdx.x], src + part.at0);
      fetch8(&rows[i % kPlaces][1][threadIdx.x], src + part.at1);
    }
    fetch_end();
    src += src_sh;
  };
  for (int i = 0; i < kAhead; ++i) fetch(i);
  float w[16], c[8], s[8];
  if (NORM) {
    const void* wt = which ? p.turn.k_weight : p.turn.q_weight;
    weights_of(wt, p.turn.weights_bf16, part.at0, w);
    weights_of(wt, p.turn.weights_bf16, part.at1, w + 8);
  }
  job_turns<MODE>(p.turn, steps, part, j, c, s);
  const int trips = max(p.per[0], p.per[1]);  // the same in a whole warp
  for (int i = 0; i < trips; ++i) {
    float v[16];
    fetch_wait();
    fetch(i + kAhead);
    unpack_bf16x8(rows[i % kPlaces][0][threadIdx.x], v);
    unpack_bf16x8(rows[i % kPlaces][1][threadIdx.x], v + 8);
    if (NORM) {
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) sum = fmaf(v[e], v[e], sum);
      const float r = rsqrtf(fmaf(row_sum<D>(sum), 1.f / D, p.turn.eps));
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = v[e] * r * w[e];
    }
    if (MODE != kPlain && part.freq >= 0) turn<MODE, false>(v, c, s);
    if (i < j.n) {
      store8(dst + part.at0, v);
      store8(dst + part.at1, v + 8);
    }
    dst += dst_sh;
  }
}

// Blocks [0, blocks[0]) take the queries, the others the keys, each its share
// of the jobs in a fixed order, and leave their sums of g' n, one f32 per
// element, to be added up by the kernel below.
template <int D, int MODE, bool NORM>
__global__ void __launch_bounds__(kBwdThreads, 2)
    norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int L = D / 16, kGroups = kBwdThreads / L;
  __shared__ uint64_t steps[64];
  constexpr int kParts = NORM ? 4 : 2;  // of 8 elements: gradient, row
  extern __shared__ __align__(16) uint4 rows[];  // [kPlaces][kParts][threads]
  float* sums = reinterpret_cast<float*>(rows);  // at the end: [kGroups][D]
  // the sums' kernel may be scheduled; it waits for this grid's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  load_steps<MODE>(p.turn, steps);
  const int which = static_cast<int>(blockIdx.x) >= p.blocks[0];
  const uint32_t block = blockIdx.x - (which ? p.blocks[0] : 0);
  const int group = threadIdx.x / L;
  const LanePart part =
      lane_part(threadIdx.x % L, p.turn.rope.dim, MODE == kHalves);
  float w[16], acc[16], c[8], s[8];
  if (NORM) {
    const void* wt = which ? p.turn.k_weight : p.turn.q_weight;
    weights_of(wt, p.turn.weights_bf16, part.at0, w);
    weights_of(wt, p.turn.weights_bf16, part.at1, w + 8);
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  }
  const uint32_t chunks = p.chunks[which];
  const uint32_t jobs = static_cast<uint32_t>(p.B) * p.S * chunks;
  const uint32_t stride = p.blocks[which] * kGroups;
  const int per = p.per[which];
  const int64_t x_sh = p.x[which].sh, g_sh = p.g[which].sh,
                o_sh = p.out[which].sh;
  auto job_at = [&](uint32_t base) {
    const uint32_t job = base + group;
    const uint32_t token = job / chunks;
    Job j = job_of(p, which, job < jobs ? token : 0, job - token * chunks);
    if (job >= jobs) j.n = 0;
    return j;
  };
  // the next row to fetch: row f_i of the job at f_base, across jobs
  uint32_t f_base = block * kGroups;
  int f_i = 0, f_n = 0, f_place = 0;
  const uint16_t *f_x = nullptr, *f_g = nullptr;
  auto fetch = [&] {
    if (f_i == 0 && f_base < jobs) {
      const Job j = job_at(f_base);
      f_n = j.n;
      f_g = row_at(p.g[which], j);
      if (NORM) f_x = row_at(p.x[which], j);
    }
    if (f_base < jobs && f_i < f_n) {
      uint4* place = rows + f_place * kParts * kBwdThreads + threadIdx.x;
      fetch8(place, f_g + part.at0);
      fetch8(place + kBwdThreads, f_g + part.at1);
      f_g += g_sh;
      if (NORM) {
        fetch8(place + 2 * kBwdThreads, f_x + part.at0);
        fetch8(place + 3 * kBwdThreads, f_x + part.at1);
        f_x += x_sh;
      }
    }
    fetch_end();
    f_place = (f_place + 1) % kPlaces;
    if (++f_i == per) {
      f_i = 0;
      f_base += stride;
    }
  };
  for (int i = 0; i < kAhead; ++i) fetch();
  int at = 0;
  for (uint32_t base = block * kGroups; base < jobs; base += stride) {
    const Job j = job_at(base);
    uint16_t* dst = row_at(p.out[which], j);
    job_turns<MODE>(p.turn, steps, part, j, c, s);
    for (int i = 0; i < per; ++i) {
      float h[16], v[16];
      fetch_wait();
      fetch();
      const uint4* place = rows + at * kParts * kBwdThreads + threadIdx.x;
      at = (at + 1) % kPlaces;
      unpack_bf16x8(place[0], h);
      unpack_bf16x8(place[kBwdThreads], h + 8);
      if (NORM) {
        unpack_bf16x8(place[2 * kBwdThreads], v);
        unpack_bf16x8(place[3 * kBwdThreads], v + 8);
      }
      if (MODE != kPlain && part.freq >= 0) turn<MODE, true>(h, c, s);
      if (NORM) {
        float sq = 0.f, dot = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          sq = fmaf(v[e], v[e], sq);
          dot = fmaf(h[e] * w[e], v[e], dot);
        }
        sq = row_sum<D>(sq);
        dot = row_sum<D>(dot);
        const float r = rsqrtf(fmaf(sq, 1.f / D, p.turn.eps));
        const float m = dot * r * (1.f / D);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float n = v[e] * r;
          if (i < j.n) acc[e] = fmaf(h[e], n, acc[e]);
          h[e] = r * fmaf(-n, m, h[e] * w[e]);
        }
      }
      if (i < j.n) {
        store8(dst + part.at0, h);
        store8(dst + part.at1, h + 8);
      }
      dst += o_sh;
    }
  }
  if (NORM && p.partial != nullptr) {
    __syncthreads();  // (no row is on its way or being read)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sums[group * D + part.at0 + e] = acc[e];
      sums[group * D + part.at1 + e] = acc[8 + e];
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float sum = 0.f;
#pragma unroll 8
      for (int i = 0; i < kGroups; ++i) sum += sums[i * D + threadIdx.x];
      p.partial[static_cast<size_t>(blockIdx.x) * D + threadIdx.x] = sum;
    }
  }
}

// dw: 32 columns of the blocks' sums per CTA, a warp per every 32nd block.
__global__ void __launch_bounds__(1024)
    norm_rope_dw_kernel(const __grid_constant__ NormRopeParams p) {
  const int per = p.D / 32, which = blockIdx.x / per;
  const int col = blockIdx.x % per * 32 + threadIdx.x % 32;
  const int warp = threadIdx.x / 32;
  __shared__ float part[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.dw[which] == nullptr) return;
  const int first = which ? p.blocks[0] : 0;
  float sum = 0.f;
#pragma unroll 4
  for (int i = warp; i < p.blocks[which]; i += 32)
    sum += p.partial[static_cast<size_t>(first + i) * p.D + col];
  part[warp][threadIdx.x % 32] = sum;
  __syncthreads();
  if (warp > 0) return;
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) sum += part[i][threadIdx.x];
  p.dw[which][col] = sum;
}

// Heads per group of lanes: as many as leave `groups` groups with work, up to
// 8, and then as many as make a token's groups equal.
void choose_chunks(NormRopeParams& p, int64_t groups) {
  const int64_t tokens = static_cast<int64_t>(p.B) * p.S;
  const int64_t rows = tokens * (p.heads[0] + p.heads[1]);
  int per = 1;
  while (per < 8 && rows / (2 * per) >= groups) per *= 2;
  for (int i = 0; i < 2; ++i) {
    p.chunks[i] = (p.heads[i] + per - 1) / per;
    p.per[i] = p.chunks[i] ? (p.heads[i] + p.chunks[i] - 1) / p.chunks[i] : 0;
  }
}

int mode_of(const NormRopeParams& p) {
  return p.turn.rope.dim == 0 ? kPlain
         : p.turn.rope.interleaved ? kPairs
                                   : kHalves;
}

template <int D, int MODE>
void launch_fwd(const NormRopeParams& p, cudaStream_t stream) {
  constexpr int kGroups = kFwdThreads / (D / 16);
  const int64_t jobs =
      static_cast<int64_t>(p.B) * p.S * (p.chunks[0] + p.chunks[1]);
  const unsigned grid = static_cast<unsigned>((jobs + kGroups - 1) / kGroups);
  if (p.turn.norm)
    norm_rope_kernel<D, MODE, true><<<grid, kFwdThreads, 0, stream>>>(p);
  else if (MODE != kPlain)
    norm_rope_kernel<D, MODE, MODE == kPlain>
        <<<grid, kFwdThreads, 0, stream>>>(p);
}

template <int D, int MODE, bool NORM>
cudaError_t launch_bwd_as(const NormRopeParams& p, cudaStream_t stream) {
  constexpr int kSmem = kPlaces * (NORM ? 4 : 2) * kBwdThreads * 16;
  static_assert(!NORM || kBwdThreads / (D / 16) * D * 4 <= kSmem, "sums");
  const cudaError_t e = cudaFuncSetAttribute(
      norm_rope_bwd_kernel<D, MODE, NORM>,
      cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  norm_rope_bwd_kernel<D, MODE, NORM>
      <<<p.blocks[0] + p.blocks[1], kBwdThreads, kSmem, stream>>>(p);
  return cudaGetLastError();
}

template <int D, int MODE>
cudaError_t launch_bwd(const NormRopeParams& p, cudaStream_t stream) {
  if (p.turn.norm) return launch_bwd_as<D, MODE, true>(p, stream);
  // (neither norm nor rotation: refused before)
  return launch_bwd_as<D, MODE == kPlain ? kHalves : MODE, false>(p, stream);
}

}  // namespace

cudaError_t launch_norm_rope(NormRopeParams& p, int num_sms,
                             cudaStream_t stream) {
  choose_chunks(p, int64_t{64} * num_sms);
  const int mode = mode_of(p);
  if (p.D == 128)
    mode == kPlain    ? launch_fwd<128, kPlain>(p, stream)
    : mode == kHalves ? launch_fwd<128, kHalves>(p, stream)
                      : launch_fwd<128, kPairs>(p, stream);
  else
    mode == kPlain    ? launch_fwd<64, kPlain>(p, stream)
    : mode == kHalves ? launch_fwd<64, kHalves>(p, stream)
                      : launch_fwd<64, kPairs>(p, stream);
  return cudaGetLastError();
}

cudaError_t launch_norm_rope_bwd(NormRopeParams& p, int num_sms,
                                 cudaStream_t stream) {
  choose_chunks(p, int64_t{64} * num_sms);
  const int groups = kBwdThreads / (p.D / 16);
  // blocks of queries and keys by their rows, all resident at once
  const int64_t tokens = static_cast<int64_t>(p.B) * p.S;
  const int64_t all = std::min(2 * num_sms, kNormRopeMaxBlocks - 2);
  const int64_t heads = std::max(p.heads[0] + p.heads[1], 1);
  for (int i = 0; i < 2; ++i) {
    const int64_t need = (tokens * p.chunks[i] + groups - 1) / groups;
    const int64_t share = (all * p.heads[i] + heads / 2) / heads;
    p.blocks[i] = static_cast<int32_t>(
        std::min(need, std::max<int64_t>(share, p.heads[i] > 0 ? 1 : 0)));
  }
  const bool dw = p.dw[0] != nullptr || p.dw[1] != nullptr;
  if (!dw) p.partial = nullptr;
  const int mode = mode_of(p);
  cudaError_t e = cudaSuccess;
  if (p.blocks[0] + p.blocks[1] == 0)
    ;  // no rows: sums of nothing below
  else if (p.D == 128)
    e = mode == kPlain    ? launch_bwd<128, kPlain>(p, stream)
        : mode == kHalves ? launch_bwd<128, kHalves>(p, stream)
                          : launch_bwd<128, kPairs>(p, stream);
  else
    e = mode == kPlain    ? launch_bwd<64, kPlain>(p, stream)
        : mode == kHalves ? launch_bwd<64, kHalves>(p, stream)
                          : launch_bwd<64, kPairs>(p, stream);
  if (e != cudaSuccess || !dw) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * p.D / 32);
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_rope_dw_kernel, p);
}

}  // namespace bsm
