// Mixture-of-experts layer on packed 4-bit weights: router, slot lists,
// expert-selected products and the whole layer.
//
// Token m has top_k choices; slot p = m * top_k + j is its choice j, an
// expert e with a weight r. With W_e the expert's matrix,
// w[n,k] = (q[n,k] - z[n,k/bs]) * s[n,k/bs]:
//   product   Y[p] = W_e A[m or p] + b_e
//   layer     Y[m] = sum_j r_j (Wd_e (silu(Wg_e x + bg) * (Wu_e x + bu)) + bd)
// The page "Qwen3 CPU Inference Critical Path" lists MoE and QMoE in its
// operator inventory; the router's conventions are in moe_route.cuh.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <initializer_list>
#include <utility>

#include "mnb_common.cuh"
#include "mnb_launch.h"
#include "moe.h"
#include "moe_half.cuh"
#include "moe_lists.cuh"
#include "moe_route.cuh"
#include "moe_stream.h"
#include "moe_tile.h"

namespace mnb {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kPrepWarps = 32;  // a warp per token of a short input
constexpr int kPrepThreads = kPrepWarps * 32;

__device__ __forceinline__ void store_f(void *p, bool f32, int64_t i, float v) {
  if (f32) static_cast<float *>(p)[i] = v;
  else static_cast<uint16_t *>(p)[i] = static_cast<uint16_t>(bf16_bits(v));
}

// ---- re-layout of a stack of weights ---------------------------------------

// Row n of the padded stack is row n % Np of expert n / Np (Np = N rounded up
// to whole tiles); padding rows are zero codes and zero scales.
__global__ void pack_expert_codes_kernel(const uint8_t *__restrict__ B,
                                         uint32_t *__restrict__ out, int64_t N, int64_t Np,
                                         int64_t K, int bs, int64_t nb, int64_t K64,
                                         int64_t words) {
  for (int64_t w = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; w < words;
       w += (int64_t)gridDim.x * blockDim.x) {
    const int64_t chunk = w >> 7;
    const int idx = static_cast<int>(w & 127);
    const int lane = idx >> 2, j = idx & 3, g = lane >> 2, t = lane & 3;
    const int64_t tile = chunk / K64, c = chunk % K64;
    const int64_t k0 = c * kChunkK + 16 * j + 4 * t;
    uint32_t word = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t row = tile * kTileN + g + 8 * h, e = row / Np, n = row % Np;
      if (n >= N) continue;
      // Blocks have 16 codes or more: four consecutive codes share a block.
      const uint8_t *src =
          B + ((e * N + n) * nb + k0 / bs) * (bs / 2) + (k0 % bs) / 2;
#pragma unroll
      for (int o = 0; o < 4; ++o)
        if (k0 + o < K)
          word |= static_cast<uint32_t>((src[o >> 1] >> (4 * (o & 1))) & 15) << code_shift(o, h);
    }
    out[w] = word;
  }
}

template <typename T>
__global__ void pack_expert_scales_kernel(const T *__restrict__ s, T *__restrict__ out,
                                          int64_t N, int64_t Np, int64_t nb, int64_t total) {
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t tb = i >> 4, tile = tb / nb, b = tb % nb;
    const int64_t row = tile * kTileN + (i & 15), e = row / Np, n = row % Np;
    out[i] = n < N ? s[(e * N + n) * nb + b] : T(0);
  }
}

__global__ void pack_expert_zp_kernel(const uint8_t *__restrict__ zp,
                                      uint64_t *__restrict__ out, int64_t N, int64_t Np,
                                      int64_t nb, int64_t nbz, int64_t total) {
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t tile = i / nbz, b = i % nbz;
    uint64_t word = 0;
    for (int r = 0; r < kTileN && b < nb; ++r) {
      const int64_t row = tile * kTileN + r, e = row / Np, n = row % Np;
      if (n >= N) break;
      const uint8_t byte = zp[(e * N + n) * ((nb + 1) / 2) + b / 2];
      word |= static_cast<uint64_t>((byte >> (4 * (b & 1))) & 15) << (4 * r);
    }
    out[i] = word;
  }
}

// Per packed row: the power of two that brings its largest |scale| into
// 2^14 .. 2^15; per expert: the largest |scale| (bits, cleared before). A warp
// per 16-row tile.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    row_scales_kernel(const T *__restrict__ s, float *__restrict__ rows, uint32_t *smax, int64_t E,
                      int64_t N16, int64_t nb) {
  const int lane = threadIdx.x & 31, r = lane & 15;
  for (int64_t tile = blockIdx.x * int64_t(kWarps) + (threadIdx.x >> 5); tile < E * N16;
       tile += int64_t(gridDim.x) * kWarps) {
    uint32_t top = 0;
    for (int64_t b = lane >> 4; b < nb; b += 2) {
      const T v = s[(tile * nb + b) * kTileN + r];
      const uint32_t u = sizeof(T) == 4 ? __float_as_uint(v) : uint32_t(v) << 16;
      top = max(top, u & 0x7FFFFFFFu);
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
    if (lane < 16) rows[tile * kTileN + r] = exp2i(row_shift(top));
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) atomicMax(smax + tile / N16, top);
  }
}

inline unsigned grid_of(int64_t total, int per) {
  return static_cast<unsigned>(
      std::max<int64_t>(1, std::min<int64_t>(ceil_div(total, per), 1 << 20)));
}

// ---- router --------------------------------------------------------------------

// A warp per token.
__global__ void __launch_bounds__(kThreads)
    route_kernel(const void *logits, bool f32, int64_t M, int E, int top_k, bool normalize,
                 float *weights, int32_t *experts) {
  extern __shared__ uint32_t keys_all[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_dependents_launch();
  for (int64_t m = blockIdx.x * (int64_t)kWarps + warp; m < M; m += (int64_t)gridDim.x * kWarps) {
    int e;
    float r;
    route_row(logits, f32, m, E, top_k, normalize, keys_all + warp * E, e, r);
    if (lane < top_k) {
      experts[m * top_k + lane] = e;
      weights[m * top_k + lane] = r;
    }
  }
}

// Bits of the largest magnitude of row `row` of A [.., K], by one block.
__device__ __forceinline__ uint32_t row_top(const void *A, bool f32, bool vec, int64_t row,
                                            int K, uint32_t *scratch) {
  uint32_t top = 0;
  const int64_t at = row * K;
  if (vec) {
    const uint4 *a = reinterpret_cast<const uint4 *>(static_cast<const char *>(A) +
                                                     at * (f32 ? 4 : 2));
    const int n = K / (f32 ? 4 : 8);
#pragma unroll 2
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const uint4 x = a[i];
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        top = max(top, w[q] & (f32 ? 0x7FFFFFFFu : 0x7FFF0000u));
        if (!f32) top = max(top, (w[q] << 16) & 0x7FFF0000u);
      }
    }
  } else {
    for (int i = threadIdx.x; i < K; i += blockDim.x)
      top = max(top, (f32 ? static_cast<const uint32_t *>(A)[at + i]
                          : uint32_t(static_cast<const uint16_t *>(A)[at + i]) << 16) &
                         0x7FFFFFFFu);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = top;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  top = lane < blockDim.x >> 5 ? scratch[lane] : 0;
  top = __reduce_max_sync(0xffffffffu, top);
  return top;
}

// What the products need ahead, for a few slots, in one launch. Block 0: the
// router (or a table of experts) and the lists; the blocks after it: the
// largest magnitude of an activation row each, and cleared words.
struct PrepArgs {
  const void *logits;    // the router, or null:
  const int32_t *table;  // experts of the slots
  int logits_f32, normalize;
  int M, E, top_k, gt_log2;
  float *weights;
  int32_t *experts, *offsets, *order, *n_groups;  // weights, experts: router only
  SlotGroup *groups;                              // and n_groups: may be null
  const void *A;
  int a_f32, a_vec, K, rows;
  uint32_t *tops;
  uint32_t *clear;  // words to clear
  int n_clear;
};
__global__ void __launch_bounds__(kPrepThreads) prep_kernel(const PrepArgs a) {
  extern __shared__ __align__(16) int prep_smem[];
  __shared__ uint32_t scratch[kPrepWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = a.M * a.top_k;
  const SlotLists L = slot_lists(prep_smem, P, a.E);
  if (blockIdx.x == 0) clear_lists(L, a.E);
  grid_dependency_wait();
  grid_dependents_launch();
  if (blockIdx.x > 0) {
    if (blockIdx.x == 1)
      for (int i = threadIdx.x; i < a.n_clear; i += kPrepThreads) a.clear[i] = 0;
    const int64_t row = blockIdx.x - 1;
    const uint32_t top = row_top(a.A, a.a_f32, a.a_vec, row, a.K, scratch);
    if (threadIdx.x == 0) a.tops[row] = top;
    return;
  }
  if (a.logits) {
    uint32_t *keys = reinterpret_cast<uint32_t *>(prep_smem + slot_lists_ints(P, a.E)) + warp * a.E;
#pragma unroll 1
    for (int m = warp; m < a.M; m += kPrepWarps) {
      int e;
      float r;
      route_row(a.logits, a.logits_f32, m, a.E, a.top_k, a.normalize, keys, e, r);
      if (lane < a.top_k) {
        const int q = m * a.top_k + lane;
        a.experts[q] = e;
        a.weights[q] = r;
        L.e[q] = e < 0 ? a.E : e;
      }
    }
  } else {
    for (int i = threadIdx.x; i < P; i += kPrepThreads) {
      const int e = a.table[i];
      L.e[i] = e >= 0 && e < a.E ? e : a.E;
    }
  }
  __syncthreads();
  build_lists(L, P, a.E, a.gt_log2);
#pragma unroll 1
  for (int i = threadIdx.x; i <= a.E; i += kPrepThreads) a.offsets[i] = L.off[i];
#pragma unroll 1
  for (int i = threadIdx.x; i < P; i += kPrepThreads) a.order[i] = L.order[i];
  if (a.groups) {
#pragma unroll 1
    for (int i = threadIdx.x; i < *L.ngrp; i += kPrepThreads) a.groups[i] = L.grp[i];
    if (threadIdx.x == 0) *a.n_groups = *L.ngrp;
  }
}

// The row magnitudes of many rows, and cleared words.
__global__ void __launch_bounds__(kThreads)
    row_tops_kernel(const void *A, bool f32, bool vec, int64_t rows, int K, uint32_t *tops,
                    uint32_t *clear, int64_t n_clear) {
  __shared__ uint32_t scratch[kWarps];
  grid_dependency_wait();
  grid_dependents_launch();
  for (int64_t i = blockIdx.x * int64_t(kThreads) + threadIdx.x; i < n_clear;
       i += int64_t(gridDim.x) * kThreads)
    clear[i] = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const uint32_t top = row_top(A, f32, vec, row, K, scratch);
    if (threadIdx.x == 0) tops[row] = top;
    __syncthreads();
  }
}

// ---- many slots, bf16: lists over several blocks, fp16 rows, scales ----------

// Slots by expert over many blocks of kSortSlots slots: a stable counting
// sort. First launch: each block's slots per expert, [blocks][E + 1] (slots
// without an expert count as expert E).
constexpr int kSortSlots = 1024;
__global__ void __launch_bounds__(kThreads)
    count_kernel(const int32_t *experts, int64_t P, int E, int32_t *counts) {
  extern __shared__ int32_t cnt[];  // [E + 1]
  for (int i = threadIdx.x; i <= E; i += kThreads) cnt[i] = 0;
  grid_dependency_wait();
  grid_dependents_launch();
  __syncthreads();
  const int64_t lo = int64_t(blockIdx.x) * kSortSlots;
  const int n = static_cast<int>(P - lo < kSortSlots ? P - lo : kSortSlots);
#pragma unroll
  for (int i = threadIdx.x; i < kSortSlots; i += kThreads)
    if (i < n) {
      const int e = experts[lo + i];
      atomicAdd(cnt + (e >= 0 && e < E ? e : E), 1);
    }
  __syncthreads();
  for (int i = threadIdx.x; i <= E; i += kThreads) counts[int64_t(blockIdx.x) * (E + 1) + i] = cnt[i];
}

// Slots per group of an expert's c slots: as even as whole runs of `unit` let
// them be, at most gt (a multiple of unit).
__device__ __forceinline__ int group_size(int c, int gt, int unit) {
  const int n = (c + gt - 1) / gt;
  return n ? (c + unit * n - 1) / (unit * n) * unit : gt;
}

// Between them, for many blocks: each expert's counts become sums over the
// blocks before, in place, and row `blocks` the sum of all. A block for 32
// experts, each warp a run of the rows.
__global__ void __launch_bounds__(1024) scan_counts_kernel(int32_t *counts, int64_t blocks, int E) {
  __shared__ int32_t sums[32][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.x * 32 + lane;
  const int64_t lo = blocks * warp / 32, hi = blocks * (warp + 1) / 32;
  grid_dependency_wait();
  grid_dependents_launch();
  int32_t *c = counts + e;
  int sum = 0;
  if (e <= E) {
#pragma unroll 8
    for (int64_t b = lo; b < hi; ++b) sum += c[b * (E + 1)];
  }
  sums[warp][lane] = sum;
  __syncthreads();
  int at = 0;
  for (int w = 0; w < warp; ++w) at += sums[w][lane];
  if (e > E) return;
  for (int64_t b0 = lo; b0 < hi; b0 += 8) {
    int v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = b0 + q < hi ? c[(b0 + q) * (E + 1)] : 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (b0 + q < hi) c[(b0 + q) * (E + 1)] = at;
      at += v[q];
    }
  }
  if (warp == 31) c[blocks * (E + 1)] = at;
}

// Last launch: places. Each block learns how many slots of each expert stand
// before it and in all (from scan_counts_kernel, or by adding up the counts),
// scans the experts, and places its slots in order; block 0 writes the offsets
// and the groups. place[p]: where slot p stands in the order, counting from 0;
// slots without an expert come last. Blocks of 2048 slots are slower for 3000
// slots (router and lists 9.1 us against 7.4).
constexpr int kPlaceThreads = 512;
constexpr int kPlaceWarps = kPlaceThreads / 32;
__global__ void __launch_bounds__(kPlaceThreads)
    place_kernel(const int32_t *experts, int64_t P, int E, const int32_t *counts, bool scanned,
                 int32_t *offsets, int32_t *order, int32_t *place, SlotGroup *groups,
                 int32_t *n_groups, int gt, int unit) {
  extern __shared__ int32_t mem[];
  int32_t *start = mem, *gstart = mem + E + 1;  // [E + 1] each
  int32_t *cnt = mem + 2 * (E + 1);             // [kPlaceWarps][E + 1]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kPlaceWarps * (E + 1); i += kPlaceThreads) cnt[i] = 0;
  for (int i = threadIdx.x; i < 2 * (E + 1); i += kPlaceThreads) mem[i] = 0;
  grid_dependency_wait();
  grid_dependents_launch();
  constexpr int kPer = kSortSlots / kPlaceWarps, kEach = kPer / 32;
  const int64_t lo = int64_t(blockIdx.x) * kSortSlots + warp * kPer + lane;
  int key[kEach];  // experts of the warp's slots, 32 at a time; -1: past the end
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    key[i] = -1;
    if (lo + 32 * i < P) {
      const int e = experts[lo + 32 * i];
      key[i] = e >= 0 && e < E ? e : E;
    }
  }
  __syncthreads();
  int32_t *mine = cnt + warp * (E + 1);
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (key[i] >= 0) atomicAdd(mine + key[i], 1);
  // Totals, and the part of them in the blocks before (gstart until the scan):
  // read, or added up by all threads, a few blocks' counts of an expert each.
  if (scanned) {
    for (int e = threadIdx.x; e <= E; e += kPlaceThreads) {
      start[e] = counts[int64_t(gridDim.x) * (E + 1) + e];
      gstart[e] = counts[int64_t(blockIdx.x) * (E + 1) + e];
    }
  } else {
    for (int i = threadIdx.x; i < (E + 1) * kPlaceWarps; i += kPlaceThreads) {
      const int e = i % (E + 1);
      int all = 0, before = 0;
#pragma unroll 4
      for (int b = i / (E + 1); b < gridDim.x; b += kPlaceWarps) {
        const int c = counts[int64_t(b) * (E + 1) + e];
        all += c;
        if (b < blockIdx.x) before += c;
      }
      if (all) {
        atomicAdd(start + e, all);
        if (before) atomicAdd(gstart + e, before);
      }
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += kPlaceThreads) {
    int before = gstart[e];
    for (int w = 0; w < kPlaceWarps; ++w) {  // where each warp's first slot goes, less start
      const int c = cnt[w * (E + 1) + e];
      cnt[w * (E + 1) + e] = before;
      before += c;
    }
    const int all = start[e], size = group_size(all, gt, unit);
    gstart[e] = e < E ? (all + size - 1) / size : 0;
  }
  __syncthreads();
  if (warp < 2) {  // exclusive prefixes over the experts: slots, groups
    int32_t *v = warp ? gstart : start;
    int base = 0;
    for (int i = lane; i - lane <= E; i += 32) {
      const int own = i <= E ? v[i] : 0;
      int x = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (i <= E) v[i] = base + x - own;
      base += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e <= E; e += kPlaceThreads) {
      offsets[e] = start[e];
      if (groups && e < E) {
        const int first = start[e], c = start[e + 1] - first, n = gstart[e + 1] - gstart[e];
        SlotGroup *g = groups + gstart[e];
        const int size = group_size(c, gt, unit);
        for (int k = 0; k < n; ++k)
          g[k] = SlotGroup{e, first + k * size, min(size, c - k * size)};
      }
    }
    if (groups && threadIdx.x == 0) *n_groups = gstart[E];
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const unsigned same = __match_any_sync(0xffffffffu, key[i]);
    const int rank = __popc(same & ((1u << lane) - 1));
    if (key[i] >= 0) {
      const int at = start[key[i]] + mine[key[i]] + rank;
      order[at] = static_cast<int32_t>(lo + 32 * i);
      if (place) place[lo + 32 * i] = at;
    }
    __syncwarp();
    if (key[i] >= 0 && rank == 0) mine[key[i]] += __popc(same);
    __syncwarp();
  }
}

// bf16 activation rows as fp16, one copy for each routed slot, at the slot's
// place: row m of A [M, K] for slots m * copies .. (copies = top_k, or 1
// with a row per slot). A block per row. Also per place: what undoes the
// row's scale. Rows of Y of slots without an expert are cleared (Y given).
// Bound by the copies' writes: 4096 rows of 2560, 8 copies, 189 MB in 30 us =
// 6.3 TB/s. (Copies, so that a group's rows are one TMA tile: a gather by row
// would issue 8 times as many.)
struct ConvertArgs {
  const uint16_t *A;
  int a_vec, K, Kp, copies;
  const int32_t *place, *offsets;
  int E;
  uint16_t *out;
  float *unscale;
  uint16_t *Y;
  int N;
};
// A block of about a thread per 8 columns, for either kernel of rows.
int row_threads(int64_t n) {
  return static_cast<int>(std::min<int64_t>(1024, ceil_div(ceil_div(n, 8), 32) * 32));
}
// The largest of the threads' values, by a block of up to 1024.
__device__ __forceinline__ uint32_t block_max(uint32_t top, uint32_t (&scratch)[32]) {
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = top;
  __syncthreads();
  for (int w = 0; w < blockDim.x >> 5; ++w) top = max(top, scratch[w]);
  return top;
}
__device__ __forceinline__ uint32_t top_of(const float (&v)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) top = max(top, __float_as_uint(v[q]) & 0x7FFFFFFFu);
  return top;
}
__device__ __forceinline__ uint4 half8(const float (&v)[8], float f) {
  return make_uint4(pack_f16x2(v[0] * f, v[1] * f), pack_f16x2(v[2] * f, v[3] * f),
                    pack_f16x2(v[4] * f, v[5] * f), pack_f16x2(v[6] * f, v[7] * f));
}
__global__ void __launch_bounds__(1024) convert_kernel(const ConvertArgs a) {
  __shared__ uint32_t tops[32];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int64_t m = blockIdx.x;
  grid_dependency_wait();
  grid_dependents_launch();
  const int routed = a.offsets[a.E];
  uint32_t top = 0;
  for (int k = tid * 8; k < a.Kp; k += threads * 8) {
    float v[8];
    load8(a.A, false, a.a_vec, m * a.K, k, a.K, v);
    top = max(top, top_of(v));
  }
  const int shift = row_shift(block_max(top, tops));
  const float f = exp2i(shift);
  for (int j = 0; j < a.copies; ++j) {
    const int64_t slot = m * a.copies + j;
    const int at = a.place[slot];
    if (at < routed) {
      if (tid == 0) a.unscale[at] = exp2i(-shift);
    } else if (a.Y) {
      for (int n = tid; n < a.N; n += threads) a.Y[slot * a.N + n] = 0;
    }
  }
  for (int k = tid * 8; k < a.Kp; k += threads * 8) {
    float v[8];
    load8(a.A, false, a.a_vec, m * a.K, k, a.K, v);
    const uint4 h = half8(v, f);
    for (int j = 0; j < a.copies; ++j) {
      const int at = a.place[m * a.copies + j];
      if (at < routed) *reinterpret_cast<uint4 *>(a.out + int64_t(at) * a.Kp + k) = h;
    }
  }
}

// Hidden rows [places, ld] in fp32 as fp16 rows [places, Kp], zeros past K, each
// scaled by its own largest value; what undoes the scale, and its exponent
// (126, the largest, for a row of zeros). A block per place. Bound by its
// loads' latency: 32 768 rows of 768, 151 MB in 35 us = 4.3 TB/s.
__global__ void __launch_bounds__(1024)
    hidden_half_kernel(const float *hidden, int64_t ld, int K, int Kp, const int32_t *offsets,
                       int E, uint16_t *out, float *unscale, int32_t *shifts) {
  __shared__ uint32_t tops[32];
  const int tid = threadIdx.x, step = blockDim.x * 8;
  const int64_t at = blockIdx.x;
  grid_dependency_wait();
  grid_dependents_launch();
  if (at >= offsets[E]) return;
  float v[8], u[8];  // (most rows are one step long: they are read once)
  load8(hidden, true, true, at * ld, tid * 8, K, v);
  uint32_t top = top_of(v);
  for (int k = tid * 8 + step; k < K; k += step) {
    load8(hidden, true, true, at * ld, k, K, u);
    top = max(top, top_of(u));
  }
  top = block_max(top, tops);
  const int shift = top ? row_shift(top) : 126;
  const float f = exp2i(shift);
  if (tid == 0) {
    unscale[at] = exp2i(-shift);
    shifts[at] = shift;
  }
  uint16_t *dst = out + at * Kp;
  if (tid * 8 < Kp) *reinterpret_cast<uint4 *>(dst + tid * 8) = half8(v, f);
  for (int k = tid * 8 + step; k < Kp; k += step) {
    load8(hidden, true, true, at * ld, k, K, u);
    *reinterpret_cast<uint4 *>(dst + k) = half8(u, f);
  }
}

// Largest |bias| of each expert.
__global__ void __launch_bounds__(kThreads)
    bias_max_kernel(const float *bias, int N, float *bmax) {
  __shared__ uint32_t scratch[32];
  const int e = blockIdx.x;
  grid_dependency_wait();
  grid_dependents_launch();
  uint32_t top = 0;
  for (int n = threadIdx.x; n < N; n += kThreads)
    top = max(top, __float_as_uint(bias[int64_t(e) * N + n]) & 0x7FFFFFFFu);
  top = block_max(top, scratch);
  if (threadIdx.x == 0) bmax[e] = __uint_as_float(top);
}

// Sum of each token's fp16 partials (rows of ld, a multiple of 8), in slot
// order. Bound by reading them: 4096 tokens of 8 partials of 2560, 189 MB in
// 35 us = 5.4 TB/s.
__global__ void __launch_bounds__(1024)
    combine_half_kernel(const uint16_t *part, int64_t ld, const float *unscale,
                        const int32_t *place, const int32_t *offsets, int E, int64_t M, int top_k,
                        int N, uint16_t *Y) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int routed = offsets[E];
  const int64_t m = blockIdx.x;
  const bool yvec = N % 8 == 0 && reinterpret_cast<uintptr_t>(Y) % 16 == 0;
  for (int n = threadIdx.x * 8; n < N; n += blockDim.x * 8) {
    float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int j = 0; j < top_k; ++j) {
      const int at = place[m * top_k + j];
      if (at >= routed) continue;
      const float f = unscale[at];
      const uint4 x = *reinterpret_cast<const uint4 *>(part + int64_t(at) * ld + n);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[q]));
        y[2 * q] = fmaf(v.x, f, y[2 * q]);
        y[2 * q + 1] = fmaf(v.y, f, y[2 * q + 1]);
      }
    }
    uint16_t *dst = Y + m * N + n;
    if (yvec) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = bf16_bits(y[2 * q]) | (bf16_bits(y[2 * q + 1]) << 16);
      *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      for (int q = 0; q < 8; ++q)
        if (n + q < N) dst[q] = static_cast<uint16_t>(bf16_bits(y[q]));
    }
  }
}

// Sum of each token's fp32 partials, in slot order: a block per token, eight
// slots' loads at a time.
__global__ void __launch_bounds__(1024)
    combine_kernel(const float *part, const int32_t *experts, int top_k, int N, void *Y,
                   bool f32) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t m = blockIdx.x, q0 = m * top_k;
  const bool vec = N % 4 == 0;  // rows of partials start on 16 bytes
  for (int n = threadIdx.x * 4; n < N; n += blockDim.x * 4) {
    float y[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < top_k; j0 += 8) {
      float v[8][4];
      bool some[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        some[j] = j0 + j < top_k && experts[q0 + j0 + j] >= 0;
        if (j0 + j >= top_k) continue;
        const float *src = part + (q0 + j0 + j) * N + n;
        if (vec) {
          const float4 x = *reinterpret_cast<const float4 *>(src);
          v[j][0] = x.x; v[j][1] = x.y; v[j][2] = x.z; v[j][3] = x.w;
        } else {
#pragma unroll
          for (int o = 0; o < 4; ++o) v[j][o] = n + o < N ? src[o] : 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (some[j])
#pragma unroll
          for (int o = 0; o < 4; ++o) y[o] += v[j][o];
    }
#pragma unroll
    for (int o = 0; o < 4; ++o)
      if (n + o < N) store_f(Y, f32, m * N + n + o, y[o]);
  }
}

template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, int block, size_t smem, bool pdl,
                       cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

cudaError_t launch_prepack_experts(const ExpertPackArgs &a, cudaStream_t stream) {
  const int64_t nb = ceil_div(a.K, a.bs), nbz = ceil_div(nb, 2) * 2;
  const int64_t Np = ceil_div(a.N, kTileN) * kTileN, tiles = a.E * Np / kTileN;
  const int64_t K64 = ceil_div(a.K, kChunkK), words = tiles * K64 * (kChunkBytes / 4);
  pack_expert_codes_kernel<<<grid_of(words, 256), 256, 0, stream>>>(
      a.B, static_cast<uint32_t *>(a.packed_b), a.N, Np, a.K, a.bs, nb, K64, words);
  const int64_t ns = tiles * nb * kTileN;
  if (a.scale_f32)
    pack_expert_scales_kernel<float><<<grid_of(ns, 256), 256, 0, stream>>>(
        static_cast<const float *>(a.scales), static_cast<float *>(a.packed_scales), a.N, Np, nb,
        ns);
  else
    pack_expert_scales_kernel<uint16_t><<<grid_of(ns, 256), 256, 0, stream>>>(
        static_cast<const uint16_t *>(a.scales), static_cast<uint16_t *>(a.packed_scales), a.N,
        Np, nb, ns);
  if (a.zp)
    pack_expert_zp_kernel<<<grid_of(tiles * nbz, 256), 256, 0, stream>>>(
        a.zp, static_cast<uint64_t *>(a.packed_zp), a.N, Np, nb, nbz, tiles * nbz);
  uint32_t *smax = reinterpret_cast<uint32_t *>(a.packed_rows + a.E * Np);
  const cudaError_t e = cudaMemsetAsync(smax, 0, size_t(a.E) * 4, stream);
  if (e != cudaSuccess) return e;
  if (a.scale_f32)
    row_scales_kernel<float><<<grid_of(tiles, kWarps), kThreads, 0, stream>>>(
        static_cast<const float *>(a.packed_scales), a.packed_rows, smax, a.E, Np / kTileN, nb);
  else
    row_scales_kernel<uint16_t><<<grid_of(tiles, kWarps), kThreads, 0, stream>>>(
        static_cast<const uint16_t *>(a.packed_scales), a.packed_rows, smax, a.E, Np / kTileN, nb);
  return cudaGetLastError();
}


namespace {

int ilog2(int x) {
  int r = 0;
  while ((1 << r) < x) ++r;
  return r;
}

// Shared memory of a weight-streaming CTA: stage layout, and bytes of its
// parts for groups of gt slots.
struct StreamSmem {
  int st_scale, st_zp, st_tile;
  int64_t krow, sums, ring, terms;
  int64_t red(int gt) const { return int64_t(2 * 2 * 8 * kTileN * 4) * gt; }
  int64_t bytes(int gt) const {
    return red(gt) + sums + ring + ceil_div(terms * gt * krow * 2, 128) * 128;
  }
};
StreamSmem stream_smem(const ExpertStack &w, int terms) {
  StreamSmem s{};
  const int es = w.s_f32 ? 4 : 2;
  const int64_t K64 = ceil_div(w.K, kChunkK);
  // Scale blocks a stage can touch (blocks of up to 64 codes lie inside chunks).
  const int nblk = w.bs <= kChunkK ? kStreamChunks * kChunkK / w.bs
                                   : (kStreamChunks * kChunkK - 1) / w.bs + 2;
  s.st_scale = kStreamChunks * kChunkBytes;
  s.st_zp = s.st_scale + nblk * kTileN * es;
  s.st_tile = s.st_zp + (w.z ? (nblk / 2 + 1) * 16 : 0);
  s.krow = K64 * kChunkK + 16;
  s.sums = terms == 1 ? K64 * std::max(1, kChunkK / w.bs) * 64 : 0;
  s.ring = int64_t(8) * kStreamStages * 2 * s.st_tile;
  s.terms = terms;
  return s;
}
// Shared memory that lets n CTAs share an SM (1 KB of each is the system's).
int64_t stream_room(int n) { return 228 * 1024 / n - 1536; }
bool stream_fits(const ExpertStack &w, int terms) {
  return stream_smem(w, terms).bytes(1) <= stream_room(1);
}

// Fills the geometry of a weight-streaming launch. `per_expert`: the most
// slots an expert can have. false: not even one activation row fits.
struct StreamPlan {
  StreamParams p{};
  int terms = 1, grid = 1, smem = 0;
  bool zp = false, sf32 = false;
};
bool plan_stream(StreamPlan &pl, const ExpertStack &w, int mode, int terms, int64_t P,
                 int top_k, int64_t per_expert) {
  StreamParams &p = pl.p;
  pl.terms = terms;
  pl.zp = w.z != nullptr;
  pl.sf32 = w.s_f32;
  p.mode = mode;
  p.E = w.E;
  p.N = w.N;
  p.K = w.K;
  p.N16 = static_cast<int>(ceil_div(w.N, kTileN));
  p.K64 = static_cast<int>(ceil_div(w.K, kChunkK));
  p.nb = static_cast<int>(ceil_div(w.K, w.bs));
  p.nbz = (p.nb + 1) / 2 * 2;
  p.bs_log2 = ilog2(w.bs);
  p.npair = mode == kStreamGateUp ? p.N16 : (p.N16 + 1) / 2;
  p.P = static_cast<int>(P);
  p.top_k = top_k;
  // Warps per pair: what makes the longest run of work shortest, in chunks,
  // with the distinct experts that P random slots name; a step costs a warp
  // that has its pair to itself about five chunks more (it stores alone),
  // otherwise one and half a chunk per warp that meets. Measured on the layer
  // with 8 out of 128 experts, 2560 -> 768 -> 2560, this rule and 1, 2, 4 or 8
  // warps for both launches: 16 tokens 78.9 us against 86.1, 83.6, 83.6, 99.3;
  // one token 19.8 against 27.2, 21.6, 20.4, 21.0.
  const double E = w.E, distinct = E * (1 - std::pow(1 - 1 / E, double(P)));
  const int64_t groups = std::max<int64_t>(1, std::max<int64_t>(std::llround(distinct), P / 8));
  double best = 0;
  for (int ks = 1; ks <= 8 && ks <= p.K64; ks *= 2) {
    const int64_t steps = groups * ceil_div(p.npair, 8 / ks);
    const double cost = double(ceil_div(steps, kStreamCtas * sm_count())) *
                        (ceil_div(p.K64, ks) + (ks == 1 ? 5 : 1 + ks / 2));
    if (ks == 1 || cost < best) {
      best = cost;
      p.ksplit = ks;
    }
  }
  p.tpu = 8 / p.ksplit;
  p.tpu_log2 = ilog2(p.tpu);
  p.ns = static_cast<int>(ceil_div(p.npair, p.tpu));
  const StreamSmem sm = stream_smem(w, terms);
  p.st_scale = sm.st_scale;
  p.st_zp = sm.st_zp;
  p.st_tile = sm.st_tile;
  p.st_bytes = 2 * p.st_tile;
  // Slots per group: about twice the mean list, so that few experts need a
  // second pass over their weights, within what two CTAs per SM leave (one
  // CTA per SM when that is not enough for the mean).
  const int64_t mean = ceil_div(P, w.E);
  int want = 1;
  while (want < 8 && want < 2 * mean && want < per_expert) want *= 2;
  int gt = want;
  while (gt > 1 && sm.bytes(gt) > stream_room(kStreamCtas) && gt > mean) gt /= 2;
  while (gt > 1 && sm.bytes(gt) > stream_room(1)) gt /= 2;
  if (sm.bytes(gt) > stream_room(1)) return false;
  p.gt_log2 = ilog2(gt);
  p.krow = static_cast<int>(sm.krow);
  p.off_red = 0;
  p.off_sums = static_cast<int>(sm.red(gt));
  p.off_ring = static_cast<int>(p.off_sums + sm.sums);
  p.off_x = static_cast<int>(p.off_ring + sm.ring);
  pl.smem = static_cast<int>(sm.bytes(gt));
  int ctas = kStreamCtas;
  while (pl.smem > stream_room(ctas)) --ctas;
  const int64_t most = P * p.ns, slots = int64_t(sm_count()) * ctas;
  if (most > (int64_t(1) << 31) - 1) return false;
  pl.grid = static_cast<int>(std::min(most, slots));
  return true;
}

cudaError_t run_stream(const StreamPlan &pl, bool pdl, cudaStream_t stream) {
  const int bs = 1 << pl.p.bs_log2;
  auto *fn = bs == 16 ? launch_stream<1> : bs == 32 ? launch_stream<2> : launch_stream<4>;
  return fn(pl.p, pl.zp, pl.sf32, pl.terms, pl.grid, pl.smem, pdl, stream);
}

StreamMat stream_mat(const ExpertStack &w) {
  return StreamMat{static_cast<const uint4 *>(w.b), static_cast<const unsigned char *>(w.s),
                   static_cast<const unsigned char *>(w.z), w.bias};
}

bool vec_rows(const void *a, int64_t K, size_t es) {
  return reinterpret_cast<uintptr_t>(a) % 16 == 0 && K * es % 16 == 0;
}

// Carves a workspace into 256-byte aligned pieces; with a null base it only
// adds up the bytes.
struct Carve {
  unsigned char *base;
  size_t used = 0;
  template <typename T>
  T *take(size_t n) {
    T *r = base ? reinterpret_cast<T *>(base + used) : nullptr;
    used += align256(n * sizeof(T));
    return r;
  }
};

// The lists of many slots in global memory.
struct Lists {
  float *weights = nullptr;
  int32_t *experts = nullptr, *offsets = nullptr, *order = nullptr, *n_groups = nullptr;
  SlotGroup *groups = nullptr;
};

// Groups of P slots at most: every expert may leave one partly filled.
size_t max_groups(int64_t P, int E, int gt) {
  return static_cast<size_t>(std::min<int64_t>(P, P / gt + E));
}
// Counts (blocks times experts) from which on a launch of its own sums them.
// Fewer are added up by every block that places: a launch less, but work that
// grows with the square of the slots. Router and lists, 8 choices, us, added up
// by every block and by the launch:
//   experts    65 536 slots   131 072        262 144        4 M
//   64          10.9   12.9   15.9   16.8    23.3   22.8     668   266
//   128         13.0   14.1   19.4   18.5    29.5   25.8    1120   310
//   256         17.5   16.3   26.9   22.2    42.5   32.3    2041   406
//   1000        49.5   36.2   79.0   57.4   141.1   95.0    7769  1358
constexpr int64_t kScanCounts = 12288;
size_t count_words(int64_t P, int E) { return (ceil_div(P, kSortSlots) + 1) * (E + 1); }

// The lists of many slots: counts is workspace; place, and the groups of up to
// gt slots (sizes in whole `unit`s), when asked for.
cudaError_t launch_lists(const int32_t *experts, int64_t P, int E, const Lists &l,
                         int32_t *counts, int32_t *place, int gt, int unit, bool pdl,
                         cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};
  cudaError_t e =
      ensure_smem_limit(place_kernel, (2 + kPlaceWarps) * (kMoeMaxExperts + 1) * 4, done);
  if (e != cudaSuccess) return e;
  const unsigned blocks = static_cast<unsigned>(ceil_div(P, kSortSlots));
  e = launch_pdl(count_kernel, blocks, kThreads, size_t(E + 1) * 4, pdl, stream, experts, P, E,
                 counts);
  const bool scanned = int64_t(blocks) * (E + 1) >= kScanCounts;
  if (e == cudaSuccess && scanned)
    e = launch_pdl(scan_counts_kernel, static_cast<unsigned>(ceil_div(E + 1, 32)), 1024, 0, pdl,
                   stream, counts, blocks, E);
  if (e != cudaSuccess) return e;
  return launch_pdl(place_kernel, blocks, kPlaceThreads, size_t(2 + kPlaceWarps) * (E + 1) * 4,
                    pdl, stream, experts, P, E, counts, scanned, l.offsets, l.order, place, l.groups,
                    l.n_groups, gt, unit);
}

// Slots that one block lists by itself (prep_kernel); more take the router,
// the lists and the row magnitudes as kernels of their own. Router of 8 out of
// 128 experts, one block against the kernels, us: 128 slots 5.3 and 7.1, 256
// slots 7.1 both, 512 slots 11.5 and 7.5; the layer 2560 -> 768 -> 2560: 32
// slots 40.0 and 44.5, 256 slots 120.0 and 122.8.
constexpr int kFewSlots = 256;

Lists take_lists(Carve &c, int64_t P, int E, bool routed) {
  Lists l;
  if (routed) {
    l.weights = c.take<float>(P);
    l.experts = c.take<int32_t>(P);
  }
  l.offsets = c.take<int32_t>(E + 1);
  l.order = c.take<int32_t>(P);
  l.n_groups = c.take<int32_t>(1);
  l.groups = c.take<SlotGroup>(max_groups(P, E, 1));
  return l;
}

struct MoeSpace {
  Lists l;
  int32_t *counts;
  uint32_t *tops, *hidden_tops;
  float *hidden, *part;
  size_t bytes;
};
// fp32 hidden rows start on 16 bytes.
size_t hidden_ld(const ExpertStack &gate) { return ceil_div(gate.N, 4) * 4; }

MoeSpace moe_space(const MoeArgs &a) {
  const size_t P = size_t(a.M) * a.top_k;
  Carve c{a.ws};
  MoeSpace s{};
  s.l = take_lists(c, P, a.gate.E, true);
  s.counts = P > kFewSlots ? c.take<int32_t>(count_words(P, a.gate.E)) : nullptr;
  s.tops = c.take<uint32_t>(a.M);
  s.hidden_tops = c.take<uint32_t>(P);
  s.hidden = c.take<float>(P * hidden_ld(a.gate));
  s.part = c.take<float>(P * a.down.N);
  s.bytes = c.used;
  return s;
}

struct ExpertsSpace {
  Lists l;
  int32_t *counts;
  uint32_t *tops;
  size_t bytes;
};
ExpertsSpace experts_space(const ExpertsArgs &a) {
  const size_t P = size_t(a.M) * a.top_k;
  Carve c{a.ws};
  ExpertsSpace s{};
  s.l = take_lists(c, P, a.w.E, false);
  s.counts = P > kFewSlots ? c.take<int32_t>(count_words(P, a.w.E)) : nullptr;
  s.tops = c.take<uint32_t>(a.per_slot ? P : a.M);
  s.bytes = c.used;
  return s;
}

// ---- tensor-core path: bf16 activations, many slots ---------------------------

// From a mean of this many slots per expert on; fewer stream the weights past
// groups of up to 8 slots. The layer, blocks of 32, streaming and tensor-core
// path, us:
//   experts, top_k, H, I       mean 4          mean 6          mean 8
//   8, 2, 1024, 2048        25.3    33.8    29.7    34.2    32.3    34.3
//   16, 4, 1024, 512        17.2    26.0    22.5    26.3    25.7    26.9
//   32, 4, 2560, 1408       74.6    95.0    96.7    95.2   104.2    95.0
//   128, 8, 2560, 768      140.0   171.7   187.4   180.3   195.0   181.3
// A row too long for the streaming kernel's shared memory (K beyond 25 000 to
// 59 000, by block size and scale type) takes the tensor-core path as well.
constexpr int kTileMeanSlots = 6;
bool tile_path(bool a_f32, int64_t P, std::initializer_list<const ExpertStack *> w) {
  if (a_f32) return false;
  for (const ExpertStack *x : w)
    if (P >= int64_t(kTileMeanSlots) * x->E || !stream_fits(*x, 1)) return true;
  return false;
}

// Rows of partials start on 16 bytes.
int64_t part_ld(int64_t N) { return ceil_div(N, 8) * 8; }
int64_t k_pad(int64_t K) { return ceil_div(K, kChunkK) * kChunkK; }

struct TileSpace {
  Lists l;
  int32_t *counts, *place;
  uint16_t *rows;  // fp16 activations by place
  float *unscale;
  // The layer's. Each of two pieces is used twice: fp16 hidden rows take the
  // place of the activations, partials that of the fp32 hidden rows.
  float *hidden;
  uint16_t *hidden_rows, *part;
  float *h_unscale, *p_unscale;
  int32_t *h_shift;
  float *bmax;  // [E] of down, null without a bias
  size_t bytes;
};
// Of a product with w, or of the layer with gate = w and down.
TileSpace tile_space(unsigned char *ws, int64_t P, const ExpertStack &w, const ExpertStack *down) {
  Carve c{ws};
  TileSpace s{};
  const int E = w.E;
  const bool layer = down != nullptr;
  if (layer) {
    s.l.weights = c.take<float>(P);
    s.l.experts = c.take<int32_t>(P);
  }
  s.l.offsets = c.take<int32_t>(E + 1);
  s.l.order = c.take<int32_t>(P);
  s.l.n_groups = c.take<int32_t>(1);
  s.l.groups = c.take<SlotGroup>(max_groups(P, E, kTileSlots));
  s.counts = c.take<int32_t>(count_words(P, E));
  s.place = c.take<int32_t>(P);
  s.rows = c.take<uint16_t>(size_t(P) * std::max(k_pad(w.K), layer ? k_pad(down->K) : 0));
  s.unscale = c.take<float>(P);
  if (layer) {
    s.hidden_rows = s.rows;
    s.hidden = c.take<float>(size_t(P) *
                             std::max<size_t>(hidden_ld(w), ceil_div(part_ld(down->N), 2)));
    s.part = reinterpret_cast<uint16_t *>(s.hidden);
    s.h_unscale = c.take<float>(P);
    s.p_unscale = c.take<float>(P);
    s.h_shift = c.take<int32_t>(P);
    s.bmax = down->bias ? c.take<float>(E) : nullptr;
  }
  s.bytes = c.used;
  return s;
}

// w0 and w1: gate and up, or one matrix twice.
cudaError_t fill_tile(TileParams &p, int mode, const ExpertStack &w0, const ExpertStack &w1,
                      const TileSpace &s, const uint16_t *rows, int64_t P) {
  p.mode = mode;
  for (int m = 0; m < 2; ++m) {
    const ExpertStack &w = m ? w1 : w0;
    p.w[m] = stream_mat(w);
    p.ts[m] = TileScales{w.rows, w.rows + int64_t(w.E) * ceil_div(w.N, kTileN) * kTileN, s.bmax};
  }
  p.N = w0.N;
  p.N16 = static_cast<int>(ceil_div(w0.N, kTileN));
  p.K64 = static_cast<int>(ceil_div(w0.K, kChunkK));
  p.nb = static_cast<int>(ceil_div(w0.K, w0.bs));
  p.nbz = (p.nb + 1) / 2 * 2;
  p.ntile = static_cast<int>(ceil_div(w0.N, mode == kStreamGateUp ? 64 : 128));
  p.order = s.l.order;
  p.n_groups = s.l.n_groups;
  p.groups = s.l.groups;
  p.weights = s.l.weights;
  const uint64_t dims[2] = {static_cast<uint64_t>(p.K64) * kChunkK, static_cast<uint64_t>(P)};
  const uint64_t strides[1] = {dims[0] * 2};
  const uint32_t box[2] = {kChunkK, kTileBox};
  return make_tmap(&p.tmb, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, rows, dims, strides, box,
                   CU_TENSOR_MAP_SWIZZLE_128B);
}

cudaError_t launch_experts_tile(const ExpertsArgs &a, cudaStream_t stream) {
  const int64_t P = a.M * a.top_k;
  const TileSpace s = tile_space(a.ws, P, a.w, nullptr);
  cudaError_t e = launch_lists(a.experts, P, a.w.E, s.l, s.counts, s.place, kTileSlots, 16, a.pdl,
                               stream);
  if (e != cudaSuccess) return e;
  ConvertArgs c{};
  c.A = static_cast<const uint16_t *>(a.A);
  c.a_vec = vec_rows(a.A, a.w.K, 2);
  c.K = a.w.K;
  c.Kp = static_cast<int>(k_pad(a.w.K));
  c.copies = a.per_slot ? 1 : a.top_k;
  c.place = s.place;
  c.offsets = s.l.offsets;
  c.E = a.w.E;
  c.out = s.rows;
  c.unscale = s.unscale;
  c.Y = static_cast<uint16_t *>(a.Y);
  c.N = a.w.N;
  e = launch_pdl(convert_kernel, static_cast<unsigned>(a.per_slot ? P : a.M), row_threads(c.Kp), 0,
                 a.pdl, stream, c);
  if (e != cudaSuccess) return e;
  TileParams p{};
  e = fill_tile(p, kStreamProduct, a.w, a.w, s, s.rows, P);
  if (e != cudaSuccess) return e;
  p.unscale = s.unscale;
  p.Y = static_cast<uint16_t *>(a.Y);
  p.y_pairs = a.w.N % 2 == 0 && reinterpret_cast<uintptr_t>(a.Y) % 4 == 0;
  return launch_tile(p, a.w.z != nullptr, a.w.s_f32, a.w.bs, a.pdl, stream);
}

cudaError_t launch_moe_tile(const MoeArgs &a, cudaStream_t stream) {
  const int64_t P = a.M * a.top_k;
  const TileSpace s = tile_space(a.ws, P, a.gate, &a.down);
  cudaError_t e = launch_pdl(route_kernel, grid_of(a.M, kWarps), kThreads,
                             size_t(kWarps) * a.gate.E * 4, a.pdl, stream, a.logits,
                             a.logits_f32, a.M, a.gate.E, a.top_k, a.normalize, s.l.weights,
                             s.l.experts);
  if (e == cudaSuccess)
    e = launch_lists(s.l.experts, P, a.gate.E, s.l, s.counts, s.place, kTileSlots, 16, a.pdl,
                     stream);
  if (e == cudaSuccess && s.bmax)
    e = launch_pdl(bias_max_kernel, a.down.E, kThreads, 0, a.pdl, stream, a.down.bias, a.down.N,
                   s.bmax);
  if (e != cudaSuccess) return e;
  ConvertArgs c{};
  c.A = static_cast<const uint16_t *>(a.X);
  c.a_vec = vec_rows(a.X, a.gate.K, 2);
  c.K = a.gate.K;
  c.Kp = static_cast<int>(k_pad(a.gate.K));
  c.copies = a.top_k;
  c.place = s.place;
  c.offsets = s.l.offsets;
  c.E = a.gate.E;
  c.out = s.rows;
  c.unscale = s.unscale;
  e = launch_pdl(convert_kernel, static_cast<unsigned>(a.M), row_threads(c.Kp), 0, a.pdl, stream, c);
  if (e != cudaSuccess) return e;
  TileParams up{}, down{};
  e = fill_tile(up, kStreamGateUp, a.gate, a.up, s, s.rows, P);
  if (e != cudaSuccess) return e;
  up.unscale = s.unscale;
  up.hidden = s.hidden;
  up.ldh = hidden_ld(a.gate);
  e = launch_tile(up, a.gate.z != nullptr, a.gate.s_f32, a.gate.bs, a.pdl, stream);
  if (e != cudaSuccess) return e;
  const int Ip = static_cast<int>(k_pad(a.down.K));
  e = launch_pdl(hidden_half_kernel, static_cast<unsigned>(P), row_threads(Ip), 0, a.pdl, stream,
                 s.hidden, up.ldh, a.down.K, Ip, s.l.offsets, a.down.E, s.hidden_rows, s.h_unscale,
                 s.h_shift);
  if (e != cudaSuccess) return e;
  e = fill_tile(down, kStreamDown, a.down, a.down, s, s.hidden_rows, P);
  if (e != cudaSuccess) return e;
  down.unscale = s.h_unscale;
  down.shift = s.h_shift;
  down.part = s.part;
  down.ldp = part_ld(a.down.N);
  down.out_unscale = s.p_unscale;
  e = launch_tile(down, a.down.z != nullptr, a.down.s_f32, a.down.bs, a.pdl, stream);
  if (e != cudaSuccess) return e;
  return launch_pdl(combine_half_kernel, static_cast<unsigned>(a.M), row_threads(a.down.N), 0,
                    a.pdl, stream,
                    s.part, part_ld(a.down.N), s.p_unscale, s.place, s.l.offsets, a.gate.E, a.M, a.top_k, a.down.N,
                    static_cast<uint16_t *>(a.Y));
}

cudaError_t launch_prep(const PrepArgs &a, bool pdl, cudaStream_t stream) {
  const int P = a.M * a.top_k;
  // Keys in shared memory for more experts than registers hold.
  const size_t smem =
      size_t(slot_lists_ints(P, a.E) + (a.logits && a.E > 256 ? kPrepWarps * a.E : 0)) * 4;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = ensure_smem_limit(
      prep_kernel, (slot_lists_ints(kFewSlots, kMoeMaxExperts) + kPrepWarps * kMoeMaxExperts) * 4,
      done);
  if (e != cudaSuccess) return e;
  return launch_pdl(prep_kernel, 1 + a.rows, kPrepThreads, smem, pdl, stream, a);
}

cudaError_t launch_row_tops(const void *A, bool f32, bool vec, int64_t rows, int K,
                            uint32_t *tops, uint32_t *clear, int64_t n_clear, bool pdl,
                            cudaStream_t stream) {
  return launch_pdl(row_tops_kernel, grid_of(rows, 1), kThreads, 0, pdl, stream, A, f32, vec,
                    rows, K, tops, clear, n_clear);
}

void set_lists(StreamParams &p, const Lists &l) {
  p.offsets = l.offsets;
  p.order = l.order;
  p.n_groups = l.n_groups;
  p.groups = l.groups;
  p.weights = l.weights;
}

}  // namespace

size_t moe_route_workspace_bytes(int64_t M, int E, int top_k) {
  const int64_t P = M * top_k;
  return P > kFewSlots ? align256(count_words(P, E) * 4) : 0;
}

cudaError_t launch_moe_route(const RouteArgs &a, cudaStream_t stream) {
  const int64_t P = a.M * a.top_k;
  if (a.order && P <= kFewSlots) {
    PrepArgs r{};
    r.logits = a.logits;
    r.logits_f32 = a.logits_f32;
    r.normalize = a.normalize;
    r.M = static_cast<int>(a.M);
    r.E = a.E;
    r.top_k = a.top_k;
    r.weights = a.weights;
    r.experts = a.experts;
    r.offsets = a.offsets;
    r.order = a.order;
    return launch_prep(r, a.pdl, stream);
  }
  cudaError_t e = launch_pdl(route_kernel, grid_of(a.M, kWarps), kThreads,
                             size_t(kWarps) * a.E * 4, a.pdl, stream, a.logits, a.logits_f32,
                             a.M, a.E, a.top_k, a.normalize, a.weights, a.experts);
  if (e == cudaSuccess && a.order) {
    Lists l;
    l.offsets = a.offsets;
    l.order = a.order;
    e = launch_lists(a.experts, P, a.E, l, reinterpret_cast<int32_t *>(a.ws), nullptr, 1, 1,
                     a.pdl, stream);
  }
  return e;
}

size_t matmul_experts_workspace_bytes(const ExpertsArgs &a) {
  ExpertsArgs b = a;
  b.ws = nullptr;
  if (tile_path(a.a_f32, a.M * a.top_k, {&a.w}))
    return tile_space(nullptr, a.M * a.top_k, a.w, nullptr).bytes;
  return experts_space(b).bytes;
}

cudaError_t launch_matmul_experts(const ExpertsArgs &a, cudaStream_t stream) {
  const int64_t P = a.M * a.top_k, rows = a.per_slot ? P : a.M;
  if (tile_path(a.a_f32, P, {&a.w})) return launch_experts_tile(a, stream);
  StreamPlan pl;
  if (!plan_stream(pl, a.w, kStreamProduct, a.a_f32 ? 2 : 1, P, a.top_k, P))
    return cudaErrorNotSupported;
  const ExpertsSpace s = experts_space(a);
  const bool vec = vec_rows(a.A, a.w.K, a.a_f32 ? 4 : 2);
  cudaError_t e;
  if (P <= kFewSlots) {
    PrepArgs r{};
    r.table = a.experts;
    r.M = static_cast<int>(a.M);
    r.E = a.w.E;
    r.top_k = a.top_k;
    r.gt_log2 = pl.p.gt_log2;
    r.offsets = s.l.offsets;
    r.order = s.l.order;
    r.n_groups = s.l.n_groups;
    r.groups = s.l.groups;
    r.A = a.A;
    r.a_f32 = a.a_f32;
    r.a_vec = vec;
    r.K = a.w.K;
    r.rows = static_cast<int>(rows);
    r.tops = s.tops;
    e = launch_prep(r, a.pdl, stream);
  } else {
    e = launch_lists(a.experts, P, a.w.E, s.l, s.counts, nullptr, 1 << pl.p.gt_log2, 1, a.pdl, stream);
    if (e == cudaSuccess)
      e = launch_row_tops(a.A, a.a_f32, vec, rows, a.w.K, s.tops, nullptr, 0, a.pdl, stream);
  }
  if (e != cudaSuccess) return e;
  StreamParams &p = pl.p;
  set_lists(p, s.l);
  p.w[0] = p.w[1] = stream_mat(a.w);
  p.A = a.A;
  p.a_vec = vec;
  p.a_f32 = a.a_f32;
  p.per_slot = a.per_slot;
  p.ld = a.w.K;
  p.tops = s.tops;
  p.Y = a.Y;
  p.y_f32 = a.a_f32;
  return run_stream(pl, a.pdl, stream);
}

size_t moe_workspace_bytes(const MoeArgs &a) {
  MoeArgs b = a;
  b.ws = nullptr;
  if (tile_path(a.a_f32, a.M * a.top_k, {&a.gate, &a.down}))
    return tile_space(nullptr, a.M * a.top_k, a.gate, &a.down).bytes;
  return moe_space(b).bytes;
}

cudaError_t launch_moe(const MoeArgs &a, cudaStream_t stream) {
  const int64_t P = a.M * a.top_k;
  const bool few = P <= kFewSlots;
  if (tile_path(a.a_f32, P, {&a.gate, &a.down})) return launch_moe_tile(a, stream);
  const MoeSpace s = moe_space(a);
  StreamPlan up, down;
  const int terms = a.a_f32 ? 2 : 1;
  if (!plan_stream(up, a.gate, kStreamGateUp, terms, P, a.top_k, a.M) ||
      !plan_stream(down, a.down, kStreamDown, terms, P, a.top_k, a.M))
    return cudaErrorNotSupported;
  // Both launches use the lists: groups of the size that fits both.
  up.p.gt_log2 = down.p.gt_log2 = std::min(up.p.gt_log2, down.p.gt_log2);
  const bool vec = vec_rows(a.X, a.gate.K, a.a_f32 ? 4 : 2);
  cudaError_t e;
  if (few) {
    PrepArgs r{};
    r.logits = a.logits;
    r.logits_f32 = a.logits_f32;
    r.normalize = a.normalize;
    r.M = static_cast<int>(a.M);
    r.E = a.gate.E;
    r.top_k = a.top_k;
    r.gt_log2 = up.p.gt_log2;
    r.weights = s.l.weights;
    r.experts = s.l.experts;
    r.offsets = s.l.offsets;
    r.order = s.l.order;
    r.n_groups = s.l.n_groups;
    r.groups = s.l.groups;
    r.A = a.X;
    r.a_f32 = a.a_f32;
    r.a_vec = vec;
    r.K = a.gate.K;
    r.rows = static_cast<int>(a.M);
    r.tops = s.tops;
    r.clear = s.hidden_tops;
    r.n_clear = static_cast<int>(P);
    e = launch_prep(r, a.pdl, stream);
  } else {
    const RouteArgs r{a.logits, a.logits_f32, a.M, a.gate.E, a.top_k, a.normalize, s.l.weights,
                      s.l.experts, nullptr, nullptr, nullptr, a.pdl};
    e = launch_moe_route(r, stream);
    if (e == cudaSuccess)
      e = launch_lists(s.l.experts, P, a.gate.E, s.l, s.counts, nullptr, 1 << up.p.gt_log2, 1, a.pdl, stream);
    if (e == cudaSuccess)
      e = launch_row_tops(a.X, a.a_f32, vec, a.M, a.gate.K, s.tops, s.hidden_tops, P, a.pdl, stream);
  }
  if (e != cudaSuccess) return e;
  set_lists(up.p, s.l);
  up.p.w[0] = stream_mat(a.gate);
  up.p.w[1] = stream_mat(a.up);
  up.p.A = a.X;
  up.p.a_vec = vec;
  up.p.a_f32 = a.a_f32;
  up.p.ld = a.gate.K;
  up.p.tops = s.tops;
  up.p.hidden = s.hidden;
  up.p.hidden_tops = s.hidden_tops;
  up.p.ldh = hidden_ld(a.gate);
  e = run_stream(up, a.pdl, stream);
  if (e != cudaSuccess) return e;
  set_lists(down.p, s.l);
  down.p.w[0] = down.p.w[1] = stream_mat(a.down);
  down.p.A = s.hidden;
  down.p.a_f32 = down.p.a_vec = down.p.per_slot = 1;
  down.p.ld = hidden_ld(a.gate);
  down.p.tops = s.hidden_tops;
  down.p.part = s.part;
  down.p.early = a.pdl;
  e = run_stream(down, a.pdl, stream);
  if (e != cudaSuccess) return e;
  const int threads =
      static_cast<int>(std::min<int64_t>(1024, ceil_div(ceil_div(a.down.N, 4), 32) * 32));
  return launch_pdl(combine_kernel, static_cast<unsigned>(a.M), threads, 0, a.pdl, stream, s.part,
                    s.l.experts, a.top_k, a.down.N, a.Y, a.a_f32);
}

}  // namespace mnb
