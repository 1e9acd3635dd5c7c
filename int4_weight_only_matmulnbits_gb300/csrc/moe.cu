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

#include "mnb_common.cuh"
#include "mnb_launch.h"
#include "moe.h"
#include "moe_route.cuh"

namespace mnb {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

__device__ __forceinline__ float load_f(const void *p, bool f32, int64_t i) {
  return f32 ? static_cast<const float *>(p)[i]
             : bf16_bits_to_f32(static_cast<const uint16_t *>(p)[i]);
}
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

// Slots by expert (one block): a stable counting sort. Each warp owns a
// contiguous range of slots and a row of counters; slots without an expert
// count as expert E.
constexpr int kListWarps = 16;
__global__ void __launch_bounds__(kListWarps * 32)
    lists_kernel(const int32_t *experts, int64_t P, int E, int32_t *offsets, int32_t *order) {
  extern __shared__ int32_t cnt[];  // [kListWarps][E + 1], then [E + 1]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t *mine = cnt + warp * (E + 1), *start = cnt + kListWarps * (E + 1);
  for (int i = threadIdx.x; i < kListWarps * (E + 1); i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  const int64_t per = ceil_div(P, kListWarps), lo = warp * per, hi = lo + per < P ? lo + per : P;
  auto key_of = [&](int64_t p) {
    const int e = experts[p];
    return e >= 0 && e < E ? e : E;
  };
  for (int64_t p = lo + lane; p < hi; p += 32) atomicAdd(mine + key_of(p), 1);
  __syncthreads();
  // Per expert: exclusive prefix over the warps; the totals go to start.
  for (int e = threadIdx.x; e <= E; e += blockDim.x) {
    int sum = 0;
    for (int w = 0; w < kListWarps; ++w) {
      const int c = cnt[w * (E + 1) + e];
      cnt[w * (E + 1) + e] = sum;
      sum += c;
    }
    start[e] = sum;
  }
  __syncthreads();
  if (warp == 0) {  // exclusive prefix over the experts
    int base = 0;
    for (int i = 0; i <= E; i += 32) {
      const int v = i + lane <= E ? start[i + lane] : 0;
      int x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (i + lane <= E) {
        start[i + lane] = base + x - v;
        offsets[i + lane] = base + x - v;
      }
      base += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
  for (int64_t p0 = lo; p0 < hi; p0 += 32) {
    const int64_t p = p0 + lane;
    const bool ok = p < hi;
    const int e = ok ? key_of(p) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const int rank = __popc(same & ((1u << lane) - 1));
    if (ok) order[start[e] + mine[e] + rank] = static_cast<int32_t>(p);
    __syncwarp();
    if (ok && rank == 0) mine[e] += __popc(same);
    __syncwarp();
  }
}

// ---- products ---------------------------------------------------------------------

// One warp forms one 16-row tile of one slot: lane (g, t) holds rows g and
// g + 8 and, of every 16 k, the elements 4t .. 4t+3 of the packed word.
__device__ __forceinline__ void tile_dot(const ExpertStack &w, int64_t tile, const void *a,
                                         bool a_f32, int64_t a0, float (&acc)[2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int K64 = static_cast<int>(ceil_div(w.K, kChunkK));
  const int64_t nb = ceil_div(w.K, w.bs), nbz = ceil_div(nb, 2) * 2;
  acc[0] = acc[1] = 0.f;
  for (int c = 0; c < K64; ++c) {
    const uint4 v = reinterpret_cast<const uint4 *>(w.b)[(tile * K64 + c) * 32 + lane];
    const uint32_t words[4] = {v.x, v.y, v.z, v.w};
    for (int j = 0; j < 4; ++j) {
      const int k0 = c * kChunkK + 16 * j + 4 * t;
      if (k0 >= w.K) break;
      const int64_t b = k0 / w.bs;
      float d[2] = {0.f, 0.f};
      uint64_t zw = 0x8888888888888888ull;
      if (w.z) zw = static_cast<const uint64_t *>(w.z)[tile * nbz + b];
      for (int o = 0; o < 4 && k0 + o < w.K; ++o) {
        const float x = load_f(a, a_f32, a0 + k0 + o);
        for (int h = 0; h < 2; ++h) {
          const int q = (words[j] >> code_shift(o, h)) & 15;
          const int z = static_cast<int>(zw >> (4 * (g + 8 * h))) & 15;
          d[h] = fmaf(static_cast<float>(q - z), x, d[h]);
        }
      }
      for (int h = 0; h < 2; ++h)
        acc[h] = fmaf(load_f(w.s, w.s_f32, (tile * nb + b) * kTileN + g + 8 * h), d[h], acc[h]);
    }
  }
  for (int h = 0; h < 2; ++h) {
    acc[h] += __shfl_xor_sync(0xffffffffu, acc[h], 1);
    acc[h] += __shfl_xor_sync(0xffffffffu, acc[h], 2);
  }
}

__global__ void __launch_bounds__(kThreads) product_kernel(ExpertsArgs a) {
  const int lane = threadIdx.x & 31, g = lane >> 2;
  const int64_t N16 = ceil_div(a.w.N, kTileN), items = a.M * a.top_k * N16;
  for (int64_t it = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; it < items;
       it += ((int64_t)gridDim.x * blockDim.x) >> 5) {
    const int64_t p = it / N16, nt = it % N16;
    const int e = a.experts[p];
    const bool some = e >= 0 && e < a.w.E;
    float acc[2] = {0.f, 0.f};
    if (some)
      tile_dot(a.w, e * N16 + nt, a.A, a.a_f32, (a.per_slot ? p : p / a.top_k) * a.w.K, acc);
    for (int h = 0; h < 2; ++h) {
      const int64_t n = nt * kTileN + g + 8 * h;
      if ((lane & 3) || n >= a.w.N) continue;
      if (some && a.w.bias) acc[h] += a.w.bias[int64_t(e) * a.w.N + n];
      store_f(a.Y, a.a_f32, p * a.w.N + n, acc[h]);
    }
  }
}

__global__ void __launch_bounds__(kThreads)
    gate_up_kernel(MoeArgs a, const int32_t *experts, float *hidden) {
  const int lane = threadIdx.x & 31, g = lane >> 2;
  const int64_t N16 = ceil_div(a.gate.N, kTileN), items = a.M * a.top_k * N16;
  for (int64_t it = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; it < items;
       it += ((int64_t)gridDim.x * blockDim.x) >> 5) {
    const int64_t p = it / N16, nt = it % N16;
    const int e = experts[p];
    if (e < 0) continue;
    float vg[2], vu[2];
    tile_dot(a.gate, e * N16 + nt, a.X, a.a_f32, p / a.top_k * a.gate.K, vg);
    tile_dot(a.up, e * N16 + nt, a.X, a.a_f32, p / a.top_k * a.gate.K, vu);
    for (int h = 0; h < 2; ++h) {
      const int64_t n = nt * kTileN + g + 8 * h;
      if ((lane & 3) || n >= a.gate.N) continue;
      if (a.gate.bias) vg[h] += a.gate.bias[int64_t(e) * a.gate.N + n];
      if (a.up.bias) vu[h] += a.up.bias[int64_t(e) * a.up.N + n];
      hidden[p * a.gate.N + n] = vg[h] / (1.f + expf(-vg[h])) * vu[h];
    }
  }
}

__global__ void __launch_bounds__(kThreads)
    down_kernel(MoeArgs a, const int32_t *experts, const float *weights, const float *hidden) {
  const int lane = threadIdx.x & 31, g = lane >> 2;
  const int64_t N16 = ceil_div(a.down.N, kTileN), items = a.M * N16;
  for (int64_t it = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; it < items;
       it += ((int64_t)gridDim.x * blockDim.x) >> 5) {
    const int64_t m = it / N16, nt = it % N16;
    float y[2] = {0.f, 0.f};
    for (int j = 0; j < a.top_k; ++j) {
      const int64_t p = m * a.top_k + j;
      const int e = experts[p];
      if (e < 0) continue;
      float v[2];
      tile_dot(a.down, e * N16 + nt, hidden, true, p * a.down.K, v);
      for (int h = 0; h < 2; ++h) {
        const int64_t n = nt * kTileN + g + 8 * h;
        if (n >= a.down.N) continue;
        if (a.down.bias) v[h] += a.down.bias[int64_t(e) * a.down.N + n];
        y[h] = fmaf(weights[p], v[h], y[h]);
      }
    }
    for (int h = 0; h < 2; ++h) {
      const int64_t n = nt * kTileN + g + 8 * h;
      if (!(lane & 3) && n < a.down.N) store_f(a.Y, a.a_f32, m * a.down.N + n, y[h]);
    }
  }
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
  return cudaGetLastError();
}

cudaError_t launch_moe_route(const RouteArgs &a, cudaStream_t stream) {
  const size_t keys = size_t(kWarps) * a.E * 4;
  route_kernel<<<grid_of(a.M, kWarps), kThreads, keys, stream>>>(
      a.logits, a.logits_f32, a.M, a.E, a.top_k, a.normalize, a.weights, a.experts);
  if (a.order) {
    static std::atomic<unsigned long long> done{0};
    const int bytes = (kListWarps + 1) * (kMoeMaxExperts + 1) * 4;
    const cudaError_t e = ensure_smem_limit(lists_kernel, bytes, done);
    if (e != cudaSuccess) return e;
    lists_kernel<<<1, kListWarps * 32, size_t(kListWarps + 1) * (a.E + 1) * 4, stream>>>(
        a.experts, a.M * a.top_k, a.E, a.offsets, a.order);
  }
  return cudaGetLastError();
}

cudaError_t launch_matmul_experts(const ExpertsArgs &a, cudaStream_t stream) {
  const int64_t items = a.M * a.top_k * ceil_div(a.w.N, kTileN);
  product_kernel<<<grid_of(items, kWarps), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

size_t moe_route_workspace_bytes(int64_t, int, int) { return 0; }
size_t matmul_experts_workspace_bytes(const ExpertsArgs &) { return 0; }

size_t moe_workspace_bytes(const MoeArgs &a) {
  const size_t P = size_t(a.M) * a.top_k;
  return 2 * align256(P * 4) + align256(P * a.gate.N * 4);
}

cudaError_t launch_moe(const MoeArgs &a, cudaStream_t stream) {
  const size_t P = size_t(a.M) * a.top_k;
  float *weights = reinterpret_cast<float *>(a.ws);
  int32_t *experts = reinterpret_cast<int32_t *>(a.ws + align256(P * 4));
  float *hidden = reinterpret_cast<float *>(a.ws + 2 * align256(P * 4));
  RouteArgs r{a.logits, a.logits_f32, a.M, a.gate.E, a.top_k, a.normalize, weights, experts,
              nullptr, nullptr, nullptr, a.pdl};
  const cudaError_t e = launch_moe_route(r, stream);
  if (e != cudaSuccess) return e;
  gate_up_kernel<<<grid_of(P * ceil_div(a.gate.N, kTileN), kWarps), kThreads, 0, stream>>>(
      a, experts, hidden);
  down_kernel<<<grid_of(a.M * ceil_div(a.down.N, kTileN), kWarps), kThreads, 0, stream>>>(
      a, experts, weights, hidden);
  return cudaGetLastError();
}

}  // namespace mnb
