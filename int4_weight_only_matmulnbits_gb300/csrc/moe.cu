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
#include "moe_lists.cuh"
#include "moe_route.cuh"
#include "moe_stream.h"

namespace mnb {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

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

// Slots by expert (one block): a stable counting sort. Each warp owns a
// contiguous range of slots and a row of counters; slots without an expert
// count as expert E.
constexpr int kListWarps = 16;
__global__ void __launch_bounds__(kListWarps * 32)
    lists_kernel(const int32_t *experts, int64_t P, int E, int32_t *offsets, int32_t *order) {
  extern __shared__ int32_t cnt[];  // [kListWarps][E + 1], then [E + 1]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t *mine = cnt + warp * (E + 1), *start = cnt + kListWarps * (E + 1);
  grid_dependency_wait();
  grid_dependents_launch();
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

// Router and lists of a few slots in one block.
__global__ void __launch_bounds__(kThreads) route_few_kernel(RouteArgs a) {
  extern __shared__ __align__(16) int few_smem[];
  const int P = static_cast<int>(a.M) * a.top_k;
  const SlotLists L = slot_lists(few_smem, P, a.E);
  uint32_t *keys = reinterpret_cast<uint32_t *>(few_smem + slot_lists_ints(P, a.E));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_dependents_launch();
  for (int m = warp; m < a.M; m += kWarps) {
    int e;
    float r;
    route_row(a.logits, a.logits_f32, m, a.E, a.top_k, a.normalize, keys + warp * a.E, e, r);
    if (lane < a.top_k) {
      a.experts[m * a.top_k + lane] = e;
      a.weights[m * a.top_k + lane] = r;
      L.e[m * a.top_k + lane] = e < 0 ? a.E : e;
    }
  }
  __syncthreads();
  build_lists(L, P, a.E, 1);
  for (int i = threadIdx.x; i <= a.E; i += kThreads) a.offsets[i] = L.off[i];
  for (int i = threadIdx.x; i < P; i += kThreads) a.order[i] = L.order[i];
}

// Sum of each token's down partials, in slot order (long inputs).
__global__ void __launch_bounds__(kThreads)
    combine_kernel(const float *part, const int32_t *experts, int64_t M, int top_k, int N,
                   void *Y, bool f32) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t total = M * N;
  for (int64_t i = blockIdx.x * int64_t(kThreads) + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * kThreads) {
    const int64_t m = i / N;
    float y = 0.f;
    for (int j = 0; j < top_k; ++j)
      if (experts[m * top_k + j] >= 0) y += part[(m * top_k + j) * N + (i - m * N)];
    store_f(Y, f32, i, y);
  }
}

template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kernel)(P...), unsigned grid, int block, size_t smem, bool pdl,
                       cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
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
  return cudaGetLastError();
}


namespace {

int ilog2(int x) {
  int r = 0;
  while ((1 << r) < x) ++r;
  return r;
}

// Fills the geometry of a weight-streaming launch. `lists_p`: slots listed in
// shared memory (0: ready lists); `per_expert`: the most slots an expert can
// have. false: not even one activation row fits.
struct StreamPlan {
  StreamParams p{};
  int terms = 1, grid = 1, smem = 0;
  bool zp = false, sf32 = false;
};
bool plan_stream(StreamPlan &pl, const ExpertStack &w, int mode, int terms, int64_t P,
                 int64_t M, int top_k, bool few, int64_t per_expert, bool keys) {
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
  p.P = static_cast<int>(P);
  p.M = static_cast<int>(M);
  p.top_k = top_k;
  const int nmat = mode == kStreamGateUp ? 2 : 1, es = w.s_f32 ? 4 : 2;
  // k ranges of at least three chunks per warp.
  p.ksplit = 8;
  while (p.ksplit > 1 && p.K64 / p.ksplit < 3) p.ksplit /= 2;
  p.tpu = 8 / p.ksplit;
  p.ns = static_cast<int>(ceil_div(p.N16, p.tpu));
  const int range = static_cast<int>(ceil_div(p.K64, p.ksplit));
  p.kc = static_cast<int>(ceil_div(range, ceil_div(range, 4)));
  const int nblk = (p.kc * kChunkK + w.bs - 1) / w.bs + 1;
  p.st_scale = p.kc * kChunkBytes;
  p.st_zp = p.st_scale + (nblk * kTileN * es + 15) / 16 * 16;
  p.st_bytes = (p.st_zp + (pl.zp ? (nblk / 2 + 1) * 16 : 0) + 127) / 128 * 128;
  const int64_t krow = int64_t(p.K64) * kChunkK + 16;
  const int64_t lists =
      (int64_t(slot_lists_ints(few ? p.P : 0, p.E)) * 4 + (few ? p.P * 4 : 0) + 127) / 128 * 128;
  const int red = 2 * 8 * nmat * kTileN * 8 * 4;
  const int64_t ring =
      std::max<int64_t>(8 * 4 * p.st_bytes, keys ? int64_t(8) * p.E * 4 : 0);
  // Slots per group: about twice the mean list, so that few experts need a
  // second pass over their weights, within what two CTAs per SM leave (one
  // CTA per SM when that is not enough for the mean).
  const int64_t mean = ceil_div(P, w.E);
  int want = 1;
  while (want < 8 && want < 2 * mean && want < per_expert) want *= 2;
  constexpr int64_t kHalf = 113 * 1024, kFull = 226 * 1024;
  auto bytes = [&](int gt) { return lists + red + ring + int64_t(terms) * gt * krow * 2; };
  int gt = want;
  while (gt > 1 && bytes(gt) > kHalf && gt > mean) gt /= 2;
  while (gt > 1 && bytes(gt) > kFull) gt /= 2;
  if (bytes(gt) > kFull) return false;
  p.gt = gt;
  p.krow = static_cast<int>(krow);
  p.off_lists = 0;
  p.off_keys = slot_lists_ints(few ? p.P : 0, p.E) * 4;
  p.off_red = static_cast<int>(lists);
  p.off_ring = p.off_red + red;
  p.off_x = static_cast<int>(p.off_ring + ring);
  pl.smem = static_cast<int>(bytes(gt));
  const int64_t most = P * p.ns, slots = int64_t(sm_count()) * (pl.smem <= kHalf ? 2 : 1);
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
  int32_t *experts = nullptr, *offsets = nullptr, *order = nullptr;
};

cudaError_t launch_lists(const int32_t *experts, int64_t P, int E, int32_t *offsets,
                         int32_t *order, bool pdl, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = ensure_smem_limit(
      lists_kernel, (kListWarps + 1) * (kMoeMaxExperts + 1) * 4, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(lists_kernel, 1, kListWarps * 32, size_t(kListWarps + 1) * (E + 1) * 4, pdl,
                    stream, experts, P, E, offsets, order);
}

struct MoeSpace {
  Lists l;
  uint16_t *hidden;
  float *part;
  unsigned *counters;
  size_t bytes;
};
MoeSpace moe_space(const MoeArgs &a) {
  const size_t P = size_t(a.M) * a.top_k;
  Carve c{a.ws};
  MoeSpace s{};
  if (P > kFewSlots) {
    s.l.weights = c.take<float>(P);
    s.l.experts = c.take<int32_t>(P);
    s.l.offsets = c.take<int32_t>(a.gate.E + 1);
    s.l.order = c.take<int32_t>(P);
  } else {
    s.counters = c.take<unsigned>(ceil_div(a.down.N, kTileN));
  }
  const size_t ldh = ceil_div(a.gate.N, 8) * 8;
  s.hidden = c.take<uint16_t>((a.a_f32 ? 3 : 2) * P * ldh);
  s.part = c.take<float>(P * a.down.N);
  s.bytes = c.used;
  return s;
}

}  // namespace

size_t moe_route_workspace_bytes(int64_t, int, int) { return 0; }

cudaError_t launch_moe_route(const RouteArgs &a, cudaStream_t stream) {
  const int64_t P = a.M * a.top_k;
  if (a.order && P <= kFewSlots) {
    const size_t smem = size_t(slot_lists_ints(static_cast<int>(P), a.E) + kWarps * a.E) * 4;
    return launch_pdl(route_few_kernel, 1, kThreads, smem, a.pdl, stream, a);
  }
  cudaError_t e = launch_pdl(route_kernel, grid_of(a.M, kWarps), kThreads,
                             size_t(kWarps) * a.E * 4, a.pdl, stream, a.logits, a.logits_f32,
                             a.M, a.E, a.top_k, a.normalize, a.weights, a.experts);
  if (e == cudaSuccess && a.order)
    e = launch_lists(a.experts, P, a.E, a.offsets, a.order, a.pdl, stream);
  return e;
}

size_t matmul_experts_workspace_bytes(const ExpertsArgs &a) {
  const size_t P = size_t(a.M) * a.top_k;
  if (P <= kFewSlots) return 0;
  return align256(size_t(a.w.E + 1) * 4) + align256(P * 4);
}

cudaError_t launch_matmul_experts(const ExpertsArgs &a, cudaStream_t stream) {
  const int64_t P = a.M * a.top_k;
  const bool few = P <= kFewSlots;
  StreamPlan pl;
  if (!plan_stream(pl, a.w, kStreamProduct, a.a_f32 ? 3 : 1, P, a.M, a.top_k, few, P, false))
    return cudaErrorNotSupported;
  Lists l;
  if (!few) {
    Carve c{a.ws};
    l.offsets = c.take<int32_t>(a.w.E + 1);
    l.order = c.take<int32_t>(P);
    const cudaError_t e =
        launch_lists(a.experts, P, a.w.E, l.offsets, l.order, a.pdl, stream);
    if (e != cudaSuccess) return e;
  }
  StreamParams &p = pl.p;
  p.w[0] = stream_mat(a.w);
  p.A = a.A;
  p.a_vec = vec_rows(a.A, a.w.K, a.a_f32 ? 4 : 2);
  p.per_slot = a.per_slot;
  p.table = a.experts;
  p.offsets = l.offsets;
  p.order = l.order;
  p.Y = a.Y;
  p.y_f32 = a.a_f32;
  return run_stream(pl, a.pdl, stream);
}

size_t moe_workspace_bytes(const MoeArgs &a) {
  MoeArgs b = a;
  b.ws = nullptr;
  return moe_space(b).bytes;
}

cudaError_t launch_moe(const MoeArgs &a, cudaStream_t stream) {
  const int64_t P = a.M * a.top_k;
  const bool few = P <= kFewSlots;
  const MoeSpace s = moe_space(a);
  StreamPlan up, down;
  if (!plan_stream(up, a.gate, kStreamGateUp, a.a_f32 ? 3 : 1, P, a.M, a.top_k, few, a.M, few) ||
      !plan_stream(down, a.down, kStreamDown, a.a_f32 ? 3 : 2, P, a.M, a.top_k, few, a.M, few))
    return cudaErrorNotSupported;
  if (!few) {
    const RouteArgs r{a.logits, a.logits_f32, a.M, a.gate.E, a.top_k, a.normalize, s.l.weights,
                      s.l.experts, s.l.offsets, s.l.order, nullptr, a.pdl};
    const cudaError_t e = launch_moe_route(r, stream);
    if (e != cudaSuccess) return e;
  }
  for (StreamParams *p : {&up.p, &down.p}) {
    if (few) {
      p->logits = a.logits;
      p->logits_f32 = a.logits_f32;
      p->normalize = a.normalize;
    } else {
      p->offsets = s.l.offsets;
      p->order = s.l.order;
      p->weights = s.l.weights;
      p->experts = s.l.experts;
    }
    p->y_f32 = a.a_f32;
    p->plane = P * (ceil_div(a.gate.N, 8) * 8);
    p->ldh = static_cast<int>(ceil_div(a.gate.N, 8) * 8);
    p->counters = s.counters;
  }
  up.p.w[0] = stream_mat(a.gate);
  up.p.w[1] = stream_mat(a.up);
  up.p.A = a.X;
  up.p.a_vec = vec_rows(a.X, a.gate.K, a.a_f32 ? 4 : 2);
  up.p.hidden = s.hidden;
  up.p.h_planes = a.a_f32 ? 3 : 2;
  up.p.n_counters = few ? down.p.ns : 0;
  cudaError_t e = run_stream(up, a.pdl, stream);
  if (e != cudaSuccess) return e;
  down.p.w[0] = stream_mat(a.down);
  down.p.A = s.hidden;
  down.p.a_vec = 1;
  down.p.part = s.part;
  down.p.Y = a.Y;
  down.p.early = few;
  e = run_stream(down, a.pdl, stream);
  if (e != cudaSuccess || few) return e;
  return launch_pdl(combine_kernel, grid_of(a.M * a.down.N, kThreads), kThreads, 0, a.pdl,
                    stream, s.part, s.l.experts, a.M, a.top_k, a.down.N, a.Y, a.a_f32);
}

}  // namespace mnb
