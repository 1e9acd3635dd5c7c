// Slots by expert inside one block: a stable counting sort of a few slots.
#pragma once

#include "mnb_common.cuh"

namespace mnb {

// Exclusive prefix sums by one warp over n values; `get(i)` yields value i,
// `put(i, sum)` receives the sum of the values before i; returns the total.
template <typename Get, typename Put>
__device__ __forceinline__ int warp_prefix(int n, Get get, Put put) {
  const int lane = threadIdx.x & 31;
  int base = 0;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    const int v = i < n ? get(i) : 0;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (i < n) put(i, base + x - v);
    base += __shfl_sync(0xffffffffu, x, 31);
  }
  return base;
}

// Shared-memory lists of P slots over E experts.
struct SlotLists {
  int *e;      // [P] expert of each slot; E: none
  int *rank;   // [P] scratch
  int *off;    // [E + 2] first place of each expert's slots; off[E]: routed slots
  int *gpre;   // [E + 1] groups (of up to gt slots) before each expert
  int *order;  // [P] slots by expert, those without one last
};
__host__ __device__ inline int slot_lists_ints(int P, int E) { return 3 * P + 2 * E + 3; }
__device__ __forceinline__ SlotLists slot_lists(int *base, int P, int E) {
  return SlotLists{base, base + P, base + 2 * P, base + 2 * P + E + 2,
                   base + 2 * P + 2 * E + 3};
}

// Builds off, gpre and order from e, by the whole block (blockDim.x threads);
// e must be written before a barrier ahead of this call. One warp walks the
// slots 32 at a time, so equal experts keep their order; P is small (a few
// hundred). Ends with a barrier.
__device__ __forceinline__ void build_lists(const SlotLists &s, int P, int E, int gt) {
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < E + 2; i += blockDim.x) s.off[i] = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    for (int p0 = 0; p0 < P; p0 += 32) {
      const int p = p0 + lane;
      const int e = p < P ? s.e[p] : E + 1;
      const unsigned same = __match_any_sync(0xffffffffu, e);
      const int before = __popc(same & ((1u << lane) - 1));
      if (p < P) s.rank[p] = s.off[e] + before;
      __syncwarp();
      if (p < P && before == 0) s.off[e] += __popc(same);
      __syncwarp();
    }
    const int groups = warp_prefix(
        E, [&](int i) { return (s.off[i] + gt - 1) / gt; }, [&](int i, int v) { s.gpre[i] = v; });
    if (lane == 0) s.gpre[E] = groups;
    warp_prefix(
        E + 1, [&](int i) { return s.off[i]; }, [&](int i, int v) { s.off[i] = v; });
  }
  __syncthreads();
  for (int p = threadIdx.x; p < P; p += blockDim.x) s.order[s.off[s.e[p]] + s.rank[p]] = p;
  __syncthreads();
}

}  // namespace mnb
