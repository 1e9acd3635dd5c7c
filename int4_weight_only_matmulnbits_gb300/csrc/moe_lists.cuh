// Slots by expert inside one block: a stable counting sort of a few slots.
// (The counting sort of many slots is in moe.cu.)
#pragma once

#include "mnb_common.cuh"
#include "moe_stream.h"

namespace mnb {

// Shared-memory lists of P slots over E experts (P a few hundred).
struct SlotLists {
  int *e;          // [P] expert of each slot; E: none
  int *rank;       // [P] scratch
  int *off;        // [E + 2] first place of each expert's slots; off[E]: routed slots
  int *order;      // [P] slots by expert, those without one last
  SlotGroup *grp;  // [P] groups of up to gt slots
  int *ngrp;       // [1] how many
};
__host__ __device__ inline int slot_lists_ints(int P, int E) { return 6 * P + E + 3; }
__device__ __forceinline__ SlotLists slot_lists(int *base, int P, int E) {
  return SlotLists{base,
                   base + P,
                   base + 2 * P,
                   base + 2 * P + E + 2,
                   reinterpret_cast<SlotGroup *>(base + 3 * P + E + 2),
                   base + 6 * P + E + 2};
}

// Before the experts are known: clears the counters.
__device__ __forceinline__ void clear_lists(const SlotLists &s, int E) {
  for (int i = threadIdx.x; i < E + 2; i += blockDim.x) s.off[i] = 0;
}

// Builds off, order and the groups of up to 2^gt_log2 slots from e, by the
// whole block, after a barrier behind clear_lists() and the writes of e. One
// warp walks the slots 32 at a time, so equal experts keep their order, and
// scans the experts, each lane a contiguous run of them. Ends with a barrier.
__device__ __forceinline__ void build_lists(const SlotLists &s, int P, int E, int gt_log2) {
  const int lane = threadIdx.x & 31;
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
    const int gt = 1 << gt_log2, per = (E + 32) / 32;  // experts per lane (E counts as one)
    const int lo = min(lane * per, E + 1), hi = min(lo + per, E + 1);
    int slots = 0, groups = 0;
    for (int i = lo; i < hi; ++i) {
      const int c = s.off[i];
      slots += c;
      if (i < E) groups += (c + gt - 1) >> gt_log2;
    }
    // Both sums stay below 2^16.
    const int own = slots | (groups << 16);
    int x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) *s.ngrp = x >> 16;
    x -= own;
    int at = x & 0xFFFF, g = x >> 16;
    for (int i = lo; i < hi; ++i) {
      const int c = s.off[i];
      s.off[i] = at;
      if (i < E)
        for (int k = 0; k < c; k += gt) s.grp[g++] = SlotGroup{i, at + k, min(gt, c - k)};
      at += c;
    }
  }
  __syncthreads();
  for (int p = threadIdx.x; p < P; p += blockDim.x) s.order[s.off[s.e[p]] + s.rank[p]] = p;
  __syncthreads();
}

}  // namespace mnb
