// The top-k softmax router for one row of logits, by one warp.
//
// For a row l[0..E): p_e = exp(l_e - max l). The k largest l_e are chosen,
// largest first, ties going to the lowest index; choice j has the weight
// p_j / sum (over the chosen when normalizing, over all experts otherwise).
// -inf and NaN mask an expert: it is never chosen and adds nothing. When
// fewer than k experts are left, the remaining choices are expert -1 with
// weight 0. +inf counts as the maximum: it has p = 1, finite logits beside
// it p = 0.
//
// Selection compares 32-bit keys whose unsigned order is the order of the
// logits, so the same integer reductions serve fp32 and bf16 logits and the
// choice is exact; sums and weights are fp32.
#pragma once

#include <cstdint>
#include <type_traits>

#include "mnb_common.cuh"

namespace mnb {

// Order-preserving key of a logit: 0 for -inf and NaN (masked), otherwise
// larger for larger values; -0 and +0 share a key.
__device__ __forceinline__ uint32_t logit_key(float x) {
  if (!(x > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// The key of a bf16 logit from its upper half: the lower one is zeros for
// positive values and ones for negative ones.
__device__ __forceinline__ uint32_t bf16_key(uint32_t k) {
  return (k & 0x80000000u) ? (k & 0xFFFF0000u) : (k | 0xFFFFu);
}
// exp(l - max), with exp(inf - inf) = 1.
__device__ __forceinline__ float logit_exp(float l, float top) {
  return l == top ? 1.f : expf(l - top);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Lane j < top_k gets choice j of row m: expert (or -1) and weight. A lane
// holds KPL experts (32 KPL >= E) as a list sorted by key, then index, whose
// head it offers; the winner's lane moves on. bf16
// logits fit 16 bits: key and inverted index share a word, one reduction a
// choice; fp32 logits take a second one for the index.
template <int KPL, bool F32>
__device__ __forceinline__ void route_row_regs(const void *logits, int64_t m, int E, int top_k,
                                               bool normalize, int &expert, float &weight) {
  const int lane = threadIdx.x & 31;
  uint32_t key[KPL];
  int at[KPL];
  // Rows of whole, aligned pieces: a lane's KPL experts are neighbours and
  // come in one load (a row of 128 fp32 logits: 3.3 us, one by one 3.7).
  constexpr int kPiece = KPL * (F32 ? 4 : 2) < 16 ? KPL * (F32 ? 4 : 2) : 16;
  const bool vec = E % KPL == 0 && reinterpret_cast<uintptr_t>(logits) % kPiece == 0;
  float x[KPL];
#pragma unroll
  for (int q = 0; q < KPL; ++q) x[q] = -INFINITY;
  if (vec) {
    if (lane * KPL < E) {
      const char *src = static_cast<const char *>(logits) + (m * E + lane * KPL) * (F32 ? 4 : 2);
      uint32_t w[KPL * (F32 ? 4 : 2) / 4];
#pragma unroll
      for (int i = 0; i < KPL * (F32 ? 4 : 2) / kPiece; ++i) {
        if constexpr (kPiece == 16) {
          const uint4 v = reinterpret_cast<const uint4 *>(src)[i];
          w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        } else if constexpr (kPiece == 8) {
          const uint2 v = *reinterpret_cast<const uint2 *>(src);
          w[0] = v.x; w[1] = v.y;
        } else {
          w[0] = *reinterpret_cast<const uint32_t *>(src);
        }
      }
#pragma unroll
      for (int q = 0; q < KPL; ++q)
        x[q] = __uint_as_float(F32 ? w[q] : q & 1 ? w[q / 2] & 0xFFFF0000u : w[q / 2] << 16);
    }
  } else {
#pragma unroll
    for (int q = 0; q < KPL; ++q) {
      const int i = lane + 32 * q;
      if (i < E)
        x[q] = F32 ? static_cast<const float *>(logits)[m * E + i]
                   : bf16_bits_to_f32(static_cast<const uint16_t *>(logits)[m * E + i]);
    }
  }
#pragma unroll
  for (int q = 0; q < KPL; ++q) {
    const int i = vec ? lane * KPL + q : lane + 32 * q;
    key[q] = logit_key(x[q]);
    at[q] = i;
    if (!F32 && key[q]) key[q] = (key[q] & 0xFFFF0000u) | (0xFFFFu - i);
  }
  // The logit behind a key.
  auto value = [](uint32_t k) { return key_logit(F32 ? k : bf16_key(k)); };
  float all = 0.f;
  if (!normalize) {
    uint32_t best = key[0];
#pragma unroll
    for (int q = 1; q < KPL; ++q) best = max(best, key[q]);
    best = __reduce_max_sync(0xffffffffu, best);
#pragma unroll
    for (int q = 0; q < KPL; ++q)
      if (key[q]) all += logit_exp(value(key[q]), value(best));
    all = warp_sum(all);
  }
#pragma unroll
  for (int i = 0; i < KPL - 1; ++i)  // larger keys first; equal ones stay in order
#pragma unroll
    for (int q = 0; q < KPL - 1 - i; ++q)
      if (key[q + 1] > key[q]) {
        const uint32_t k = key[q];
        key[q] = key[q + 1];
        key[q + 1] = k;
        if (F32) {
          const int t = at[q];
          at[q] = at[q + 1];
          at[q + 1] = t;
        }
      }
  uint32_t first = 0, mine = 0;
  expert = -1;
#pragma unroll 1
  for (int j = 0; j < top_k; ++j) {
    const uint32_t win = __reduce_max_sync(0xffffffffu, key[0]);
    if (win == 0) break;  // every expert left is masked
    int e = static_cast<int>(0xFFFFu - (win & 0xFFFFu));
    bool own = key[0] == win;
    if (F32) {
      e = static_cast<int>(
          __reduce_min_sync(0xffffffffu, own ? static_cast<uint32_t>(at[0]) : 0xFFFFFFFFu));
      own = own && at[0] == e;
    }
    if (j == 0) first = win;
    if (lane == j) {
      expert = e;
      mine = win;
    }
#pragma unroll
    for (int q = 0; q < KPL; ++q) {
      key[q] = own ? (q + 1 < KPL ? key[q + 1] : 0u) : key[q];
      if (F32 && q + 1 < KPL) at[q] = own ? at[q + 1] : at[q];
    }
  }
  const float p = expert < 0 ? 0.f : logit_exp(value(mine), value(first));
  const float chosen = warp_sum(p);
  weight = expert < 0 ? 0.f : p / (normalize ? chosen : all);
}

// The same with the keys in E words of shared memory of this warp (any E).
__device__ __forceinline__ void route_row_shared(const void *logits, bool f32, int64_t m, int E,
                                          int top_k, bool normalize, uint32_t *keys,
                                          int &expert, float &weight) {
  const int lane = threadIdx.x & 31;
  uint32_t best = 0;
  int bi = 0;
  for (int i = lane; i < E; i += 32) {
    const float x =
        f32 ? static_cast<const float *>(logits)[m * E + i]
            : bf16_bits_to_f32(static_cast<const uint16_t *>(logits)[m * E + i]);
    const uint32_t k = logit_key(x);
    keys[i] = k;
    if (k > best) {
      best = k;
      bi = i;
    }
  }
  const float top = key_logit(__reduce_max_sync(0xffffffffu, best));
  float all = 0.f;
  if (!normalize) {
    for (int i = lane; i < E; i += 32)
      if (keys[i]) all += logit_exp(key_logit(keys[i]), top);
    all = warp_sum(all);
  }
  expert = -1;
  float p = 0.f;
  for (int j = 0; j < top_k; ++j) {
    const uint32_t win = __reduce_max_sync(0xffffffffu, best);
    if (win == 0) break;  // every expert left is masked
    const int at = static_cast<int>(
        __reduce_min_sync(0xffffffffu, best == win ? static_cast<uint32_t>(bi) : 0xFFFFFFFFu));
    if (lane == j) {
      expert = at;
      p = logit_exp(key_logit(win), top);
    }
    if ((at & 31) == lane) {  // this lane's next best
      keys[at] = 0;
      best = 0;
      for (int i = lane; i < E; i += 32)
        if (keys[i] > best) {
          best = keys[i];
          bi = i;
        }
    }
  }
  const float chosen = warp_sum(p);
  weight = expert < 0 ? 0.f : p / (normalize ? chosen : all);
}

// keys: E words of shared memory of this warp (used when E > 256).
__device__ __forceinline__ void route_row(const void *logits, bool f32, int64_t m, int E,
                                          int top_k, bool normalize, uint32_t *keys,
                                          int &expert, float &weight) {
  auto regs = [&](auto kpl) {
    if (f32) route_row_regs<kpl.value, true>(logits, m, E, top_k, normalize, expert, weight);
    else route_row_regs<kpl.value, false>(logits, m, E, top_k, normalize, expert, weight);
  };
  if (E <= 64) regs(std::integral_constant<int, 2>());
  else if (E <= 128) regs(std::integral_constant<int, 4>());
  else if (E <= 256) regs(std::integral_constant<int, 8>());
  else route_row_shared(logits, f32, m, E, top_k, normalize, keys, expert, weight);
}

}  // namespace mnb
