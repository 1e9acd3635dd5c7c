// Rotary positions: tables of cosines and sines, and norms, rotation and
// cache writes of the query, key and value rows that a projection made.
//
// Row x of a head at position p (page "Qwen3 CPU Inference Critical Path",
// the fusion of QK layout, RoPE and cache; half-split RoPE of the model's
// contract):
//   y = x / sqrt(mean x^2 + eps) * gamma
//   (y_a, y_b) <- (y_a c - y_b s, y_b c + y_a s),  c, s = cos, sin[p][i]
// for pair i of the first `rot` elements: (a, b) = (i, i + rot/2), or
// (2i, 2i + 1) interleaved. All in fp32, rounded once when it is stored.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attn.h"
#include "mnb_common.cuh"
#include "mnb_launch.h"

namespace mnb {
namespace {

// ---- tables ---------------------------------------------------------------------

// An angle p f is held in turns as a 64-bit fraction: p times the fraction of
// f / 2 pi, modulo 2^64, is exact but for the rounding of f / 2 pi to 2^-64,
// at any position, with one integer product. The nearest quarter turn is
// taken off in integers too; the rest, at most pi / 4, is split at its nearest
// multiple of 2^-32 turns, so that it keeps all of its 24 bits however near a
// zero of the sine or cosine the angle lies, on either side, and goes through
// the Taylor series of sine (to x^9) and cosine (to x^10), which end below 2^-28
// there; in fp32, which leaves an error of 3 to 4e-8 where 64-bit results rounded
// once have 2 to 3e-8, at a fraction of the work. Bound by the writes (8 bytes an
// entry) and issue slots (some 40 instructions) alike: 147457 x 64 entries, 15.5
// us, are 11.3 of the one and about 10 of the other.
struct TableParams {
  uint64_t turns[kMaxPairs];
  int pairs;
  int64_t first, n;
  float mag, mag_lo;  // the magnitude in two parts
  float *cos, *sin;
};

__device__ __forceinline__ void table_entry(uint64_t turns, float mag, float mag_lo, float &c,
                                            float &s) {
  // In 2^-32 turns, to the nearest, from an eighth of a turn below.
  const uint32_t top = static_cast<uint32_t>((turns + 0x2000000080000000ull) >> 32);
  const uint32_t quarter = top >> 30;  // 0 .. 3 (4 as 0)
  // The rest's high part, and the signed low one: 2^-64 turns.
  const int32_t hi = static_cast<int32_t>((top & 0x3FFFFFFFu) - (1u << 29));
  const float lo = static_cast<float>(static_cast<int32_t>(turns));
  const float x = fmaf(static_cast<float>(hi), 0x1p32f, lo) * 0x1.921fb6p-62f;  // 2 pi 2^-64
  const float x2 = x * x;
  float p = fmaf(x2, 1.f / 362880.f, -1.f / 5040.f);
  p = fmaf(x2, p, 1.f / 120.f);
  p = fmaf(x2, p, -1.f / 6.f);
  float y = fmaf(x * x2, p, x);
  float q = fmaf(x2, -1.f / 3628800.f, 1.f / 40320.f);
  q = fmaf(x2, q, -1.f / 720.f);
  q = fmaf(x2, q, 1.f / 24.f);
  q = fmaf(x2, q, -0.5f);
  float z = fmaf(x2, q, 1.f);
  if (quarter & 1) {
    const float t = z;
    z = -y;
    y = t;
  }
  const uint32_t flip = (quarter & 2) << 30;
  z = __uint_as_float(__float_as_uint(z) ^ flip);
  y = __uint_as_float(__float_as_uint(y) ^ flip);
  c = fmaf(z, mag, z * mag_lo);
  s = fmaf(y, mag, y * mag_lo);
}

// A thread keeps V neighbouring pairs and takes every at_once-th position of its
// block's.
constexpr int kTableRows = 64;  // positions of a block: 128 leave too few blocks for 40960
template <int V>
__global__ void __launch_bounds__(256) table_kernel(const __grid_constant__ TableParams p) {
  const int per = p.pairs / V, at_once = 256 / per;
  const int j = threadIdx.x % per * V, r0 = threadIdx.x / per;
  if (r0 >= at_once) return;
  uint64_t turns[V];
#pragma unroll
  for (int e = 0; e < V; ++e) turns[e] = p.turns[j + e];
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t row0 = blockIdx.x * int64_t(kTableRows);
  const int rows = static_cast<int>(min(int64_t(kTableRows), p.n - row0));
  for (int r = r0; r < rows; r += at_once) {
    const uint64_t at = static_cast<uint64_t>(p.first + row0 + r);
    float c[V], s[V];
#pragma unroll
    for (int e = 0; e < V; ++e) table_entry(at * turns[e], p.mag, p.mag_lo, c[e], s[e]);
    float *pc = p.cos + (row0 + r) * p.pairs + j, *ps = p.sin + (row0 + r) * p.pairs + j;
    if constexpr (V == 4) {
      *reinterpret_cast<float4 *>(pc) = make_float4(c[0], c[1], c[2], c[3]);
      *reinterpret_cast<float4 *>(ps) = make_float4(s[0], s[1], s[2], s[3]);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        pc[e] = c[e];
        ps[e] = s[e];
      }
    }
  }
}

// ---- norms, rotation, cache -----------------------------------------------------

// The last sequence that begins at or before row t, by a search of 32 places a
// step; every lane of the warp takes part, with one t.
__device__ __forceinline__ int seq_of(const BatchView &b, int t, int lane) {
  int lo = 0, hi = b.n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step;
    const bool before = i < hi && b.starts[i] <= t;
    const int k = __popc(__ballot_sync(0xffffffffu, before));
    lo += k * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// Where row t goes: its position, and its place in the cache.
struct Place {
  int64_t pos;
  int64_t page;  // -1: no page holds it
  int at;
};
// False: the row belongs to no sequence. Whole warps; t0: the warp's first row.
template <bool APPEND>
__device__ __forceinline__ bool place_of(const RopeArgs &a, int64_t t, int64_t t0, int lane,
                                         Place &pl) {
  pl.page = -1;
  pl.at = 0;
  if (!APPEND) {
    pl.pos = a.pos ? a.pos[min(t, a.T - 1)] : -1;
    return t < a.T;
  }
  int s = seq_of(a.b, static_cast<int>(t0), lane);
  int end = a.b.starts[s + 1];
  while (end <= t && s + 1 < a.b.n) end = a.b.starts[++s + 1];
  if (t >= a.T || t >= end || t < a.b.starts[s]) return false;
  pl.pos = int64_t(a.b.lengths[s]) - (end - t);
  if (pl.pos >= 0 && pl.pos < int64_t(a.b.table_pages) * a.c.page_size) {
    const int i = static_cast<int>(pl.pos) / a.c.page_size;
    pl.at = static_cast<int>(pl.pos) - i * a.c.page_size;
    const int page = a.b.table[s * a.b.table_stride + i];
    if (page >= 0 && page < a.c.pages) pl.page = page;
  }
  return true;
}

template <bool F32>
struct Vec {  // 16 bytes of a row
  static constexpr int N = F32 ? 4 : 8;
  static __device__ __forceinline__ void widen(const uint4 &u, float (&v)[N]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
  static __device__ __forceinline__ uint4 narrow(const float (&v)[N]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if constexpr (F32)
        w[i] = __float_as_uint(v[i]);
      else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <int N>
__device__ __forceinline__ void load_floats(const float *p, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 x = *reinterpret_cast<const float4 *>(p + i);
    v[i] = x.x;
    v[i + 1] = x.y;
    v[i + 2] = x.z;
    v[i + 3] = x.w;
  }
}

// LANES lanes per head row, each with two 16-byte pieces that hold whole pairs:
// pieces s and s + rot/2 of the half-split layout (2s and 2s + 1 interleaved,
// and past the rotated part), so that nothing but the sum of squares crosses
// lanes. A group of lanes takes R heads of a token: their loads, which wait for
// no position, go first, all together, and its cosines and sines serve all of
// them. Bound by memory: every row is read and written once; the tables,
// shared by a token's heads, add rot * 4 bytes to it. Blocks on an SM (12 with four
// heads a group, 16 with one) count for more than registers: at the 80 and 64 that
// they leave a thread, the bf16 instances spill 76 to 84 bytes and 4 (fp32: none).
constexpr int kRopeThreads = 64;
template <bool F32, int LANES, int R, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads, R > 1 ? 12 : 16) rope_kernel(const __grid_constant__ RopeArgs a) {
  using V = Vec<F32>;
  constexpr int N = V::N;
  using E = typename std::conditional<F32, float, uint16_t>::type;
  const int lane = threadIdx.x & 31, s = threadIdx.x % LANES;
  grid_dependency_wait();
  grid_dependents_launch();
  const int rows = a.q.n + a.k.n + a.v.n, per = (rows + R - 1) / R;  // groups per token
  const int64_t g0 = (blockIdx.x * int64_t(kRopeThreads) + (threadIdx.x & ~31)) / LANES;
  const int64_t t0 = g0 / per;
  // The warp's groups are neighbours: same token, or the next ones.
  const int in = static_cast<int>(g0 - t0 * per) + lane / LANES;
  const int64_t t = t0 + in / per;
  const int h0 = (in - in / per * per) * R;
  const int pairs = a.rot / 2, slots = a.D / (2 * N), turning = a.rot / (2 * N);
  const bool mine = s < slots && t < a.T;
  const int o0 = s < turning && !a.interleaved ? s * N : s * 2 * N;
  const int o1 = s < turning && !a.interleaved ? pairs + s * N : s * 2 * N + N;
  uint4 r0[R], r1[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int h = h0 + i;
    r0[i] = r1[i] = make_uint4(0, 0, 0, 0);
    if (!mine || h >= rows) continue;
    const int kind = h < a.q.n ? 0 : h < a.q.n + a.k.n ? 1 : 2;
    const int hh = kind == 0 ? h : kind == 1 ? h - a.q.n : h - a.q.n - a.k.n;
    const Heads &src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const E *x = static_cast<const E *>(src.p) + t * src.ts + hh * src.hs;
    r0[i] = *reinterpret_cast<const uint4 *>(x + o0);
    r1[i] = *reinterpret_cast<const uint4 *>(x + o1);
  }
  Place pl;
  const bool there = place_of<APPEND>(a, t, t0, lane, pl);
  const bool turned = a.cos != nullptr && s < turning;
  const bool known = a.cos == nullptr || (pl.pos >= 0 && pl.pos < a.positions);
  float c[N], sn[N];
  if (there && turned && known) {
    load_floats<N>(a.cos + pl.pos * pairs + s * N, c);
    load_floats<N>(a.sin + pl.pos * pairs + s * N, sn);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int h = h0 + i;
    const int kind = h < a.q.n ? 0 : h < a.q.n + a.k.n ? 1 : 2;
    const int hh = kind == 0 ? h : kind == 1 ? h - a.q.n : h - a.q.n - a.k.n;
    const float *gamma = kind == 0 ? a.gq : kind == 1 ? a.gk : nullptr;
    float v0[N], v1[N];
    V::widen(r0[i], v0);
    V::widen(r1[i], v1);
    float sum = 0.f;
    if (a.gq || a.gk) {
#pragma unroll
      for (int e = 0; e < N; ++e) sum += v0[e] * v0[e] + v1[e] * v1[e];
#pragma unroll
      for (int m = 1; m < LANES; m *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    }
    if (!mine || !there || h >= rows) continue;
    E *y;
    if (kind == 0) {
      y = static_cast<E *>(a.qo.p) + t * a.qo.ts + hh * a.qo.hs;
    } else if (!APPEND) {
      y = static_cast<E *>(a.ko.p) + t * a.ko.ts + hh * a.ko.hs;
    } else {
      if (pl.page < 0) continue;
      const Pages &pg = kind == 1 ? a.c.k : a.c.v;
      y = static_cast<E *>(pg.p) + pl.page * pg.ps + hh * pg.hs + pl.at * pg.ts;
    }
    if (kind < 2) {
      if (gamma) {
        const float f = rsqrtf(sum / static_cast<float>(a.D) + a.eps);
        float g[N];
        load_floats<N>(gamma + o0, g);
#pragma unroll
        for (int e = 0; e < N; ++e) v0[e] = v0[e] * f * g[e];
        load_floats<N>(gamma + o1, g);
#pragma unroll
        for (int e = 0; e < N; ++e) v1[e] = v1[e] * f * g[e];
      }
      if (turned && known) {
        if (!a.interleaved) {
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const float p = v0[e], q = v1[e];
            v0[e] = p * c[e] - q * sn[e];
            v1[e] = q * c[e] + p * sn[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < N; e += 2) {
            const float p = v0[e], q = v0[e + 1], u = v1[e], w = v1[e + 1];
            v0[e] = p * c[e / 2] - q * sn[e / 2];
            v0[e + 1] = q * c[e / 2] + p * sn[e / 2];
            v1[e] = u * c[(N + e) / 2] - w * sn[(N + e) / 2];
            v1[e + 1] = w * c[(N + e) / 2] + u * sn[(N + e) / 2];
          }
        }
      }
      if (gamma || a.cos) {
        r0[i] = V::narrow(v0);
        r1[i] = V::narrow(v1);
      }
      if (!known) r0[i] = r1[i] = make_uint4(0, 0, 0, 0);
    }
    *reinterpret_cast<uint4 *>(y + o0) = r0[i];
    *reinterpret_cast<uint4 *>(y + o1) = r1[i];
  }
}

// Any even head size, rotated part and alignment: a warp per head row, the
// row in shared memory.
constexpr int kPlainWarps = 4;
template <bool F32, bool APPEND>
__global__ void __launch_bounds__(kPlainWarps * 32)
    rope_plain_kernel(const __grid_constant__ RopeArgs a) {
  using E = typename std::conditional<F32, float, uint16_t>::type;
  __shared__ float rows_s[kPlainWarps][kMaxHeadDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float *x = rows_s[warp];
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t t = blockIdx.x;
  Place pl;
  if (!place_of<APPEND>(a, t, t, lane, pl)) return;
  const int pairs = a.rot / 2;
  const bool known = a.cos == nullptr || (pl.pos >= 0 && pl.pos < a.positions);
  auto put = [](E *p, float v) {
    if constexpr (F32)
      *p = v;
    else
      *p = static_cast<uint16_t>(bf16_bits(v));
  };
  const int rows = a.q.n + a.k.n + a.v.n;
  for (int h = warp; h < rows; h += kPlainWarps) {
    const int kind = h < a.q.n ? 0 : h < a.q.n + a.k.n ? 1 : 2;
    const int hh = kind == 0 ? h : kind == 1 ? h - a.q.n : h - a.q.n - a.k.n;
    const Heads &src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const E *in = static_cast<const E *>(src.p) + t * src.ts + hh * src.hs;
    float sum = 0.f;
    __syncwarp();
    for (int i = lane; i < a.D; i += 32) {
      float v;
      if constexpr (F32)
        v = in[i];
      else
        v = bf16_bits_to_f32(in[i]);
      x[i] = v;
      sum += v * v;
    }
#pragma unroll
    for (int m = 1; m < 32; m *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    E *y;
    if (kind == 0) {
      y = static_cast<E *>(a.qo.p) + t * a.qo.ts + hh * a.qo.hs;
    } else if (!APPEND) {
      y = static_cast<E *>(a.ko.p) + t * a.ko.ts + hh * a.ko.hs;
    } else {
      if (pl.page < 0) continue;
      const Pages &pg = kind == 1 ? a.c.k : a.c.v;
      y = static_cast<E *>(pg.p) + pl.page * pg.ps + hh * pg.hs + pl.at * pg.ts;
    }
    const float *gamma = kind == 0 ? a.gq : kind == 1 ? a.gk : nullptr;
    if (gamma) {
      const float f = rsqrtf(sum / static_cast<float>(a.D) + a.eps);
      for (int i = lane; i < a.D; i += 32) x[i] = x[i] * f * gamma[i];
    }
    __syncwarp();
    const bool turned = kind < 2 && a.cos != nullptr;
    if (kind < 2 && !known) {
      for (int i = lane; i < a.D; i += 32) put(y + i, 0.f);
      continue;
    }
    for (int i = turned ? a.rot + lane : lane; i < a.D; i += 32) put(y + i, x[i]);
    if (turned)
      for (int i = lane; i < pairs; i += 32) {
        const int ia = a.interleaved ? 2 * i : i, ib = a.interleaved ? 2 * i + 1 : i + pairs;
        const float c = a.cos[pl.pos * pairs + i], s = a.sin[pl.pos * pairs + i];
        put(y + ia, x[ia] * c - x[ib] * s);
        put(y + ib, x[ib] * c + x[ia] * s);
      }
  }
}

bool vec_heads(const Heads &h, int64_t es) {
  return h.n == 0 || (reinterpret_cast<uintptr_t>(h.p) % 16 == 0 && h.ts * es % 16 == 0 &&
                      h.hs * es % 16 == 0);
}
bool vec_pages(const Pages &p, int64_t es) {
  return reinterpret_cast<uintptr_t>(p.p) % 16 == 0 && p.ps * es % 16 == 0 &&
         p.hs * es % 16 == 0 && p.ts * es % 16 == 0;
}
bool vec_floats(const float *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <bool F32, bool APPEND>
cudaError_t run_rope(const RopeArgs &a, cudaStream_t stream) {
  constexpr int N = Vec<F32>::N;
  constexpr int64_t es = F32 ? 4 : 2;
  const bool vec = a.D % (2 * N) == 0 && a.rot % (2 * N) == 0 && vec_heads(a.q, es) &&
                   vec_heads(a.k, es) && vec_heads(a.v, es) && vec_heads(a.qo, es) &&
                   (APPEND ? vec_pages(a.c.k, es) && vec_pages(a.c.v, es)
                           : vec_heads(a.ko, es)) &&
                   vec_floats(a.gq) && vec_floats(a.gk) && vec_floats(a.cos) &&
                   vec_floats(a.sin);
  if (!vec)
    return launch_after(rope_plain_kernel<F32, APPEND>, dim3(static_cast<unsigned>(a.T)),
                        kPlainWarps * 32, 0, a.pdl, stream, a);
  const int slots = a.D / (2 * N), rows = a.q.n + a.k.n + a.v.n;
  const int lanes = slots <= 4 ? 4 : slots <= 8 ? 8 : slots <= 16 ? 16 : 32;
  // Four heads a group once that still fills the GPU's threads; below, a head a
  // group is sooner done.
  const bool many = a.T * rows * lanes >= int64_t(4) * 2048 * std::max(1, sm_count());
  const int64_t groups = a.T * ceil_div(rows, many ? 4 : 1);
  const int64_t blocks = ceil_div(groups * lanes, kRopeThreads);
  if (blocks > (int64_t(1) << 31) - 1) return cudaErrorInvalidValue;
  void (*const kernels[2][4])(RopeArgs) = {
      {rope_kernel<F32, 4, 1, APPEND>, rope_kernel<F32, 8, 1, APPEND>,
       rope_kernel<F32, 16, 1, APPEND>, rope_kernel<F32, 32, 1, APPEND>},
      {rope_kernel<F32, 4, 4, APPEND>, rope_kernel<F32, 8, 4, APPEND>,
       rope_kernel<F32, 16, 4, APPEND>, rope_kernel<F32, 32, 4, APPEND>}};
  auto *kernel = kernels[many][lanes == 4 ? 0 : lanes == 8 ? 1 : lanes == 16 ? 2 : 3];
  return launch_after(kernel, dim3(static_cast<unsigned>(blocks)), kRopeThreads, 0, a.pdl, stream, a);
}

}  // namespace

cudaError_t launch_rope_table(const RopeTableArgs &a, cudaStream_t stream) {
  TableParams p{};
  for (int i = 0; i < a.pairs; ++i) {
    // The fraction of a turn that a position adds, rounded to 2^-64 (a double
    // keeps 53 bits of it), and its complement where it is negative.
    double f = std::fabs(a.frequencies[i]) * (0.5 / M_PI);
    f -= std::floor(f);
    p.turns[i] = static_cast<uint64_t>(f * 0x1p64 + 0.5);
    if (a.frequencies[i] < 0) p.turns[i] = 0 - p.turns[i];
  }
  p.pairs = a.pairs;
  p.first = a.first;
  p.n = a.n;
  p.mag = static_cast<float>(a.magnitude);
  p.mag_lo = static_cast<float>(a.magnitude - p.mag);
  p.cos = a.cos;
  p.sin = a.sin;
  const bool four = a.pairs % 4 == 0 && vec_floats(a.cos) && vec_floats(a.sin);
  const unsigned grid = static_cast<unsigned>(ceil_div(a.n, kTableRows));
  return launch_after(four ? table_kernel<4> : table_kernel<1>, dim3(grid), 256, 0, a.pdl, stream,
                      p);
}

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t stream) {
  if (a.f32) return a.append ? run_rope<true, true>(a, stream) : run_rope<true, false>(a, stream);
  return a.append ? run_rope<false, true>(a, stream) : run_rope<false, false>(a, stream);
}

}  // namespace mnb
