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
// taken off in integers too, so what sincospi gets, at most 1/4, has all of
// its 24 bits however near a zero of the cosine the angle lies.
struct TableParams {
  uint64_t turns[kMaxPairs];
  int pairs;
  int64_t first, n;
  float mag, mag_lo;  // the magnitude in two parts
  float *cos, *sin;
};

__device__ __forceinline__ void table_entry(uint64_t turns, float mag, float mag_lo, float &c,
                                            float &s) {
  const uint64_t quarter = (turns + (uint64_t(1) << 61)) >> 62;  // 0 .. 3 (4 as 0)
  const int64_t rest = static_cast<int64_t>(turns - (quarter << 62));
  float x, y;
  sincospif(static_cast<float>(rest) * 0x1p-63f, &y, &x);
  if (quarter & 1) {
    const float t = x;
    x = -y;
    y = t;
  }
  if (quarter & 2) {
    x = -x;
    y = -y;
  }
  c = fmaf(x, mag, x * mag_lo);
  s = fmaf(y, mag, y * mag_lo);
}

// A thread per V neighbouring pairs of a position.
template <int V>
__global__ void __launch_bounds__(256) table_kernel(const __grid_constant__ TableParams p) {
  const int per = p.pairs / V;
  const int64_t total = p.n * per;
  for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < total;
       i += gridDim.x * int64_t(256)) {
    const int64_t row = i / per;
    const int j = static_cast<int>(i - row * per) * V;
    const uint64_t at = static_cast<uint64_t>(p.first + row);
    float c[V], s[V];
#pragma unroll
    for (int e = 0; e < V; ++e) table_entry(at * p.turns[j + e], p.mag, p.mag_lo, c[e], s[e]);
    float *pc = p.cos + row * p.pairs + j, *ps = p.sin + row * p.pairs + j;
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

// The sequence that holds row t (-1: none), by a search of 32 places a step;
// every lane of the warp takes part.
__device__ __forceinline__ int seq_of(const BatchView &b, int t, int lane) {
  int lo = 0, hi = b.n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step;
    const bool before = i < hi && b.starts[i] <= t;
    const int k = __popc(__ballot_sync(0xffffffffu, before));
    lo += k * step;
    hi = min(hi, lo + step);
  }
  return b.starts[lo] <= t && t < b.starts[lo + 1] ? lo : -1;
}

// Where row t goes: its position (negative: none), and its place in the cache.
struct Place {
  int64_t pos;
  int64_t page;  // -1: no page holds it
  int at;
};
template <bool APPEND>
__device__ __forceinline__ bool place_of(const RopeArgs &a, int64_t t, int lane, Place &pl) {
  pl.page = -1;
  pl.at = 0;
  if (!APPEND) {
    pl.pos = a.pos ? a.pos[t] : -1;
    return true;
  }
  const int s = seq_of(a.b, static_cast<int>(t), lane);
  if (s < 0) return false;
  pl.pos = int64_t(a.b.lengths[s]) - (a.b.starts[s + 1] - t);
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
        w[i] = bf16_bits(v[2 * i]) | (bf16_bits(v[2 * i + 1]) << 16);
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

// One block per token; LANES lanes per head row, each with two 16-byte pieces
// that hold whole pairs: pieces s and s + rot/2 of the half-split layout (2s
// and 2s + 1 interleaved, and past the rotated part), so that nothing but the
// sum of squares crosses lanes. Cosines and sines are read once per lane and
// used for each of its heads. Bound by memory: every row is read and written
// once; the tables, shared by a token's heads, add rot * 4 bytes to it.
template <bool F32, int LANES, bool APPEND>
__global__ void __launch_bounds__(512) rope_kernel(const __grid_constant__ RopeArgs a) {
  using V = Vec<F32>;
  constexpr int N = V::N;
  using E = typename std::conditional<F32, float, uint16_t>::type;
  const int lane = threadIdx.x & 31, s = threadIdx.x % LANES;
  const int groups = blockDim.x / LANES;
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t t = blockIdx.x;
  Place pl;
  if (!place_of<APPEND>(a, t, lane, pl)) return;
  const int pairs = a.rot / 2, slots = a.D / (2 * N), turning = a.rot / (2 * N);
  const bool mine = s < slots, turned = a.cos != nullptr && s < turning;
  const bool known = a.cos == nullptr || (pl.pos >= 0 && pl.pos < a.positions);
  const int o0 = s < turning && !a.interleaved ? s * N : s * 2 * N;
  const int o1 = s < turning && !a.interleaved ? pairs + s * N : s * 2 * N + N;
  float c[N], sn[N];
  if (turned && known) {
    load_floats<N>(a.cos + pl.pos * pairs + s * N, c);
    load_floats<N>(a.sin + pl.pos * pairs + s * N, sn);
  }
  const int rows = a.q.n + a.k.n + a.v.n;
  // Whole warps go round together: the sum of squares crosses their lanes.
  for (int h0 = threadIdx.x / 32 * (32 / LANES); h0 < rows; h0 += groups) {
    const int h = h0 + lane / LANES;
    const bool live = mine && h < rows;
    const int kind = h < a.q.n ? 0 : h < a.q.n + a.k.n ? 1 : 2;
    const int hh = kind == 0 ? h : kind == 1 ? h - a.q.n : h - a.q.n - a.k.n;
    const Heads &src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    uint4 r0 = make_uint4(0, 0, 0, 0), r1 = r0;
    if (live) {
      const E *x = static_cast<const E *>(src.p) + t * src.ts + hh * src.hs;
      r0 = *reinterpret_cast<const uint4 *>(x + o0);
      r1 = *reinterpret_cast<const uint4 *>(x + o1);
    }
    const float *gamma = kind == 0 ? a.gq : kind == 1 ? a.gk : nullptr;
    float v0[N], v1[N];
    V::widen(r0, v0);
    V::widen(r1, v1);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) sum += v0[i] * v0[i] + v1[i] * v1[i];
#pragma unroll
    for (int m = 1; m < LANES; m *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (!live) continue;
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
        for (int i = 0; i < N; ++i) v0[i] = v0[i] * f * g[i];
        load_floats<N>(gamma + o1, g);
#pragma unroll
        for (int i = 0; i < N; ++i) v1[i] = v1[i] * f * g[i];
      }
      if (turned && known) {
        if (!a.interleaved) {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float p = v0[i], q = v1[i];
            v0[i] = p * c[i] - q * sn[i];
            v1[i] = q * c[i] + p * sn[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < N; i += 2) {
            const float p = v0[i], q = v0[i + 1], u = v1[i], w = v1[i + 1];
            v0[i] = p * c[i / 2] - q * sn[i / 2];
            v0[i + 1] = q * c[i / 2] + p * sn[i / 2];
            v1[i] = u * c[(N + i) / 2] - w * sn[(N + i) / 2];
            v1[i + 1] = w * c[(N + i) / 2] + u * sn[(N + i) / 2];
          }
        }
      }
      if (gamma || a.cos) {
        r0 = V::narrow(v0);
        r1 = V::narrow(v1);
      }
      if (!known) r0 = r1 = make_uint4(0, 0, 0, 0);
    }
    *reinterpret_cast<uint4 *>(y + o0) = r0;
    *reinterpret_cast<uint4 *>(y + o1) = r1;
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
  if (!place_of<APPEND>(a, t, lane, pl)) return;
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
  const dim3 grid(static_cast<unsigned>(a.T));
  if (!vec)
    return launch_after(rope_plain_kernel<F32, APPEND>, grid, kPlainWarps * 32, 0, a.pdl, stream,
                        a);
  const int slots = a.D / (2 * N), rows = a.q.n + a.k.n + a.v.n;
  const int lanes = slots <= 4 ? 4 : slots <= 8 ? 8 : slots <= 16 ? 16 : 32;
  const int threads = static_cast<int>(
      std::min<int64_t>(512, ceil_div(int64_t(rows) * lanes, 32) * 32));
  auto *kernel = lanes == 4    ? rope_kernel<F32, 4, APPEND>
                 : lanes == 8  ? rope_kernel<F32, 8, APPEND>
                 : lanes == 16 ? rope_kernel<F32, 16, APPEND>
                               : rope_kernel<F32, 32, APPEND>;
  return launch_after(kernel, grid, threads, 0, a.pdl, stream, a);
}

}  // namespace

cudaError_t launch_rope_table(const RopeTableArgs &a, cudaStream_t stream) {
  TableParams p{};
  for (int i = 0; i < a.pairs; ++i) {
    // The fraction of a turn that a position adds, rounded to 2^-64 (a double
    // keeps 53 bits of it).
    double f = a.frequencies[i] / (2.0 * M_PI);
    f -= std::floor(f);
    const double hi = std::floor(std::ldexp(f, 32));
    const double lo = std::ldexp(f, 64) - std::ldexp(hi, 32);
    p.turns[i] = (static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(lo);
  }
  p.pairs = a.pairs;
  p.first = a.first;
  p.n = a.n;
  p.mag = static_cast<float>(a.magnitude);
  p.mag_lo = static_cast<float>(a.magnitude - p.mag);
  p.cos = a.cos;
  p.sin = a.sin;
  const bool four = a.pairs % 4 == 0 && vec_floats(a.cos) && vec_floats(a.sin);
  const int64_t blocks = ceil_div(a.n * (four ? a.pairs / 4 : a.pairs), 256);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(blocks, 1 << 20));
  if (four)
    table_kernel<4><<<grid, 256, 0, stream>>>(p);
  else
    table_kernel<1><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t stream) {
  if (a.f32) return a.append ? run_rope<true, true>(a, stream) : run_rope<true, false>(a, stream);
  return a.append ? run_rope<false, true>(a, stream) : run_rope<false, false>(a, stream);
}

}  // namespace mnb
