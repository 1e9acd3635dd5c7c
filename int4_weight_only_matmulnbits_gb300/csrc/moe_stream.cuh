// Weight-streaming kernel of the expert layer, for few slots per expert.
//
// Slots are listed by expert and cut into groups of up to 8 that share an
// expert; for each group the kernel streams the expert's packed rows once
// and multiplies them with the group's activation rows:
//   product     Y[p]    = W_e a_p + b_e
//   gate + up   h[p]    = r_p * silu(Wg_e x + bg) * (Wu_e x + bu)
//   down        Y[m]    = sum over the slots of m of (Wd_e h[p] + r_p bd)
// Every weight byte is read once per group, 24 bytes a cycle and SM at full
// memory bandwidth, while a 512-byte chunk (64 k of 16 rows) costs a warp
// about 80 instructions: memory bounds it, with little to spare, as long as
// enough bytes are in flight.
//
//  * Warps are autonomous: each streams its own sequence of (tile, k range)
//    pieces through a private ring of shared-memory stages filled by
//    asynchronous 16-byte copies, across steps, tiles and experts. No
//    barrier is needed to refill a stage, and a lane reads back the very
//    16 bytes it copied.
//  * A step is `tpu` tiles of one group; `ksplit` warps share a tile's k and
//    meet in shared memory, in fixed order, once per step. CTAs take equal
//    contiguous runs of steps, so a group's activations are staged about
//    once per CTA.
//  * Codes become bf16 q - z exactly (128 + q by one logic operation per
//    pair, minus 128 + z), the products with bf16 activations are exact in
//    fp32, and a block's scale is applied to its fp32 sum: no weight is
//    rounded. fp32 activations enter as three bf16 parts by truncation
//    (8 + 8 + 8 bits: their sum is the value), hidden values as two (bf16
//    activations, 2^-16) or three.
//  * The layer takes two launches. Both run the router for themselves, so
//    the second needs nothing from the first but the hidden rows: it routes
//    and fills its rings before it waits for the first kernel to finish.
//    Down partials go to a workspace; the CTA that completes a column
//    group, by an arrival counter, adds them in slot order, so the result
//    does not depend on which CTA that is.
#pragma once

#include <cuda_bf16.h>

#include <atomic>

#include "mnb_common.cuh"
#include "mnb_launch.h"
#include "moe_lists.cuh"
#include "moe_route.cuh"
#include "moe_stream.h"

namespace mnb {
namespace stream {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCols = 8;    // slots per group at most
constexpr int kStages = 4;  // ring depth per warp

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t bf16x2_sub(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Where a warp stands in its sequence of stages.
struct Cursor {
  int step, e, group, nstep;  // step; its group's expert, id and column step
  int mat, c;                 // matrix and first chunk of the stage
};

template <int SPB, bool ZP, bool SF32, int TERMS>
__global__ void __launch_bounds__(kThreads, 2) stream_kernel(const StreamParams p) {
  constexpr int kEs = SF32 ? 4 : 2;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const bool ready = p.offsets != nullptr;  // lists in global memory
  const SlotLists L = slot_lists(reinterpret_cast<int *>(smem + p.off_lists), ready ? 0 : p.P, p.E);
  float *s_w = reinterpret_cast<float *>(smem + p.off_keys);  // weights [P] (few slots)
  __shared__ int s_last;

  if (!p.early) {
    grid_dependency_wait();
    grid_dependents_launch();
  }
  // ---- lists --------------------------------------------------------------------
  if (ready) {
    for (int i = tid; i <= p.E; i += kThreads) L.off[i] = p.offsets[i];
    __syncthreads();
    if (warp == 0) {
      const int n = warp_prefix(
          p.E, [&](int i) { return (L.off[i + 1] - L.off[i] + p.gt - 1) / p.gt; },
          [&](int i, int v) { L.gpre[i] = v; });
      if (lane == 0) L.gpre[p.E] = n;
    }
    __syncthreads();
  } else {
    if (p.logits) {
      uint32_t *keys = reinterpret_cast<uint32_t *>(smem + p.off_ring) + warp * p.E;
      for (int m = warp; m < p.M; m += kWarps) {
        int e;
        float r;
        route_row(p.logits, p.logits_f32 != 0, m, p.E, p.top_k, p.normalize != 0, keys, e, r);
        if (lane < p.top_k) {
          L.e[m * p.top_k + lane] = e < 0 ? p.E : e;
          s_w[m * p.top_k + lane] = r;
        }
      }
    } else {
      for (int i = tid; i < p.P; i += kThreads) {
        const int e = p.table[i];
        L.e[i] = e >= 0 && e < p.E ? e : p.E;
      }
    }
    __syncthreads();
    build_lists(L, p.P, p.E, p.gt);
  }
  const int32_t *order = ready ? p.order : L.order;
  const float *weights = ready ? p.weights : s_w;
  const int routed = L.off[p.E];

  // ---- this CTA's steps ------------------------------------------------------------
  const int groups = L.gpre[p.E];
  const int64_t total = int64_t(groups) * p.ns;
  const int lo = static_cast<int>(total * blockIdx.x / gridDim.x);
  const int hi = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x);
  const int nmat = p.mode == kStreamGateUp ? 2 : 1;
  const int ks = warp % p.ksplit, tl = warp / p.ksplit;
  const int c0 = p.K64 * ks / p.ksplit, c1 = p.K64 * (ks + 1) / p.ksplit;
  unsigned char *ring = smem + p.off_ring + warp * (kStages * p.st_bytes);
  const uint32_t ring_u = smem_addr(ring);

  auto expert_of = [&](int e, int group) {
    while (L.gpre[e + 1] <= group) ++e;
    return e;
  };
  auto has_tile = [&](const Cursor &q) { return q.nstep * p.tpu + tl < p.N16; };
  auto next_step = [&](Cursor &q) {
    ++q.step;
    if (++q.nstep == p.ns) {
      q.nstep = 0;
      ++q.group;
      if (q.step < hi) q.e = expert_of(q.e, q.group);
    }
  };
  Cursor pre;  // next stage to fetch
  pre.step = lo;
  pre.group = lo / p.ns;
  pre.nstep = lo - pre.group * p.ns;
  pre.e = lo < hi ? expert_of(0, pre.group) : 0;
  pre.mat = 0;
  pre.c = c0;
  Cursor cur = pre;
  while (pre.step < hi && !has_tile(pre)) next_step(pre);

  auto fetch = [&](int slot) {
    if (pre.step < hi) {
      const int64_t tile = int64_t(pre.e) * p.N16 + pre.nstep * p.tpu + tl;
      const int n = min(p.kc, c1 - pre.c);
      const uint32_t dst = ring_u + slot * p.st_bytes + lane * 16;
      const uint4 *src = p.w[pre.mat].b + (tile * p.K64 + pre.c) * 32 + lane;
      for (int i = 0; i < n; ++i) cp16(dst + i * kChunkBytes, src + i * 32);
      const int b0 = (pre.c * kChunkK) >> p.bs_log2;
      const int b1 = min(p.nb, (((pre.c + n) * kChunkK - 1) >> p.bs_log2) + 1);
      const unsigned char *ss = p.w[pre.mat].s + (tile * p.nb + b0) * (kTileN * kEs);
      for (int i = lane; i < (b1 - b0) * kEs; i += 32)
        cp16(ring_u + slot * p.st_bytes + p.st_scale + i * 16, ss + i * 16);
      if (ZP) {
        // Pairs of words from an even block on.
        const unsigned char *zz = p.w[pre.mat].z + (tile * p.nbz + (b0 & ~1)) * 8;
        for (int i = lane; i < (b1 + 1) / 2 - b0 / 2; i += 32)
          cp16(ring_u + slot * p.st_bytes + p.st_zp + i * 16, zz + i * 16);
      }
      pre.c += p.kc;
      if (pre.c >= c1) {
        pre.c = c0;
        if (++pre.mat == nmat) {
          pre.mat = 0;
          do next_step(pre);
          while (pre.step < hi && !has_tile(pre));
        }
      }
    }
    cp_commit();
  };
  // (The routers' keys lay in the rings; building the lists ended with a barrier.)
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i);

  if (p.early) grid_dependency_wait();
  if (p.mode == kStreamGateUp && blockIdx.x == 0)
    for (int i = tid; i < p.n_counters; i += kThreads) p.counters[i] = 0;

  // Rows that no step writes: slots without an expert (product), every token
  // when nothing is routed (down).
  if (p.mode == kStreamProduct) {
    for (int i = routed + blockIdx.x; i < p.P; i += gridDim.x) {
      const int64_t row = int64_t(order[i]) * p.N;
      for (int n = tid; n < p.N; n += kThreads) {
        if (p.y_f32) static_cast<float *>(p.Y)[row + n] = 0.f;
        else static_cast<uint16_t *>(p.Y)[row + n] = 0;
      }
    }
  } else if (p.mode == kStreamDown && groups == 0) {
    const int64_t n = int64_t(p.M) * p.N;
    for (int64_t i = blockIdx.x * int64_t(kThreads) + tid; i < n; i += int64_t(gridDim.x) * kThreads) {
      if (p.y_f32) static_cast<float *>(p.Y)[i] = 0.f;
      else static_cast<uint16_t *>(p.Y)[i] = 0;
    }
  }

  uint16_t *sx = reinterpret_cast<uint16_t *>(smem + p.off_x);
  const int xterm = p.gt * p.krow;  // elements between the parts
  float *red = reinterpret_cast<float *>(smem + p.off_red);
  int slot = 0, staged = -1, cols = 0, first = 0;

  for (; cur.step < hi; next_step(cur)) {
    if (cur.group != staged) {
      // ---- stage the group's activation rows ------------------------------------
      first = L.off[cur.e] + (cur.group - L.gpre[cur.e]) * p.gt;
      cols = min(p.gt, L.off[cur.e + 1] - first);
      // (Every warp is done with the rows before: the last join had a barrier.)
      staged = cur.group;
      const int pieces = p.K64 * (kChunkK / 8);
      const int planes = p.mode == kStreamDown ? TERMS : 1;
      for (int i = tid; i < planes * cols * pieces; i += kThreads) {
        const int row = i / pieces, k = (i - row * pieces) * 8;
        const int plane = row / cols, col = row - plane * cols;
        const int slot_id = order[first + col];
        uint16_t *dst = sx + col * p.krow + k;
        if (TERMS == 3 && p.mode != kStreamDown) {
          const float *a = static_cast<const float *>(p.A) +
                           int64_t(p.per_slot ? slot_id : slot_id / p.top_k) * p.K;
          float v[8];
          if (p.a_vec && k + 8 <= p.K) {
            const float4 x = *reinterpret_cast<const float4 *>(a + k);
            const float4 y = *reinterpret_cast<const float4 *>(a + k + 4);
            v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
            v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
          } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = k + q < p.K ? a[k + q] : 0.f;
          }
#pragma unroll
          for (int part = 0; part < 3; ++part) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t x = __float_as_uint(v[2 * q]) & 0xFFFF0000u;
              const uint32_t y = __float_as_uint(v[2 * q + 1]) & 0xFFFF0000u;
              v[2 * q] -= __uint_as_float(x);
              v[2 * q + 1] -= __uint_as_float(y);
              w[q] = (x >> 16) | y;
            }
            *reinterpret_cast<uint4 *>(dst + part * xterm) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          const int64_t row0 = p.mode == kStreamDown
                                   ? plane * p.plane + int64_t(slot_id) * p.ldh
                                   : int64_t(p.per_slot ? slot_id : slot_id / p.top_k) * p.K;
          const uint16_t *a = static_cast<const uint16_t *>(p.A) + row0;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (p.a_vec && k + 8 <= p.K) {
            v = __ldcg(reinterpret_cast<const uint4 *>(a + k));
          } else {
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (k + q < p.K) w[q >> 1] |= uint32_t(__ldcg(a + k + q)) << (16 * (q & 1));
            v = make_uint4(w[0], w[1], w[2], w[3]);
          }
          *reinterpret_cast<uint4 *>(dst + plane * xterm) = v;
        }
      }
      __syncthreads();
    }

    // ---- the warp's part of its tile --------------------------------------------
    float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    if (has_tile(cur)) {
      const bool have = g < cols;
      const uint16_t *xrow = sx + (have ? g : 0) * p.krow + 4 * t;
#pragma unroll
      for (int mat = 0; mat < 2; ++mat) {
        if (mat >= nmat) break;
        for (int c = c0; c < c1; c += p.kc) {
          cp_wait<kStages - 2>();
          __syncwarp();  // the stage is there, and every lane is done with the one before
          fetch(slot == 0 ? kStages - 1 : slot - 1);
          const unsigned char *st = ring + slot * p.st_bytes;
          const int n = min(p.kc, c1 - c);
          const int b0 = (c * kChunkK) >> p.bs_log2;
          const unsigned char *sc = st + p.st_scale + g * kEs;
          const unsigned char *sz = st + p.st_zp + (b0 & 1) * 8;
#pragma unroll 1
          for (int i = 0; i < n; ++i) {
            const uint4 w4 = *reinterpret_cast<const uint4 *>(st + i * kChunkBytes + lane * 16);
            const uint32_t wv[4] = {w4.x, w4.y, w4.z, w4.w};
            const uint16_t *xk = xrow + (c + i) * kChunkK;
            constexpr int kBlocks = 4 / SPB;  // scale blocks a chunk touches
            // Blocks past the last hold only k >= K, whose activations are
            // zero: any finite scale serves.
            const int bc = ((c + i) * kChunkK) >> p.bs_log2;
#pragma unroll
            for (int bb = 0; bb < kBlocks; ++bb) {
              const int bi = min(bc + bb, p.nb - 1) - b0;
              float s0, s1;
              if (SF32) {
                s0 = *reinterpret_cast<const float *>(sc + bi * (kTileN * 4));
                s1 = *reinterpret_cast<const float *>(sc + bi * (kTileN * 4) + 32);
              } else {
                s0 = bf16_bits_to_f32(*reinterpret_cast<const uint16_t *>(sc + bi * (kTileN * 2)));
                s1 = bf16_bits_to_f32(
                    *reinterpret_cast<const uint16_t *>(sc + bi * (kTileN * 2) + 16));
              }
              uint32_t z0 = 0x43084308u, z1 = z0;  // 128 + 8
              if (ZP) {
                const uint2 zw = *reinterpret_cast<const uint2 *>(sz + bi * 8);
                z0 = 0x43004300u | (((zw.x >> (4 * g)) & 15u) * 0x10001u);
                z1 = 0x43004300u | (((zw.y >> (4 * g)) & 15u) * 0x10001u);
              }
              float d[4];
#pragma unroll
              for (int jj = 0; jj < SPB; ++jj) {
                const int j = bb * SPB + jj;
                uint32_t wf[4];
                codes_to_bf16x2(wv[j], wf);
                wf[0] = bf16x2_sub(wf[0], z0);
                wf[1] = bf16x2_sub(wf[1], z1);
                wf[2] = bf16x2_sub(wf[2], z0);
                wf[3] = bf16x2_sub(wf[3], z1);
#pragma unroll
                for (int part = 0; part < TERMS; ++part) {
                  uint2 b = make_uint2(0, 0);
                  if (have) b = *reinterpret_cast<const uint2 *>(xk + part * xterm + 16 * j);
                  if (jj == 0 && part == 0) mma_bf16_16816_zero(d, wf, b.x, b.y);
                  else mma_bf16_16816(d, wf, b.x, b.y);
                }
              }
              acc[mat][0] = fmaf(s0, d[0], acc[mat][0]);
              acc[mat][1] = fmaf(s0, d[1], acc[mat][1]);
              acc[mat][2] = fmaf(s1, d[2], acc[mat][2]);
              acc[mat][3] = fmaf(s1, d[3], acc[mat][3]);
            }
          }
          slot = slot == kStages - 1 ? 0 : slot + 1;
        }
      }
    }

    // ---- join the k ranges and store -----------------------------------------------
    // Two buffers by turns: a buffer is written again only after the barrier
    // of the step in between.
    float *rb = red + ((cur.step - lo) & 1) * (kWarps * nmat * kTileN * kCols);
#pragma unroll
    for (int mat = 0; mat < 2; ++mat) {
      if (mat >= nmat) break;
      float *r = rb + (mat * kWarps + warp) * (kTileN * kCols) + 2 * t;
      *reinterpret_cast<float2 *>(r + g * kCols) = make_float2(acc[mat][0], acc[mat][1]);
      *reinterpret_cast<float2 *>(r + (g + 8) * kCols) = make_float2(acc[mat][2], acc[mat][3]);
    }
    __syncthreads();
    const int rows = p.tpu * kTileN, n0 = cur.nstep * rows;
    for (int i = tid; i < rows * cols; i += kThreads) {
      const int col = i / rows, r = i - col * rows, n = n0 + r;
      if (n >= p.N) continue;
      const int slot_id = order[first + col];
      const float *rr = rb + ((r >> 4) * p.ksplit * kTileN + (r & 15)) * kCols + col;
      float v[2] = {0.f, 0.f};
#pragma unroll
      for (int mat = 0; mat < 2; ++mat) {
        if (mat >= nmat) break;
        for (int k2 = 0; k2 < p.ksplit; ++k2)
          v[mat] += rr[(mat * kWarps + k2) * (kTileN * kCols)];
      }
      const int64_t bn = int64_t(cur.e) * p.N + n;
      if (p.mode == kStreamProduct) {
        const float y = p.w[0].bias ? v[0] + p.w[0].bias[bn] : v[0];
        const int64_t o = int64_t(slot_id) * p.N + n;
        if (p.y_f32) static_cast<float *>(p.Y)[o] = y;
        else static_cast<uint16_t *>(p.Y)[o] = static_cast<uint16_t>(bf16_bits(y));
      } else if (p.mode == kStreamGateUp) {
        const float a = p.w[0].bias ? v[0] + p.w[0].bias[bn] : v[0];
        const float u = p.w[1].bias ? v[1] + p.w[1].bias[bn] : v[1];
        float h = a / (1.f + expf(-a)) * u * weights[slot_id];
        for (int pl = 0; pl < p.h_planes; ++pl) {  // parts by truncation
          const uint32_t x = __float_as_uint(h) & 0xFFFF0000u;
          p.hidden[pl * p.plane + int64_t(slot_id) * p.ldh + n] = static_cast<uint16_t>(x >> 16);
          h -= __uint_as_float(x);
        }
      } else {
        p.part[int64_t(slot_id) * p.N + n] =
            p.w[0].bias ? fmaf(weights[slot_id], p.w[0].bias[bn], v[0]) : v[0];
      }
    }
    if (p.mode == kStreamDown && p.counters) {
      // The last group of this column range adds the partials of each token.
      __syncthreads();
      if (tid == 0) {
        __threadfence();
        s_last = atomicAdd(p.counters + cur.nstep, 1u) == static_cast<unsigned>(groups - 1);
        __threadfence();
      }
      __syncthreads();
      if (s_last) {
        const int width = min(rows, p.N - n0);
        for (int i = tid; i < p.M * width; i += kThreads) {
          const int m = i / width, n = n0 + i - m * width;
          float y = 0.f;
          for (int j = 0; j < p.top_k; ++j) {
            const int q = m * p.top_k + j;
            if (L.e[q] < p.E) y += __ldcg(p.part + int64_t(q) * p.N + n);
          }
          const int64_t o = int64_t(m) * p.N + n;
          if (p.y_f32) static_cast<float *>(p.Y)[o] = y;
          else static_cast<uint16_t *>(p.Y)[o] = static_cast<uint16_t>(bf16_bits(y));
        }
      }
    }
  }
  cp_wait<0>();
}

template <int SPB, bool ZP, bool SF32, int TERMS>
cudaError_t launch_one(const StreamParams &p, int grid, int smem, bool pdl, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};
  auto *kernel = stream_kernel<SPB, ZP, SF32, TERMS>;
  const cudaError_t e = ensure_smem_limit(kernel, 227 * 1024 - 1024, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int SPB, bool ZP, bool SF32>
cudaError_t launch_terms(const StreamParams &p, int terms, int grid, int smem, bool pdl,
                         cudaStream_t stream) {
  return terms == 1   ? launch_one<SPB, ZP, SF32, 1>(p, grid, smem, pdl, stream)
         : terms == 2 ? launch_one<SPB, ZP, SF32, 2>(p, grid, smem, pdl, stream)
                      : launch_one<SPB, ZP, SF32, 3>(p, grid, smem, pdl, stream);
}

}  // namespace stream

template <int SPB>
cudaError_t launch_stream(const StreamParams &p, bool zp, bool sf32, int terms, int grid,
                          int smem, bool pdl, cudaStream_t s) {
  using namespace stream;
  if (zp)
    return sf32 ? launch_terms<SPB, true, true>(p, terms, grid, smem, pdl, s)
                : launch_terms<SPB, true, false>(p, terms, grid, smem, pdl, s);
  return sf32 ? launch_terms<SPB, false, true>(p, terms, grid, smem, pdl, s)
              : launch_terms<SPB, false, false>(p, terms, grid, smem, pdl, s);
}

}  // namespace mnb
