// Weight-streaming kernel of the expert layer, for few slots per expert.
//
// Slots are listed by expert and cut into groups of up to 8 that share an
// expert; for each group the kernel streams the expert's packed rows once
// and multiplies them with the group's activation rows:
//   product     Y[p]    = W_e a_p + b_e
//   gate + up   h[p]    = r_p * silu(Wg_e x + bg) * (Wu_e x + bu)
//   down        Y[m]    = sum over the slots of m of (Wd_e h[p] + r_p bd)
// Every weight byte is read once per group. At full memory bandwidth an SM
// receives 24 bytes a cycle, so a 512-byte chunk (64 k of 16 rows) may take
// it about 24 cycles, some 60 to 70 issued instructions: the unpacking, not
// the products, is what competes with the memory.
//
//  * Activations become fp16, each row scaled by a power of two so that its
//    largest magnitude lies in 2^14 .. 2^15 (bf16 values are then exact down
//    to 2^-28 of it); fp32 activations become two fp16 parts, 22 bits.
//  * A code becomes an fp16 by one logic operation per pair: 1024 + q for
//    the low nibble of a byte (tile rows 0-7), 1024 + 16 q for the high one
//    (rows 8-15, whose sums are 16 times too large until the end); one shift
//    per eight codes. For one-part activations the offset comes off a block
//    as a whole: the MMA sums of a block start at minus the offset times the
//    block's sum of activations (staged beside them). That costs rounding of
//    2^-24 of some 200 times the result, far below a bf16 result's; two-part
//    activations (fp32 results) take it off every code exactly.
//  * A block's scale is applied to its fp32 sums: no weight is rounded.
//  * Warps are autonomous: each streams its own sequence of (tile pair, k
//    range) pieces through a private ring of shared-memory stages filled by
//    asynchronous 16-byte copies, across tiles and experts. No barrier is
//    needed to refill a stage, and a lane reads back the very 16 bytes of
//    codes it copied. A warp works on two tiles at a time (gate and up of
//    the same rows, or two neighbours), which share the activation loads.
//  * A step is `tpu` pairs of one group; `ksplit` warps share a pair's k and
//    meet in shared memory, in fixed order (ksplit 1: no meeting, no
//    barrier). CTAs take equal contiguous runs of steps, so a group's
//    activations are staged about once per CTA.
//  * The lists and the rows' largest magnitudes come from a small kernel
//    ahead (moe.cu); the layer is two launches of this one. The second needs
//    nothing from the first but the hidden rows and their magnitudes: it
//    fills its rings before it waits for the first to finish. Down partials
//    go to a workspace, and a launch of its own adds a token's in slot order.
//  * What runs once per launch is kept short and rolled up: fetching
//    instructions is most of the time of a call for one token.
//  * Measured, 8 out of 128 experts, 2560 -> 768 -> 2560, blocks of 32: 16
//    tokens 47 us for gate and up (171 MB, 3.6 TB/s, 54 % of the issue slots)
//    and 28 for down (85 MB, 3.0 TB/s); one token 11 and 9 us, of which the
//    weights (17 and 9 MB) are 4. The first takes some 75 instructions per
//    chunk, 54 % of the issue slots (the MMAs of 8 columns take a quarter of
//    the tensor pipe), and loses a third to the division of work: whole steps
//    over 456 CTAs are 65 chunk times by the rule's own cost (moe.cu) where an
//    even share is 43 (down: 32 and 21). The second is bound by the launches
//    and chains of dependent loads.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "mnb_common.cuh"
#include "mnb_launch.h"
#include "moe_half.cuh"
#include "moe_stream.h"

namespace mnb {
namespace stream {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCols = 8;  // slots per group at most
constexpr int kStages = kStreamStages;
constexpr int kChunks = kStreamChunks;  // chunks per stage and tile

// D += A * B, m16n8k16, fp16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint2 b) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}

// D = A * B + C.
__device__ __forceinline__ void mma_f16_from(float (&d)[4], const uint32_t (&a)[4], uint2 b,
                                             float c0, float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y), "f"(c0), "f"(c1),
        "f"(c2), "f"(c3));
}

// Where a warp stands in its sequence of stages.
struct Cursor {
  int step, e, group, nstep;  // step; its group's expert, id and column step
  int c;                      // first chunk of the stage
};

template <int SPB, bool ZP, bool SF32, int TERMS>
__global__ void __launch_bounds__(kThreads, kStreamCtas) stream_kernel(const StreamParams p) {
  constexpr int kEs = SF32 ? 4 : 2;
  constexpr int kBlocks = 4 / SPB;       // scale blocks (or parts of one) per chunk
  constexpr bool kSums = TERMS == 1;     // the codes' offset goes by the blocks' sums
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  __shared__ float s_unscale[kCols];  // what undoes a column's row scale

  if (!p.early) {
    grid_dependency_wait();
    grid_dependents_launch();
  }
  // ---- this CTA's steps ------------------------------------------------------------
  const int32_t *order = p.order;
  const SlotGroup *grp = p.groups;
  const int groups = *p.n_groups;
  const int64_t total = int64_t(groups) * p.ns;
  const int lo = static_cast<int>(total * blockIdx.x / gridDim.x);
  const int hi = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x);
  const bool gate_up = p.mode == kStreamGateUp;
  const int ks = warp % p.ksplit, tl = warp / p.ksplit;
  const int c0 = p.K64 * ks / p.ksplit, c1 = p.K64 * (ks + 1) / p.ksplit;
  unsigned char *ring = smem + p.off_ring + warp * (kStages * p.st_bytes);
  const uint32_t ring_u = smem_addr(ring);

  auto has_pair = [&](const Cursor &q) { return q.nstep * p.tpu + tl < p.npair; };
  // The tile of matrix `mat` in pair i of an expert (a pair past an odd
  // number of tiles repeats the last one).
  auto tile_of = [&](int i, int mat) { return gate_up ? i : min(2 * i + mat, p.N16 - 1); };
  auto next_step = [&](Cursor &q) {
    ++q.step;
    if (++q.nstep == p.ns) {
      q.nstep = 0;
      ++q.group;
      if (q.step < hi) q.e = grp[q.group].e;
    }
  };
  Cursor pre;  // next stage to fetch
  pre.step = lo;
  pre.group = lo / p.ns;
  pre.nstep = lo - pre.group * p.ns;
  pre.e = lo < hi ? grp[pre.group].e : 0;
  pre.c = c0;
  Cursor cur = pre;
  while (pre.step < hi && !has_pair(pre)) next_step(pre);

  // Sources of the next stage; lane l copies the 16-byte pieces l of the
  // codes of a chunk, and of a stage's scales and zero points (at most 32).
  const uint4 *fw[2];
  const unsigned char *fs[2], *fz[2];
  // First block of the stage at chunk c, and the one past its last.
  auto block_lo = [&](int c) { return SPB == 4 ? (c * kChunkK) >> p.bs_log2 : c * kBlocks; };
  auto block_hi = [&](int c) {
    return SPB == 4 ? ((c * kChunkK - 1) >> p.bs_log2) + 1 : c * kBlocks;
  };
  auto aim = [&] {
#pragma unroll
    for (int mat = 0; mat < 2; ++mat) {
      const int64_t tile = int64_t(pre.e) * p.N16 + tile_of(pre.nstep * p.tpu + tl, mat);
      fw[mat] = p.w[mat].b + (tile * p.K64 + c0) * 32 + lane;
      // Blocks of 64 and more codes: from the tile's start on.
      fs[mat] = p.w[mat].s + (tile * p.nb + (SPB == 4 ? 0 : c0 * kBlocks)) * (kTileN * kEs) +
                lane * 16;
      if (ZP) fz[mat] = p.w[mat].z + tile * p.nbz * 8 + lane * 16;
    }
  };
  if (pre.step < hi) aim();
  uint32_t fdst = ring_u + lane * 16;
  auto fetch = [&] {
    if (pre.step < hi) {
      const int c = pre.c, b0 = block_lo(c);
      const bool two = c + 1 < c1;
      const int need = SPB == 4 ? block_hi(c + (two ? 2 : 1)) - b0 : (two ? 2 : 1) * kBlocks;
      const int have = min(p.nb - b0, need);
#pragma unroll
      for (int mat = 0; mat < 2; ++mat) {
        const uint32_t dst = fdst + mat * p.st_tile;
        cp16(dst, fw[mat]);
        if (two) cp16(dst + kChunkBytes, fw[mat] + 32);
        if (lane < have * kEs)
          cp16(dst + p.st_scale, SPB == 4 ? fs[mat] + b0 * (kTileN * kEs) : fs[mat]);
        if (ZP)  // pairs of words from an even block on
          if (lane < (b0 + have + 1) / 2 - b0 / 2) cp16(dst + p.st_zp, fz[mat] + (b0 / 2) * 16);
        fw[mat] += kChunks * 32;
        if (SPB < 4) fs[mat] += kChunks * kBlocks * (kTileN * kEs);
      }
      // Blocks past the last hold only k >= K, whose activations are zero;
      // their scales are zeros, so that nothing stale meets them.
      if (have < need && lane >= have * kEs && lane < need * kEs)
        for (int mat = 0; mat < 2; ++mat)
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(fdst + mat * p.st_tile +
                                                                      p.st_scale),
                       "r"(0)
                       : "memory");
      fdst += p.st_bytes;
      if (fdst == ring_u + lane * 16 + kStages * p.st_bytes) fdst = ring_u + lane * 16;
      pre.c = c + kChunks;
      if (pre.c >= c1) {
        pre.c = c0;
        do next_step(pre);
        while (pre.step < hi && !has_pair(pre));
        if (pre.step < hi) aim();
      }
    }
    cp_commit();
  };
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) fetch();

  if (p.early) grid_dependency_wait();
  // Rows that no step writes: slots without an expert (product).
  auto store = [&](int64_t i, float v) {
    if (p.y_f32) static_cast<float *>(p.Y)[i] = v;
    else static_cast<uint16_t *>(p.Y)[i] = static_cast<uint16_t>(bf16_bits(v));
  };
  if (p.mode == kStreamProduct) {
    // (Unsigned: the last step may pass 2^31.)
    for (unsigned i = p.offsets[p.E] + blockIdx.x; i < unsigned(p.P); i += gridDim.x) {
      const int64_t row = int64_t(order[i]) * p.N;
      for (int n = tid; n < p.N; n += kThreads) store(row + n, 0.f);
    }
  }

  uint16_t *sx = reinterpret_cast<uint16_t *>(smem + p.off_x);
  const int xterm = p.krow << p.gt_log2;  // elements between the parts
  // Per block and pair of columns 2t, 2t+1: what the MMAs start from, or (ZP)
  // what it is made of: -1024 S and -S.
  float4 *sums = reinterpret_cast<float4 *>(smem + p.off_sums);  // [K64 * kBlocks][4]
  float *red = reinterpret_cast<float *>(smem + p.off_red);
  int slot = 0, staged = -1, cols = 0, first = 0;

  for (; cur.step < hi; next_step(cur)) {
    if (cur.group != staged) {
      // ---- stage the group's activation rows ------------------------------------
      first = grp[cur.group].first;
      cols = grp[cur.group].cols;
      if (staged >= 0) __syncthreads();  // every warp is done with the rows before
      staged = cur.group;
      const int pieces = p.K64 * (kChunkK / 8);
      // The warps share the rows out, so that all rows' loads overlap: 8, 4, 2
      // warps or one to a row.
      const int share_log2 = cols == 1 ? 3 : cols == 2 ? 2 : cols <= 4 ? 1 : 0;
      const int col = warp >> share_log2, part = warp - (col << share_log2);
      if (col < cols) {
        int row = order[first + col];
        if (!p.per_slot) row /= p.top_k;
        const int shift = row_shift(__ldcg(p.tops + row));
        const float f = exp2i(shift);
        if (part == 0 && lane == 0) s_unscale[col] = exp2i(-shift);
        // Pieces are a multiple of 8; a block's sum is formed by up to 8
        // neighbouring lanes.
#pragma unroll 1
        for (int i0 = part * 32; i0 < pieces; i0 += 32 << share_log2) {
          const int i = i0 + lane, k = i * 8;
          float v[8];
          load8(p.A, p.a_f32, p.a_vec, row * p.ld, k, p.K, v);  // zeros past K
          uint32_t hi4[4], lo4[4];
          float sum = 0.f;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float x = v[2 * q] * f, y = v[2 * q + 1] * f;
            hi4[q] = pack_f16x2(x, y);
            const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi4[q]));
            if (kSums) sum += h.x + h.y;
            else lo4[q] = pack_f16x2(x - h.x, y - h.y);
          }
          uint16_t *dst = sx + col * p.krow + k;
          if (i < pieces) {
            *reinterpret_cast<uint4 *>(dst) = make_uint4(hi4[0], hi4[1], hi4[2], hi4[3]);
            if (!kSums)
              *reinterpret_cast<uint4 *>(dst + xterm) = make_uint4(lo4[0], lo4[1], lo4[2], lo4[3]);
          }
          if (kSums) {
            constexpr int kLanes = kChunkK / kBlocks / 8;  // lanes per block
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (i < pieces && lane % kLanes == 0) {
              // Offsets 1024 + z (rows g) and 1024 + 16 z (rows g + 8), z = 8.
              float *q = reinterpret_cast<float *>(sums) + (i / kLanes) * 16 + (col >> 1) * 4 +
                         (col & 1);
              q[0] = (ZP ? -1024.f : -1032.f) * sum;
              q[2] = (ZP ? -1.f : -1152.f) * sum;
            }
          }
        }
      }
      __syncthreads();
    }

    // ---- the warp's part of its pair --------------------------------------------
    float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    if (has_pair(cur)) {
      // Lanes of columns past the group's slots read its first row: their
      // sums are never looked at.
      const uint16_t *xrow = sx + (g < cols ? g : 0) * p.krow + 4 * t;
      for (int c = c0; c < c1; c += kChunks) {
        cp_wait<kStages - 2>();
        __syncwarp();  // the stage is there, and every lane is done with the one before
        fetch();
        const unsigned char *st = ring + slot * p.st_bytes;
        const int b0 = block_lo(c);
        const unsigned char *sc = st + p.st_scale + g * kEs;
        const unsigned char *sz = st + p.st_zp + (b0 & 1) * 8;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          if (i > 0 && c + i >= c1) break;
          const unsigned char *wp = st + lane * 16 + i * kChunkBytes;
          const uint16_t *xk = xrow + (c + i) * kChunkK;
          const float4 *sk = sums + (c + i) * (kBlocks * 4) + t;
          uint32_t wv[2][4];
#pragma unroll
          for (int mat = 0; mat < 2; ++mat) {
            const uint4 w4 = *reinterpret_cast<const uint4 *>(wp + mat * p.st_tile);
            wv[mat][0] = w4.x; wv[mat][1] = w4.y; wv[mat][2] = w4.z; wv[mat][3] = w4.w;
          }
          const int bi = SPB == 4 ? (((c + i) * kChunkK) >> p.bs_log2) - b0 : i * kBlocks;
          const unsigned char *scb = sc + bi * (kTileN * kEs);
          const unsigned char *szb = sz + bi * 8;
#pragma unroll
          for (int bb = 0; bb < kBlocks; ++bb) {
            float d[2][4];
            uint32_t z0[2], z1[2], y1[2];
            float4 sv;
            if (kSums) sv = sk[bb * 4];
#pragma unroll
            for (int mat = 0; mat < 2; ++mat) {
              uint32_t q0 = 8, q1 = 8;
              if (ZP) {
                const uint2 zw =
                    *reinterpret_cast<const uint2 *>(szb + mat * p.st_tile + bb * 8);
                q0 = (zw.x >> (4 * g)) & 15u;
                q1 = (zw.y >> (4 * g)) & 15u;
              }
              if (kSums && ZP) {
                // z and 16 z as floats: 2^23 + n in bits, less 2^23.
                const float f0 = __uint_as_float(0x4B000000u | q0) - 8388608.f;
                const float f1 = __uint_as_float(0x4B000000u | (q1 << 4)) - 8388608.f;
                d[mat][0] = fmaf(f0, sv.z, sv.x);
                d[mat][1] = fmaf(f0, sv.w, sv.y);
                d[mat][2] = fmaf(f1, sv.z, sv.x);
                d[mat][3] = fmaf(f1, sv.w, sv.y);
              } else if (!kSums) {
                // 1024 + z, and -(64 + z) for the sixteenth of 1024 + 16 q.
                z0[mat] = 0x64006400u | (q0 * 0x10001u);
                z1[mat] = f16x2_sub(0x64006400u | (q1 * 0x10001u), 0x63806380u);  // 64 + z
                y1[mat] = z1[mat] ^ 0x80008000u;
                d[mat][0] = d[mat][1] = d[mat][2] = d[mat][3] = 0.f;
              }
            }
#pragma unroll
            for (int jj = 0; jj < SPB; ++jj) {
              const int j = bb * SPB + jj;
              uint2 xb[TERMS];
#pragma unroll
              for (int part = 0; part < TERMS; ++part)
                xb[part] = *reinterpret_cast<const uint2 *>(xk + part * xterm + 16 * j);
#pragma unroll
              for (int mat = 0; mat < 2; ++mat) {
                uint32_t wf[4];
                codes_to_f16x2(wv[mat][j], wf);
                if (!kSums) {
                  constexpr uint32_t kSixteenth = 0x2C002C00u;  // 2^-4
                  wf[0] = f16x2_sub(wf[0], z0[mat]);
                  wf[1] = f16x2_fma(wf[1], kSixteenth, y1[mat]);
                  wf[2] = f16x2_sub(wf[2], z0[mat]);
                  wf[3] = f16x2_fma(wf[3], kSixteenth, y1[mat]);
                }
#pragma unroll
                for (int part = 0; part < TERMS; ++part) {
                  if (kSums && !ZP && jj == 0)
                    mma_f16_from(d[mat], wf, xb[part], sv.x, sv.y, sv.z, sv.w);
                  else
                    mma_f16(d[mat], wf, xb[part]);
                }
              }
            }
#pragma unroll
            for (int mat = 0; mat < 2; ++mat) {
              const unsigned char *sm = scb + mat * p.st_tile + bb * (kTileN * kEs);
              float s0, s1;
              if (SF32) {
                s0 = *reinterpret_cast<const float *>(sm);
                s1 = *reinterpret_cast<const float *>(sm + 32);
              } else {
                s0 = bf16_bits_to_f32(*reinterpret_cast<const uint16_t *>(sm));
                s1 = bf16_bits_to_f32(*reinterpret_cast<const uint16_t *>(sm + 16));
              }
              acc[mat][0] = fmaf(s0, d[mat][0], acc[mat][0]);
              acc[mat][1] = fmaf(s0, d[mat][1], acc[mat][1]);
              acc[mat][2] = fmaf(s1, d[mat][2], acc[mat][2]);
              acc[mat][3] = fmaf(s1, d[mat][3], acc[mat][3]);
            }
          }
        }
        slot = slot == kStages - 1 ? 0 : slot + 1;
      }
    }

    // ---- store ---------------------------------------------------------------------
    // The warps of a pair meet in shared memory, a warp that has its pair to
    // itself meets its own lanes there. Two buffers by turns: a buffer is
    // written again only after the barrier of the step in between.
    constexpr float kUpper = kSums ? 0.0625f : 1.f;  // rows 8-15 of a tile
    const bool alone = p.ksplit == 1;
    const int gt = 1 << p.gt_log2;
    float *rb = red + (((cur.step - lo) & 1) * 2 * kWarps << p.gt_log2) * kTileN;
#pragma unroll
    for (int mat = 0; mat < 2; ++mat) {
      float *r = rb + ((mat * kWarps + warp) * kTileN + g) * gt;
#pragma unroll
      for (int o = 0; o < 2; ++o)
        if (2 * t + o < cols) {
          r[2 * t + o] = acc[mat][o];
          r[8 * gt + 2 * t + o] = acc[mat][2 + o] * kUpper;
        }
    }
    if (alone) __syncwarp();
    else __syncthreads();
    // Columns of a pair: 16 (of both matrices) for gate and up, else 32. Item
    // i: row r of the step (of the warp's pair), column `col`.
    const int wide_log2 = gate_up ? 4 : 5;
    const int rows_log2 = alone ? wide_log2 : wide_log2 + p.tpu_log2, rows = 1 << rows_log2;
    const int part0 = cur.nstep * p.tpu + (alone ? warp : 0), n0 = part0 << wide_log2;
#pragma unroll 1
    for (int i0 = alone ? 0 : warp * 32; i0 < cols << rows_log2; i0 += alone ? 32 : kThreads) {
      const int i = i0 + lane, col = i >> rows_log2, r = i & (rows - 1), n = n0 + r;
      uint32_t top = 0;  // hidden value's magnitude
      int id = 0;
      if (col < cols && n < p.N) {
        const int w0 = alone ? warp : (r >> wide_log2) * p.ksplit;
        const float *rr =
            rb + (((gate_up ? 0 : (r >> 4) & 1) * kWarps + w0) * kTileN + (r & 15)) * gt + col;
        float v0 = 0.f, v1 = 0.f;
#pragma unroll 1
        for (int k2 = 0; k2 < p.ksplit; ++k2, rr += kTileN * gt) {
          v0 += rr[0];
          if (gate_up) v1 += rr[kWarps * kTileN * gt];
        }
        const float f = s_unscale[col];
        id = order[first + col];
        const int64_t bn = int64_t(cur.e) * p.N + n;
        v0 *= f;
        const float b0 = p.w[0].bias ? p.w[0].bias[bn] : 0.f;
        if (gate_up) {
          v0 += b0;
          v1 *= f;
          if (p.w[1].bias) v1 += p.w[1].bias[bn];
          const float h = v0 / (1.f + expf(-v0)) * v1 * p.weights[id];
          p.hidden[id * p.ldh + n] = h;
          top = __float_as_uint(h) & 0x7FFFFFFFu;
        } else if (p.mode == kStreamProduct) {
          store(int64_t(id) * p.N + n, v0 + b0);
        } else {
          p.part[int64_t(id) * p.N + n] = b0 != 0.f ? fmaf(p.weights[id], b0, v0) : v0;
        }
      }
      if (gate_up) {  // 16 lanes share a column
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        if ((lane & 15) == 0 && top) atomicMax(p.hidden_tops + id, top);
      }
    }
  }
  cp_wait<0>();
}

template <int SPB, bool ZP, bool SF32, int TERMS>
cudaError_t launch_one(const StreamParams &p, int grid, int smem, bool pdl, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};
  auto *kernel = stream_kernel<SPB, ZP, SF32, TERMS>;
  const cudaError_t e = ensure_smem_limit(kernel, 226 * 1024 + 512, done);
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

}  // namespace stream

template <int SPB>
cudaError_t launch_stream(const StreamParams &p, bool zp, bool sf32, int terms, int grid,
                          int smem, bool pdl, cudaStream_t s) {
  using namespace stream;
  auto one = [&](auto *fn) { return fn(p, grid, smem, pdl, s); };
  if (terms == 1)
    return zp ? one(sf32 ? launch_one<SPB, true, true, 1> : launch_one<SPB, true, false, 1>)
              : one(sf32 ? launch_one<SPB, false, true, 1> : launch_one<SPB, false, false, 1>);
  return zp ? one(sf32 ? launch_one<SPB, true, true, 2> : launch_one<SPB, true, false, 2>)
            : one(sf32 ? launch_one<SPB, false, true, 2> : launch_one<SPB, false, false, 2>);
}

}  // namespace mnb
