// Tensor-core (tcgen05 / TMEM) kernel of the expert layer, for many slots.
//
// One unit of work is a group of up to 192 slots that share an expert times
// two column tiles of the expert's weight, one for each CTA of a pair: 128
// weight rows each (64 of gate and the same 64 of up, or 128 of one matrix).
// The weight rows are the MMA's A operand (cta_group::2, M = 256), the slots
// its columns (N = slots rounded up to 32), so ragged lists cost little:
//   D[row, slot] = sum_k w[row, k] x[slot, k]
//
//  * A comes from TMEM. A lane's 16 fp16 pairs of a packed 16 x 64 chunk are
//    exactly the registers of a 16x256b TMEM store, so the unpacking warps
//    write each dequantised chunk with one store, without shared memory,
//    swizzles or a proxy fence: 64 TMEM columns per stage of two chunks (128
//    k), two stages. The other 384 columns are two accumulators: a unit is
//    stored while the next one is computed. One CTA per SM.
//  * Weights are fp16, w' = (q - z) s' 2^-24, with each row's scales brought
//    to at most 2^15 by a power of two that the epilogue undoes: one rounding
//    of 2^-11 of the weight, or 2^-15 of its row's largest scale where that
//    is more, and for odd z above 8 one of z s' beside it: an eighth of a
//    bf16 weight's. A code's fp16 form costs one mask (see the unpacking).
//  * B are fp16 activation rows, scaled by a power of two per row, in the
//    order of the lists: TMA tiles of 32 rows x 64 k, 128-byte swizzle. Each
//    CTA of a pair loads half of a group's rows: alone, with 128 weight rows
//    and all of the slots, it would take 64 bytes of activations a cycle.
//  * Hidden values leave as fp32, the router's weight applied; a small kernel
//    makes them fp16 rows scaled by their own largest value, as the streaming
//    kernel does. (A scale from a bound known ahead, such as 15 s |x|_1 for
//    gate and for up, saves that kernel, but rows far below their bound lose
//    their bits: all of them where SiLU makes a row 2^-40 of it.) Down partials
//    are fp16, scaled by the bound 15 s K max|h| of their hidden row; they are
//    added per token by a kernel that follows.
//  * Warps 0-15 unpack, each its own tile's codes and scales from a private
//    ring of asynchronous copies, in two groups that alternate stages; warps
//    16-23 store; one warp each issues the TMA loads, issues the MMAs, and
//    gathers what a unit's columns need for the epilogue.
//  * What bounds it is the unpacking: per 16 x 64 chunk a warp takes about 117
//    instructions (23 to fetch, 48 to unpack, 20 of them for the scales, the
//    rest for a stage's waits, store and arrival; 140 with zero points). They
//    take 52 to 59 % of the issue slots: a stage's two chunks follow one
//    another through one set of registers, and four unpacking warps a
//    scheduler do not fill the gaps. Lists above 192 slots take several
//    groups, and every group unpacks the weights again. Measured, 8 out of 128
//    experts, 2560 -> 768 -> 2560, 4096 tokens: gate and up 207 us = 1250
//    TFLOP/s, tensor pipe 59 % busy, down 139 us = 930; 6 out of 64, 2560 ->
//    1408 -> 2560, 192 tokens: 102 us = 2.4 TB/s of weights, and 56. Groups
//    of 64 slots with 6 TMEM stages and 8 activation stages, for few slots per
//    expert, were no faster (before hidden rows were fp32: 166.6 against 165.5
//    us for the layer at a mean of 4, 183.0 against 181.0 at 16).
#include <cuda_fp16.h>

#include <algorithm>

#include "mnb_common.cuh"
#include "mnb_launch.h"
#include "moe.h"
#include "moe_half.cuh"
#include "moe_tile.h"
#include "umma.cuh"

namespace mnb {

__device__ unsigned int g_fault_moe = 0;

namespace {

constexpr int kDqGroups = 2;  // groups of unpacking warps: group i takes the stages i, i + 2, ..
constexpr int kDqGroupWarps = 8;
constexpr int kDqWarps = kDqGroups * kDqGroupWarps;  // warps 0-15 unpack
constexpr int kEpWarps = 8;                          // warps 16-23 store
constexpr int kTmaWarp = kDqWarps + kEpWarps, kMmaWarp = kTmaWarp + 1, kColWarp = kTmaWarp + 2;
constexpr int kThreads = 32 * (kTmaWarp + 3);
constexpr int kChunks = 2;    // 64-wide k chunks per stage
constexpr int kAStages = kDqGroups;  // TMEM A stages (64 columns each), one per group
constexpr int kBStages = 5;   // activation stages
constexpr int kRing = 3;      // weight stages per warp in flight
constexpr int kBChunkBytes = kTileSlots / 2 * 128;  // a CTA's half of the slots
constexpr int kBStageBytes = kChunks * kBChunkBytes;
constexpr int kTmemCols = 512;  // A, and two accumulators of kTileSlots columns
static_assert(kAStages * kChunks * 32 + 2 * kTileSlots == kTmemCols, "all of TMEM");

// D fp32, A and B fp16, K-major, M = 256 over the pair.
__host__ __device__ constexpr uint32_t idesc_f16(int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (16u << 24);
}
__device__ __forceinline__ int columns_of(int slots) { return (slots + 31) & ~31; }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Address of this CTA's shared variable `p` in CTA `rank` of the pair.
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
  return r;
}
// Arrival on a barrier of either CTA. What it publishes lies in tensor memory
// (stores waited for and fenced before it) or in shared memory that TMA
// wrote: nothing a cluster-scope release of this thread's writes would add.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// Bounded wait that sleeps in the hardware for up to 50 us at a time: a warp
// that polls takes issue slots from the unpacking. At most about a second.
__device__ __forceinline__ bool mbar_sleep(uint64_t *bar, uint32_t parity) {
  for (uint32_t i = 0; i < 20000u; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(50000u)
        : "memory");
    if (ok) return true;
  }
  return false;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

// D += A x B^T over the pair: each CTA's 128 rows of A in its tensor memory,
// each CTA's half of B's rows in its shared memory, at the same offsets.
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrival, once the MMAs issued so far are complete, on the barrier at `bar`'s
// offset in each CTA of `mask`.
__device__ __forceinline__ void umma_commit(uint64_t *bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_addr(bar)),
      "h"(mask)
      : "memory");
}
// 16 lanes x 32 columns: lane (g, t) writes, for j < 4, columns 8j + 2t and
// 8j + 2t + 1 of TMEM lanes g (r[4j], r[4j+1]) and g + 8 (r[4j+2], r[4j+3]).
__device__ __forceinline__ void tmem_st_16x64(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

struct Layout {  // shared memory, from a 1024-byte aligned base
  int scale, zp, fac, stage_bytes;  // a warp's weight stage
  int off_ring, off_col, off_bar, total;
};
// What the epilogue needs of a column: a undoes the activation row's scale
// (down: and applies the output's); b is the slot's weight times the output's
// scale (down); out the slot (product).
struct Columns {
  float2 ab[kTileSlots];
  int out[kTileSlots];
};

// Scale blocks of a stage (128 k; stages start at multiples of it), and of a
// step of all groups.
template <int BS>
constexpr int kStageBlocks = BS <= kChunks * kChunkK ? kChunks * kChunkK / BS : 1;

template <int BS, bool SF32, bool ZP>
__host__ __device__ constexpr Layout make_layout() {
  Layout l{};
  l.scale = kChunks * kChunkBytes;
  l.zp = l.scale + kStageBlocks<BS> * kTileN * (SF32 ? 4 : 2);
  l.fac = l.zp + (ZP ? (kStageBlocks<BS> / 2 + 1) * 16 : 0);
  l.stage_bytes = l.fac + 8 * 8;
  l.off_ring = kBStages * kBStageBytes;
  l.off_col = l.off_ring + kDqWarps * kRing * l.stage_bytes;
  l.off_bar = l.off_col + 2 * static_cast<int>(sizeof(Columns));
  l.total = l.off_bar + 256;
  return l;
}

// Smallest e with x < 2^e, for x >= 0 (0: a very small one; not finite: 128).
__device__ __forceinline__ int expo(float x) {
  return static_cast<int>(__float_as_uint(x) >> 23) - 126;
}

template <int BS, bool ZP, bool SF32>
__global__ void __launch_bounds__(kThreads, 1) tile_kernel(const __grid_constant__ TileParams p) {
  constexpr Layout kL = make_layout<BS, SF32, ZP>();
  constexpr int kEs = SF32 ? 4 : 2;
  constexpr int kBlk = BS < kChunkK ? kChunkK / BS : 1;  // blocks per chunk
  constexpr int kSpb = 4 / kBlk;                         // 16-wide steps per block
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint64_t *afull = reinterpret_cast<uint64_t *>(smem + kL.off_bar);
  uint64_t *aempty = afull + kAStages;
  uint64_t *bfull = aempty + kAStages;
  uint64_t *bempty = bfull + kBStages;
  uint64_t *cfull = bempty + kBStages;
  uint64_t *cempty = cfull + 2;
  uint64_t *dfull = cempty + 2;
  uint64_t *dempty = dfull + 2;
  uint64_t *done = dempty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  Columns *cols2 = reinterpret_cast<Columns *>(smem + kL.off_col);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  if (tid == 0) {
    for (int i = 0; i < kAStages; ++i) {
      mbar_init(afull + i, 2 * kDqGroupWarps);  // both CTAs' warps, at CTA 0
      mbar_init(aempty + i, 1);
    }
    for (int i = 0; i < kBStages; ++i) {
      mbar_init(bfull + i, rank == 0 ? 2 : 1);  // at CTA 0, CTA 1's half as well
      mbar_init(bempty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(cfull + i, 1);
      mbar_init(cempty + i, kEpWarps);
      mbar_init(dfull + i, 1);
      mbar_init(dempty + i, 2 * kEpWarps);  // both CTAs' warps, at CTA 0
    }
    mbar_init(done, 1);
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before any remote arrival
  tc_fence_after();
  const uint32_t tmem_a = *tmem_slot, tmem_d = tmem_a + kAStages * kChunks * 32;

  grid_dependency_wait();
  grid_dependents_launch();
  // A pair of CTAs takes two neighbouring column tiles of a group.
  const int np = (p.ntile + 1) / 2, units = *p.n_groups * np;
  const int u0 = blockIdx.x >> 1, du = gridDim.x >> 1;
  const bool gate_up = p.mode == kStreamGateUp;
  const int stages = (p.K64 + kChunks - 1) / kChunks;  // per unit

  if (warp == kTmaWarp) {
    // ---- TMA: activation rows (issued as the MMAs are, below) ---------------------
    int s = 0, it = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = u0; u < units && ok; u += du) {
      const SlotGroup sg = p.groups[u / np];
      const int cols = __shfl_sync(0xffffffffu, sg.cols, 0), half = columns_of(cols) / 2;
      const int first = __shfl_sync(0xffffffffu, sg.first, 0) + static_cast<int>(rank) * half;
      const int boxes = (half + kTileBox - 1) / kTileBox;
      for (int kb = 0; kb < p.K64; kb += kChunks, ++it) {
        if (it >= kBStages) ok = __all_sync(0xffffffffu, mbar_sleep(bempty + s, phase ^ 1));
        if (!ok) {
          if (lane == 0) record_fault(&g_fault_moe, kFaultMoeWait);
          break;
        }
        const int nc = min(kChunks, p.K64 - kb);
        if (elect_one()) {
          mbar_arrive_expect_tx(bfull + s, nc * boxes * kTileBox * 128);
          for (int c = 0; c < nc; ++c)
            for (int b = 0; b < boxes; ++b)
              tma_load_2d(smem + s * kBStageBytes + c * kBChunkBytes + b * kTileBox * 128, &p.tmb,
                          (kb + c) * kChunkK, first + b * kTileBox, bfull + s);
        }
        __syncwarp();
        if (++s == kBStages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    // Given up: the copies in flight land before the CTA leaves.
    if (!ok)
      for (int i = max(0, it - kBStages); i < it; ++i)
        mbar_sleep(bfull + i % kBStages, (i / kBStages) & 1);
  } else if (warp == kMmaWarp) {
    bool ok = true;
    if (rank == 0) {  // ---- MMAs of the pair ---------------------------------------------
      // The whole warp goes round and one elected lane issues, so that the
      // instructions' operands stay in uniform registers: moving them there
      // for every MMA took a thread on its own 100 cycles each.
      int as = 0, bs = 0, n = 0;
      uint32_t aphase = 0, bphase = 0;
      const uint64_t desc0 = smem_desc_sw128(smem_addr(smem));
      int slots = u0 < units ? p.groups[u0 / np].cols : 0;
      for (int u = u0; u < units && ok; u += du, ++n) {
        const uint32_t idesc = idesc_f16(columns_of(__shfl_sync(0xffffffffu, slots, 0)));
        const uint32_t d = tmem_d + (n & 1) * kTileSlots;
        if (u + du < units) slots = p.groups[(u + du) / np].cols;
        if (n >= 2) ok = __all_sync(0xffffffffu, mbar_sleep(dempty + (n & 1), (n / 2 - 1) & 1));
        tc_fence_after();
        for (int kb = 0; kb < p.K64 && ok; kb += kChunks) {
          ok = mbar_sleep(bfull + bs, bphase) && mbar_sleep(afull + as, aphase);
          ok = __all_sync(0xffffffffu, ok);
          tc_fence_after();
          const uint32_t ta = tmem_a + as * (kChunks * 32);
          const uint64_t desc = desc0 + bs * (kBStageBytes >> 4);
          if (ok && elect_one()) {
            // A chunk's MMAs step A by 8 columns and B's descriptor by 32 bytes.
            umma_ts(d, ta, desc, idesc, kb);
#pragma unroll
            for (int kk = 1; kk < 4; ++kk) umma_ts(d, ta + kk * 8, desc + kk * 2, idesc, 1);
            if (kb + 1 < p.K64)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_ts(d, ta + 32 + kk * 8, desc + (kBChunkBytes >> 4) + kk * 2, idesc, 1);
            umma_commit(aempty + as, 3);
            umma_commit(bempty + bs, 3);
          }
          __syncwarp();
          if (++as == kAStages) {
            as = 0;
            aphase ^= 1;
          }
          if (++bs == kBStages) {
            bs = 0;
            bphase ^= 1;
          }
        }
        if (ok && elect_one()) umma_commit(dfull + (n & 1), 3);
        __syncwarp();
      }
      // Every MMA issued is complete before the tensor memory is released.
      if (elect_one()) umma_commit(done, 1);
      __syncwarp();
      if (!__all_sync(0xffffffffu, mbar_sleep(done, 0)) || !ok)
        if (lane == 0) record_fault(&g_fault_moe, kFaultMoeWait);
    } else if (lane == 0) {  // ---- CTA 1: tells CTA 0 that its half has landed -----------
      const uint32_t peer = cluster_addr(bfull, 0);
      int it = 0;
      for (int u = u0; u < units && ok; u += du)
        for (int kb = 0; kb < p.K64; kb += kChunks, ++it) {
          ok = mbar_sleep(bfull + it % kBStages, (it / kBStages) & 1);
          if (!ok) break;
          mbar_arrive_cluster(peer + 8 * (it % kBStages));
        }
      // CTA 0's commits arrive on this CTA's barriers as well, and nothing here
      // waits for the last of them: this CTA must not be gone when they land.
      for (int i = max(0, it - kBStages); i < it && ok; ++i)
        ok = mbar_sleep(bempty + i % kBStages, (i / kBStages) & 1);
      for (int i = max(0, it - kAStages); i < it && ok; ++i)
        ok = mbar_sleep(aempty + i % kAStages, (i / kAStages) & 1);
      if (!ok) record_fault(&g_fault_moe, kFaultMoeWait);
    }
  } else if (warp == kColWarp) {
    // ---- columns ------------------------------------------------------------------
    int n = 0;
    for (int u = u0; u < units; u += du, ++n) {
      if (n >= 2 && !mbar_sleep(cempty + (n & 1), (n / 2 - 1) & 1)) {
        if (lane == 0) record_fault(&g_fault_moe, kFaultMoeWait);
        break;
      }
      const SlotGroup sg = p.groups[u / np];
      Columns &cl = cols2[n & 1];
      auto most = [&](const float *v) { return v ? v[sg.e] : 0.f; };
      for (int c = lane; c < sg.cols; c += 32) {
        const int place = sg.first + c, id = p.order[place];
        float a = p.unscale[place], b = 1.f;
        if (p.mode != kStreamProduct) b = p.weights[id];
        if (p.mode == kStreamDown) {
          // |sum| <= 15 s K max|h|, and the bias; a hidden row's largest value
          // is below 2^(15 - p.shift).
          const int e = max(expo(15.01f * most(p.ts[0].smax) *
                                 static_cast<float>(p.K64 * kChunkK) * 32768.f) - p.shift[place],
                            expo(most(p.ts[0].bmax) * b)) + 1;
          // a = 2^(shift - p.shift) stays finite: an expert of zero scales has
          // a bound of 0, and 0 * inf would be NaN.
          const int shift = max(-126, min(min(126, 126 + p.shift[place]), 15 - e));
          a *= exp2i(shift);
          b *= exp2i(shift);
          if (u % np == 0 && rank == 0) p.out_unscale[place] = exp2i(-shift);
        }
        cl.ab[c] = make_float2(a, b);
        cl.out[c] = id;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(cfull + (n & 1));
    }
  } else if (warp < kDqWarps) {
    // ---- unpacking ------------------------------------------------------------------
    const int g = lane >> 2, grp = warp / kDqGroupWarps;
    // TMEM lanes 32 quarter + 16 half ..
    const int quarter = warp & 3, half = (warp % kDqGroupWarps) >> 2;
    unsigned char *ring = smem + kL.off_ring + warp * (kRing * kL.stage_bytes);
    const uint32_t ring_u = smem_addr(ring);
    const int mat = gate_up ? half : 0;
    // The tile of a unit this warp unpacks (past the last: the last again,
    // its rows are never stored).
    auto tile_of = [&](int e, int pair) {
      const int nt = 2 * pair + static_cast<int>(rank);
      const int i = gate_up ? 4 * nt + quarter : 8 * nt + 2 * quarter + half;
      return int64_t(e) * p.N16 + min(i, p.N16 - 1);
    };
    // Fetch cursor: unit, stage in it, ring slot, sources; the expert of the
    // unit after its own is loaded a unit ahead, the row factors as it enters
    // a unit. Lane l copies the 16-byte pieces l of a chunk's codes, and of a
    // stage's scales and zero points (at most 32 each).
    int fu = u0, fj = grp, fslot = 0, ne = 0;
    float nf0 = 0.f, nf1 = 0.f;
    const uint4 *fw = nullptr;
    const unsigned char *fs = nullptr, *fz = nullptr;
    auto block_of = [&](int j) { return j * (kChunks * kChunkK) / BS; };
    auto aim = [&] {
      const int64_t tile = tile_of(ne, fu % np);
      fw = p.w[mat].b + (tile * p.K64 + fj * kChunks) * 32 + lane;
      fs = p.w[mat].s + (tile * p.nb + block_of(fj)) * (kTileN * kEs) + lane * 16;
      if (ZP) fz = p.w[mat].z + tile * p.nbz * 8 + lane * 16;
      nf0 = p.ts[mat].fac[tile * kTileN + g];
      nf1 = p.ts[mat].fac[tile * kTileN + g + 8] * 0.0625f;  // high nibbles: 16 q
      if (fu + du < units) ne = p.groups[(fu + du) / np].e;
    };
    // Into the unit that holds the stage fj counts past this one's end.
    auto settle = [&] {
      bool moved = false;
      while (fj >= stages && fu < units) {
        fj -= stages;
        fu += du;
        if (moved && fu < units) ne = p.groups[fu / np].e;  // (units of one stage)
        moved = true;
      }
      if (moved && fu < units) aim();
    };
    auto fetch = [&] {
      if (fu < units) {
        const uint32_t off = fslot * kL.stage_bytes, dst = ring_u + off + lane * 16;
        cp16(dst, fw);
        const int b0 = block_of(fj);
        if (fj + 1 < stages) {
          cp16(dst + kChunkBytes, fw + 32);
          if (lane < kStageBlocks<BS> * kEs) cp16(dst + kL.scale, fs);
        } else {
          // The last stage may have one chunk, and blocks past the last: those
          // hold only k >= K, whose activations are zero, and get scales 0.
          if (fj * kChunks + 1 < p.K64) cp16(dst + kChunkBytes, fw + 32);
          const int b1 = min(p.nb - b0, kStageBlocks<BS>);
          if (lane < b1 * kEs) cp16(dst + kL.scale, fs);
          else if (lane < kStageBlocks<BS> * kEs)
            *reinterpret_cast<uint4 *>(ring + off + kL.scale + lane * 16) =
                make_uint4(0, 0, 0, 0);
        }
        // Pairs of zero-point words from an even block on.
        if (ZP && lane < (min(p.nb, b0 + kStageBlocks<BS>) + 1) / 2 - b0 / 2)
          cp16(dst + kL.zp, fz + (b0 / 2) * 16);
        if ((lane & 3) == 0)
          *reinterpret_cast<float2 *>(ring + off + kL.fac + g * 8) = make_float2(nf0, nf1);
        fslot = fslot == kRing - 1 ? 0 : fslot + 1;
        fw += kDqGroups * kChunks * 32;
        fs += kDqGroups * kChunks * kChunkK / BS * (kTileN * kEs);
        fj += kDqGroups;
        if (fj >= stages) settle();
      }
      cp_commit();
    };
    static_assert(kDqGroups * kChunks * kChunkK % BS == 0, "whole blocks per step");
    if (fu < units) {
      ne = p.groups[fu / np].e;
      aim();
      if (fj >= stages) settle();
    }
    for (int i = 0; i < kRing - 1; ++i) fetch();

    const uint32_t afull0 = cluster_addr(afull, 0);
    int slot = 0, j = grp, use = 0;  // use: of this group's TMEM stage
    bool ok = true;
    for (int u = u0; u < units && ok; u += du, j -= stages) {
      for (; j < stages; j += kDqGroups, ++use) {
        cp_wait<kRing - 2>();
        __syncwarp();  // the stage is there, and every lane is done with the one before
        fetch();
        const unsigned char *st = ring + slot * kL.stage_bytes;
        slot = slot == kRing - 1 ? 0 : slot + 1;
        const int odd = ZP ? block_of(j) & 1 : 0;  // the first word of its pair, or the second
        const float2 f = *reinterpret_cast<const float2 *>(st + kL.fac + g * 8);
        auto unpack = [&](int cc, uint32_t (&r)[16]) {
          const uint4 w4 = *reinterpret_cast<const uint4 *>(st + cc * kChunkBytes + lane * 16);
          const uint32_t wv[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int bb = 0; bb < kBlk; ++bb) {
            // The block's place in the stage.
            const int bi = BS > kChunkK ? 0 : cc * kBlk + bb;
            float s0, s1;
            if (SF32) {
              const float *sc = reinterpret_cast<const float *>(st + kL.scale) + bi * kTileN + g;
              s0 = sc[0];
              s1 = sc[8];
            } else {
              const uint16_t *sc =
                  reinterpret_cast<const uint16_t *>(st + kL.scale) + bi * kTileN + g;
              s0 = bf16_bits_to_f32(sc[0]);
              s1 = bf16_bits_to_f32(sc[8]);
            }
            s0 *= f.x;
            s1 *= f.y;
            // s' = s times the row's factor, at most 2^15. A code under its mask
            // is the fp16 subnormal q 2^-24 (high nibbles: q 2^-20 with s' / 16),
            // so that one fused multiply-add gives (q - z) s' 2^-24, rounded
            // once. z s' is exact for z up to 8 and even z (bf16 scales).
            const uint32_t h0 = pack_f16x2(s0, s0), h1 = pack_f16x2(s1, s1);
            uint32_t z0, z1;
            if (ZP) {
              const uint2 zw = *reinterpret_cast<const uint2 *>(st + kL.zp + (bi + odd) * 8);
              // -z 2^-24 as a pair; for rows g + 8, -z 2^-20.
              z0 = f16x2_mul(h0, 0x80008000u | (((zw.x >> (4 * g)) & 15u) * 0x10001u));
              z1 = f16x2_mul(h1, 0x80008000u | (((zw.y >> (4 * g)) & 15u) * 0x100010u));
            } else {
              z0 = f16x2_mul(h0, 0x80088008u);
              z1 = f16x2_mul(h1, 0x80808080u);
            }
            auto scaled = [&](uint32_t c, uint32_t z, uint32_t h, float s, uint32_t zs) {
              if (!SF32) return f16x2_fma(c, h, z);
              // fp32 scales: from exact q - z, rounded once as well.
              const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&c));
              const float2 n = __half22float2(*reinterpret_cast<const __half2 *>(&zs));
              return pack_f16x2((v.x + n.x) * s, (v.y + n.y) * s);
            };
            uint32_t n0 = 0x80088008u, n1 = 0x80808080u;  // -z as the codes are held
            if (SF32 && ZP) {
              const uint2 zw = *reinterpret_cast<const uint2 *>(st + kL.zp + (bi + odd) * 8);
              n0 = 0x80008000u | (((zw.x >> (4 * g)) & 15u) * 0x10001u);
              n1 = 0x80008000u | (((zw.y >> (4 * g)) & 15u) * 0x100010u);
            }
#pragma unroll
            for (int jj = 0; jj < kSpb; ++jj) {
              const int j = bb * kSpb + jj;
              const uint32_t w = wv[j], v = w >> 8;
              r[4 * j] = scaled(w & 0x000F000Fu, z0, h0, s0, n0);
              r[4 * j + 1] = scaled(v & 0x000F000Fu, z0, h0, s0, n0);
              r[4 * j + 2] = scaled(w & 0x00F000F0u, z1, h1, s1, n1);
              r[4 * j + 3] = scaled(v & 0x00F000F0u, z1, h1, s1, n1);
            }
          }
        };
        // One chunk after the other through the same registers: at 72 a thread
        // there is no room for two sets, so the second is unpacked behind the
        // first one's store.
        uint32_t r0[16];
        unpack(0, r0);
        if (use > 0 && !mbar_sleep(aempty + grp, (use - 1) & 1)) {
          record_fault(&g_fault_moe, kFaultMoeWait);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t ta = tmem_a + grp * (kChunks * 32) +
                            (static_cast<uint32_t>(32 * quarter + 16 * half) << 16);
        tmem_st_16x64(ta, r0);
        if (j * kChunks + 1 < p.K64) {
          unpack(1, r0);
          tmem_st_16x64(ta + 32, r0);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(afull0 + 8 * grp);
      }
    }
    cp_wait<0>();
  } else {
    // ---- epilogue: TMEM lanes of a quarter, half of the columns ---------------------
    const int quarter = warp & 3, half = (warp - kDqWarps) >> 2;
    const uint32_t dempty0 = cluster_addr(dempty, 0);
    int n = 0;
    for (int u = u0; u < units; u += du, ++n) {
      const SlotGroup sg = p.groups[u / np];
      const int nt = 2 * (u % np) + static_cast<int>(rank);
      // TMEM lane of a thread: gate rows 0-15 and up rows 16-31 of a quarter,
      // or row 32 quarter + lane of the tile.
      const Columns &cl = cols2[n & 1];
      const int row = gate_up ? 64 * nt + 16 * quarter + (lane & 15)
                              : 128 * nt + 32 * quarter + lane;
      const bool live = row < p.N, up = gate_up && lane >= 16;
      const int m = up ? 1 : 0;
      const int64_t srow = int64_t(sg.e) * p.N16 * kTileN + (live ? row : 0);
      // The inverse of a power of two, and the 2^-24 that the codes carry.
      const float rinv =
          __uint_as_float((254u << 23) - __float_as_uint(p.ts[m].fac[srow])) * 16777216.f;
      const float bias =
          p.w[m].bias && live ? p.w[m].bias[int64_t(sg.e) * p.N + row] : 0.f;
      const uint32_t d = tmem_d + (n & 1) * kTileSlots + (static_cast<uint32_t>(32 * quarter) << 16);
      if (!mbar_sleep(cfull + (n & 1), (n / 2) & 1) || !mbar_sleep(dfull + (n & 1), (n / 2) & 1)) {
        record_fault(&g_fault_moe, kFaultMoeWait);
        break;
      }
      tc_fence_after();
      const int share = (sg.cols + 63) / 64 * 32;  // columns per half
      for (int c0 = share * half; c0 < share * (half + 1) && c0 < sg.cols; c0 += 32) {
        float v[32];
        tmem_ld32(d + c0, v);
        // Lanes of neighbouring rows exchange, so that each stores two rows of
        // every other column: a pair of columns (c, c + 1) in `u`, own row.
        auto pair_rows = [&](uint32_t u) {
          const uint32_t w = __shfl_xor_sync(0xffffffffu, u, 1);
          return __byte_perm(u, w, lane & 1 ? 0x3276 : 0x5410);
        };
        if (gate_up) {
          // Lanes below 16 take columns 0-15, the others 16-31: each sends
          // what the other half-warp lacks.
          const int mine0 = c0 + (up ? 16 : 0);
          float *dst = p.hidden + int64_t(sg.first + mine0) * p.ldh + row;
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float4 ck = *reinterpret_cast<const float4 *>(&cl.ab[mine0 + i]);
            const float4 cs = *reinterpret_cast<const float4 *>(&cl.ab[c0 + i + (up ? 0 : 16)]);
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              const float keep = up ? v[16 + i + o] : v[i + o];
              const float send = up ? v[i + o] : v[16 + i + o];
              const float k = fmaf(keep * rinv, o ? ck.z : ck.x, bias);
              const float got = __shfl_xor_sync(
                  0xffffffffu, fmaf(send * rinv, o ? cs.z : cs.x, bias), 16);
              const float gv = up ? got : k, uv = up ? k : got;
              // silu(g) = g / (1 + e^-g), for g < 0 as g e^g / (1 + e^g): neither the
              // divisor nor a factor of the product overflows on the way.
              const float ex = __expf(-fabsf(gv));
              const float h = __fdividef(gv < 0.f ? gv * ex : gv, 1.f + ex) * uv *
                              (o ? ck.w : ck.y);
              if (live && mine0 + i + o < sg.cols) dst[(i + o) * p.ldh] = h;
            }
          }
        } else if (p.mode == kStreamProduct) {
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float4 ck = *reinterpret_cast<const float4 *>(&cl.ab[c0 + i]);
            const uint32_t u = f32x2_to_bf16x2(fmaf(v[i] * rinv, ck.x, bias),
                                               fmaf(v[i + 1] * rinv, ck.z, bias));
            if (p.y_pairs) {
              const uint32_t w = pair_rows(u);
              const int c = c0 + i + (lane & 1);
              if ((row & ~1) < p.N && c < sg.cols)
                *reinterpret_cast<uint32_t *>(p.Y + int64_t(cl.out[c]) * p.N + (row & ~1)) = w;
            } else if (live) {
              if (c0 + i < sg.cols)
                p.Y[int64_t(cl.out[c0 + i]) * p.N + row] = static_cast<uint16_t>(u);
              if (c0 + i + 1 < sg.cols)
                p.Y[int64_t(cl.out[c0 + i + 1]) * p.N + row] = static_cast<uint16_t>(u >> 16);
            }
          }
        } else {
          uint16_t *dst = p.part + int64_t(sg.first + c0 + (lane & 1)) * p.ldp + (row & ~1);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float4 ck = *reinterpret_cast<const float4 *>(&cl.ab[c0 + i]);
            const uint32_t w = pair_rows(pack_f16x2(fmaf(v[i] * rinv, ck.x, bias * ck.y),
                                                    fmaf(v[i + 1] * rinv, ck.z, bias * ck.w)));
            if ((row & ~1) < p.N && c0 + i + (lane & 1) < sg.cols)
              *reinterpret_cast<uint32_t *>(dst + i * p.ldp) = w;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_cluster(dempty0 + 8 * (n & 1));
        mbar_arrive(cempty + (n & 1));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA releases the tensor memory while the pair uses it
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_a),
                 "r"(kTmemCols)
                 : "memory");
  }
}

template <int BS, bool ZP, bool SF32>
cudaError_t launch_one(const TileParams &p, bool pdl, cudaStream_t stream) {
  constexpr int kSmem = make_layout<BS, SF32, ZP>().total + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static std::atomic<unsigned long long> done{0};
  auto *kernel = tile_kernel<BS, ZP, SF32>;
  const cudaError_t e = ensure_smem_limit(kernel, kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(sm_count() & ~1);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int BS>
cudaError_t launch_bs(const TileParams &p, bool zp, bool sf32, bool pdl, cudaStream_t s) {
  if (zp) return sf32 ? launch_one<BS, true, true>(p, pdl, s) : launch_one<BS, true, false>(p, pdl, s);
  return sf32 ? launch_one<BS, false, true>(p, pdl, s) : launch_one<BS, false, false>(p, pdl, s);
}

}  // namespace

cudaError_t launch_tile(const TileParams &p, bool zp, bool sf32, int bs, bool pdl,
                        cudaStream_t stream) {
  switch (bs) {
    case 16: return launch_bs<16>(p, zp, sf32, pdl, stream);
    case 32: return launch_bs<32>(p, zp, sf32, pdl, stream);
    case 64: return launch_bs<64>(p, zp, sf32, pdl, stream);
    case 128: return launch_bs<128>(p, zp, sf32, pdl, stream);
    default: return launch_bs<256>(p, zp, sf32, pdl, stream);
  }
}

cudaError_t moe_take_fault(unsigned int *out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_fault_moe, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_fault_moe, &zero, sizeof zero);
}

}  // namespace mnb
