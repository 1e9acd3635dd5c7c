// Attention of many new tokens over the pages of a cache on the tensor cores
// (tcgen05 / TMEM), bf16, head sizes 64 and 128.
//
//   o_i = sum_j w_ij v_j / sum_j w_ij,  w_ij = exp(scale q_i . k_j),
// one pass over the keys with a running maximum and sum per row.
//
// Rows of a sequence are (token, head of the key head's group), token first.
// A unit is 256 of them, two tiles of 128, times the keys that they attend, in
// blocks of 128 keys. plan_kernel lists the units of a key head with their
// blocks; all blocks of all key heads form one line, of which every CTA (one
// per SM, persistent) takes an equal part: ragged batches, causal prompts and
// a few rows over a long cache share out alike, whatever the device arrays
// hold. Pieces of units that several CTAs share are joined by combine_kernel.
//
// In a CTA the two tiles take turns: while one tile's softmax runs in its
// warps (a thread per row), the tensor core works for the other.
//   S_i = Q_i K^T   128 x 128 fp32 in TMEM, Q and K in shared memory
//   P_i = weights   bf16, written over S_i, an operand from TMEM
//   O_i += P_i V    V as it lies in shared memory (keys by rows: the N-major
//                   form of the B operand)
// S and O of both tiles fill the 512 columns of TMEM. MMAs execute in the
// order of their issue, so S of the next block may follow directly on the
// product that reads P out of the same columns, and the arrival that tells of
// S tells that O is at rest too: a row's O is rescaled by its own thread, and
// only when its maximum has grown by 2^8 in weight (weights above 1 up to 2^8
// do no harm in bf16 or in the fp32 sums; a known refinement of the running
// maximum).
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "attn_tile.h"
#include "mnb_common.cuh"
#include "mnb_launch.h"
#include "umma.cuh"

namespace mnb {

__device__ unsigned int g_fault_attn = 0;

namespace {

constexpr int kTile = 128;                 // rows of an MMA, keys of a block
constexpr int kUnit = 2 * kTile;           // rows of a unit
constexpr int kSoftWarps = 8;              // two tiles of four warps
constexpr int kTmaWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1;
constexpr int kScanWarp = kSoftWarps + 2, kScanWarps = 2;
constexpr int kThreads = 32 * (kSoftWarps + 4);
// Registers: of the 3 x 168 a lane that the launch has, the softmax takes more.
constexpr int kSoftRegs = 216, kOtherRegs = 72;
static_assert(2 * kSoftRegs + kOtherRegs <= 3 * 168, "within the launch's registers");
constexpr int kInfo = 8;                   // blocks whose masks are kept, masked ones in flight
constexpr int kPieces = 8;                 // pieces of units that are known ahead
constexpr int kTmemCols = 512;
constexpr int kHeader = 8;                 // ints
constexpr float kGrow = 8.f;               // rescale from 2^8 on
// A unit counts for as many blocks more than it has: its masked block, results
// and first scores stand for some 6000 cycles, a block in full swing for 2650.
constexpr int kUnitCost = 2;
// Blocks whose products are added up in tensor memory. The tensor cores cut off
// what they add, relative to the sum so far: 1 M keys of equal weight in one run
// came out 0.37 % low, 4 M 2.2 %. So after a run a row's O goes to its thread's
// place in global memory, added there with rounding: at most 4096 additions of the
// tensor cores stand in a row, some 2^-12. (Runs past 65536 keys alone: 38912 rows
// over 1 M keys take 12.86 ms, 12.74 in one sum.)
constexpr int kRun = 512;

template <int D>
struct Cfg {
  static constexpr int tile = kTile * D * 2;       // bytes of 128 rows of q, k or v
  static constexpr int half = kTile * 128;         // bytes of their 64 columns
  static constexpr int stages = D == 128 ? 5 : 10;
  static constexpr int off_ring = 2 * tile;
  static constexpr int off_info = off_ring + stages * tile;
  static constexpr int off_todo = off_info + kInfo * 32;  // of masked blocks: tile, or -1
  static constexpr int off_pieces = off_todo + kInfo * 4;
  static constexpr int off_bar = off_pieces + kPieces * 48;
  static constexpr int total = off_bar + 768;
};
static_assert(Cfg<128>::total + 1024 <= 227 * 1024, "shared memory");

struct Info {       // of a block of keys
  uint32_t pages;   // bit g: keys 16 g .. 16 g + 15 have a page
  int scan;         // masked: the how-manieth masked block it is, else -1
  uint32_t pad[2];
  uint32_t bad[4];  // masked: keys whose values are not finite
};
static_assert(sizeof(Info) == 32, "");

// Bounded wait that sleeps in the hardware for up to 50 us at a time: a warp
// that polls takes issue slots from the softmax. At most about a second.
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
// The same for what a whole run of blocks may stand before: the next masked block,
// or the next unit for a tile that the present one leaves out. 2^31 keys are 2^24
// blocks at 1.4 us, 23 s; the copying warp says when it has given up.
__device__ __forceinline__ bool mbar_sleep_long(uint64_t *bar, uint32_t parity,
                                                const volatile int *given_up) {
  for (int i = 0; i < 40; ++i) {
    if (mbar_sleep(bar, parity)) return true;
    if (*given_up) return false;
  }
  return false;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void tma_load_4d(void *dst, const void *tmap, int x, int y, int z,
                                            int w, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}
// D fp32, A and B bf16, M = 128; B's rows are its N (n_major: its K) index.
__host__ __device__ constexpr uint32_t idesc_bf16(int n, bool b_n_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_n_major ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kTile >> 4) << 24);
}
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_commit(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(bar))
      : "memory");
}
// V's descriptor: rows of 64 columns (128 bytes, swizzled), one per key; groups
// of 8 keys lie 1024 bytes apart (stride offset), the halves of 64 columns
// `half` bytes apart (leading offset).
__device__ __forceinline__ uint64_t smem_desc_rows(uint32_t addr, uint32_t half) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr & 0x3FFFF) >> 4);
  d |= static_cast<uint64_t>(half >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// 32 consecutive fp32 columns of this thread's TMEM lane, without waiting for
// them; and the wait, which hands the registers on.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}
// 32 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
      :
      : "r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
  uint32_t r[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
  tmem_st32(taddr, r);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      :
      : "r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Two fp32 numbers at a time.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---- the line of blocks -------------------------------------------------------------

struct Unit {
  int t0, n, len, tile;  // rows tile * 256 .. of a sequence's n tokens from row t0 on
  int block0, blocks;    // of keys
  int b;                 // the sequence
};

__device__ __forceinline__ int units_of(const Seq &s, int G) {
  return (s.n * G + kUnit - 1) / kUnit;
}
__device__ __forceinline__ int first_pos(const Unit &u, int G) {
  return u.len - u.n + u.tile * kUnit / G;
}
__device__ __forceinline__ int last_pos(const Unit &u, int G) {
  return u.len - u.n + min(u.n - 1, (u.tile * kUnit + kUnit - 1) / G);
}

// Inclusive sums over the block's threads.
template <typename I>
__device__ __forceinline__ I block_scan(I v, I *sums, int tid) {
  const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
  for (int m = 1; m < 32; m *= 2) {
    const I o = __shfl_up_sync(0xffffffffu, v, m);
    if (lane >= m) v += o;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    I w = sums[lane];
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
      const I o = __shfl_up_sync(0xffffffffu, w, m);
      if (lane >= m) w += o;
    }
    sums[lane] = w;
  }
  __syncthreads();
  return warp ? v + sums[warp - 1] : v;
}

// Lists the units of a key head and where in the line each begins: one block,
// a warp per sequence. Latency-bound. (Sequences that overlap, which `starts`
// must not describe, could make more units than there is room for: those past
// it are left out.)
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads)
    plan_kernel(const __grid_constant__ AttnTileParams p) {
  __shared__ int64_t sums[32];
  __shared__ int64_t offset[kPlanThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dependency_wait();
  grid_dependents_launch();
  int64_t base = 0;
  for (int b0 = 0; b0 < p.b.n; b0 += kPlanThreads) {
    int mine = 0;
    if (b0 + tid < p.b.n) mine = units_of(load_seq(p.b, b0 + tid, p.T, p.window), p.G);
    const int64_t upto = block_scan<int64_t>(mine, sums, tid);
    offset[tid] = base + upto - mine;
    base += sums[31];
    __syncthreads();
    for (int i = warp; i < min(kPlanThreads, p.b.n - b0); i += 32) {
      const Seq s = load_seq(p.b, b0 + i, p.T, p.window);
      const int64_t n = min(int64_t(units_of(s, p.G)), p.most - offset[i]);
      for (int t = lane; t < n; t += 32) {
        Unit u{s.t0, s.n, s.len, t, 0, 0, b0 + i};
        if (p.window > 0)
          u.block0 = min(max(0, max(0, first_pos(u, p.G)) - p.window + 1), p.cap) / kTile;
        u.blocks = max(1, (min(last_pos(u, p.G), p.cap - 1) + kTile) / kTile - u.block0);
        p.units[2 * (offset[i] + t)] = make_int4(u.t0, u.n, u.len, u.tile);
        p.units[2 * (offset[i] + t) + 1] = make_int4(u.block0, u.blocks, u.b, 0);
      }
    }
    __syncthreads();
  }
  base = min(base, p.most);
  __shared__ int longest;  // unit's blocks
  if (tid == 0) longest = 0;
  __syncthreads();
  int64_t at = 0;
  for (int64_t u0 = 0; u0 < base; u0 += kPlanThreads) {
    const int blocks = u0 + tid < base ? p.units[2 * (u0 + tid) + 1].y : 0;
    const int64_t mine = u0 + tid < base ? blocks + int64_t(kUnitCost) : 0;
    const int most = __reduce_max_sync(0xffffffffu, blocks);
    if (lane == 0) atomicMax(&longest, most);
    const int64_t upto = block_scan<int64_t>(mine, sums, tid);
    if (u0 + tid < base) p.first[u0 + tid] = at + upto - mine;
    at += sums[31];
    __syncthreads();
  }
  if (tid == 0) {
    p.first[base] = at;
    p.line[0] = at;
    p.line[1] = base;
    p.line[2] = longest;
  }
}

constexpr int kSplit = 3;  // a CTA has sqrt(longest unit / kSplit) places at least

// A CTA's part of the line, piece by piece; the unit after the present one is
// loaded ahead. A unit's own cost stands before its blocks: block k is at
// kUnitCost + k, and who has that place has the block.
struct Walk {
  const AttnTileParams &p;
  int64_t at, x1, total;  // at: the unit's place in the line
  int parts, n_units, unit, head, k0, k1;
  Unit u, after;
  __device__ __forceinline__ explicit Walk(const AttnTileParams &p_) : p(p_) {}
  __device__ __forceinline__ Unit load(int i) const {
    const int4 a = p.units[2 * i], b = p.units[2 * i + 1];
    return Unit{a.x, a.y, a.z, a.w, b.x, b.y, b.z};
  }
  // Blocks of the unit at `from` that lie before place x.
  __device__ __forceinline__ int before(int64_t x, int64_t from, const Unit &v) const {
    return static_cast<int>(max(int64_t(0), min(int64_t(v.blocks), x - from - kUnitCost)));
  }
  __device__ __forceinline__ void enter() {
    k1 = before(x1, at, u);
    if (at + u.blocks + kUnitCost < x1) after = load(unit + 1 == n_units ? 0 : unit + 1);
  }
  // Whole warps; false: nothing for this CTA.
  __device__ __forceinline__ bool start(int lane) {
    const int64_t per = p.line[0];
    n_units = static_cast<int>(p.line[1]);
    total = per * p.kv_heads;
    // Of a long unit the pieces take as long to join as to make when a CTA has
    // sqrt(unit / kSplit) blocks (128 rows over 16000 keys: 30 us, 69 with a place of
    // the line each; over 2000 18 and 20).
    const int least =
        max(1, static_cast<int>(sqrtf(static_cast<float>(p.line[2]) / kSplit) + 0.5f));
    parts = static_cast<int>(min(int64_t(gridDim.x), (total + least - 1) / least));
    if (static_cast<int>(blockIdx.x) >= parts) return false;
    const int64_t x0 = blockIdx.x * total / parts;
    x1 = (blockIdx.x + 1) * total / parts;
    head = static_cast<int>(x0 / per);
    const int64_t in = x0 - head * per;
    int lo = 0, hi = n_units;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step;
      const int k = __popc(__ballot_sync(0xffffffffu, i < hi && p.first[i] <= in));
      lo += k * step;
      hi = min(hi, lo + step);
    }
    unit = lo;
    at = head * per + p.first[unit];
    u = load(unit);
    k0 = before(x0, at, u);
    enter();
    return k0 < k1 || next();
  }
  // Another piece follows.
  __device__ __forceinline__ bool more() const {
    return at + u.blocks + 2 * kUnitCost < x1;
  }
  __device__ __forceinline__ bool next() {
    if (!more()) return false;
    at += u.blocks + kUnitCost;
    k0 = 0;
    if (++unit == n_units) {
      unit = 0;
      ++head;
    }
    u = after;
    enter();
    return true;
  }
  // The CTAs after this one that have a piece of the unit that ends this part.
  __device__ __forceinline__ int others() const {
    if (k0 > 0 || k1 == u.blocks) return 0;
    const int64_t last = at + kUnitCost + u.blocks - 1;  // the last block's place
    int64_t c = ((last + 1) * parts - 1) / total;
    while (c * total / parts > last) --c;
    while (c + 1 < parts && (c + 1) * total / parts <= last) ++c;
    return static_cast<int>(c) - static_cast<int>(blockIdx.x);
  }
  // The unit has rows in its second tile.
  __device__ __forceinline__ bool two(const Unit &v) const {
    return v.n * p.G > v.tile * kUnit + kTile;
  }
};

// A piece as the copying warp hands it to the others.
struct Piece {
  int t0, n, len, tile, block0, blocks, head, k0, k1;
  int more;  // another one follows
  int none;  // this CTA has no part of the line
  int pad;
};
static_assert(sizeof(Piece) == 48, "");

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    tile_kernel(const __grid_constant__ AttnTileParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  Info *infos = reinterpret_cast<Info *>(smem + C::off_info);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::off_bar);
  uint64_t *empty = full + C::stages;
  uint64_t *known = empty + C::stages;  // a block's info is there
  uint64_t *sfull = known + kInfo;      // per tile
  uint64_t *pfull = sfull + 2;
  uint64_t *qfull = pfull + 2;
  uint64_t *ofull = qfull + 2;
  uint64_t *toscan = ofull + 2;         // a masked block's values are to be looked over
  uint64_t *scanned = toscan + kInfo;   // and have been
  uint64_t *listed = scanned + kInfo;   // a piece is there
  uint64_t *taken = listed + kPieces;   // and has been read by every warp it concerns
  uint64_t *qfree = taken + kPieces;    // per tile: its rows have been used
  uint64_t *done = qfree + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *given_up = reinterpret_cast<int *>(tmem_slot + 1);  // the copying warp has
  static_assert((2 * C::stages + 3 * kInfo + 2 * kPieces + 11) * 8 + 8 <= 768, "barriers");
  int *todo = reinterpret_cast<int *>(smem + C::off_todo);
  Piece *pieces = reinterpret_cast<Piece *>(smem + C::off_pieces);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < C::stages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < kInfo; ++i) {
      mbar_init(known + i, 1);
      mbar_init(toscan + i, 1);
      mbar_init(scanned + i, kScanWarps);
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(listed + i, 1);
      mbar_init(taken + i, kSoftWarps + 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sfull + i, 1);
      mbar_init(pfull + i, 4);
      mbar_init(qfull + i, p.q_tma ? 1 : 4);
      mbar_init(qfree + i, 1);
      mbar_init(ofull + i, 1);
    }
    mbar_init(done, 1);
    *given_up = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  grid_dependency_wait();
  grid_dependents_launch();
  // The pieces, as every warp but the copying ones takes them: copied to
  // registers, so that the place is free again at once.
  auto take_piece = [&](int n, bool &ok) {
    ok = __all_sync(0xffffffffu,
                    mbar_sleep_long(listed + n % kPieces, (n / kPieces) & 1, given_up));
    const Piece pc = pieces[n % kPieces];
    __syncwarp();
    if (lane == 0) mbar_arrive(taken + n % kPieces);
    return pc;
  };
  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kTmaWarp) {
      // ---- keys and values ----------------------------------------------------------
      const int nbox = kTile / p.box;  // copies of 64 columns: nbox for each half
      const int box = lane % nbox, col = lane / nbox;
      const bool copies = lane < nbox * (D / 64);
      Walk w(p);
      const bool any = w.start(lane);
      int tiles = 0, blocks = 0, scans = 0, listing = 0, uses[2] = {0, 0};
      bool ok = true;
      if (!any && lane == 0) {
        pieces[0].none = 1;
        mbar_arrive(listed);
      }
      if (any) do {
        const int ps = listing % kPieces;
        if (listing >= kPieces)
          ok = __all_sync(0xffffffffu, mbar_sleep(taken + ps, (listing / kPieces - 1) & 1));
        if (!ok) break;
        const bool two = w.two(w.u);
        if (lane == 0) {
          pieces[ps] = Piece{w.u.t0,     w.u.n,  w.u.len, w.u.tile, w.u.block0, w.u.blocks,
                             w.head,     w.k0,   w.k1,    w.more(), 0,          0};
          mbar_arrive(listed + ps);
        }
        ++listing;
        const int bottom = first_pos(w.u, p.G);
        const int last = max(last_pos(w.u, p.G), -1), end = min(w.u.len, p.cap);
        // Lane g < 8: the page of the keys 16 g on of the next block.
        auto page_of = [&](int kb) {
          const int j = (w.u.block0 + kb) * kTile + (lane & 7) * 16;
          int page = -1;
          if (j < end && j <= last) page = p.b.table[w.u.b * p.b.table_stride + j / p.page_size];
          return page >= 0 && page < p.pages ? page : -1;
        };
        int page = page_of(w.k0);
        for (int kb = w.k0; kb < w.k1; ++kb, ++blocks) {
          const int now = page;
          if (kb + 1 < w.k1) page = page_of(kb + 1);
          const uint32_t bits = __ballot_sync(0xffffffffu, now >= 0 && lane < 8);
          const int mine = __shfl_sync(0xffffffffu, now, box * (p.box / 16) & 7);
          const int j0 = (w.u.block0 + kb) * kTile, at = (j0 + box * p.box) % p.page_size;
          // Masks are needed where some row of the unit does not attend some key
          // (both tiles alike: they share what is done to the values).
          const bool masked = bits != 0xFFu || j0 + kTile - 1 > bottom ||
                              (p.window > 0 && j0 <= last - p.window);
          for (int v = 0; v < 2; ++v, ++tiles) {
            const int s = tiles % C::stages;
            if (tiles >= C::stages) {
              ok = __all_sync(0xffffffffu, mbar_sleep(empty + s, (tiles / C::stages - 1) & 1));
              if (!ok) break;
            }
            if (v == 0 && lane == 0) {
              // (A free stage for these keys means that the block eight before
              // them is done with.)
              Info &f = infos[blocks % kInfo];
              f.pages = bits;
              f.scan = masked ? scans : -1;
              f.bad[0] = f.bad[1] = f.bad[2] = f.bad[3] = 0;
              mbar_arrive(known + blocks % kInfo);
            }
            if (v == 1 && masked) {
              // Not before this stage is free: until then its barrier may be a phase
              // behind, and the parity that the values are waited for by taken for the
              // one before it. (As many masked blocks are never in flight.)
              if (lane == 0) {
                todo[scans % kInfo] = blocks;
                mbar_arrive(toscan + scans % kInfo);
              }
              ++scans;
            }
            if (lane == 0) mbar_arrive_expect_tx(full + s, C::tile);
            __syncwarp();
            if (copies)
              tma_load_4d(smem + C::off_ring + s * C::tile + col * C::half + box * p.box * 128,
                          v ? &p.tv : &p.tk, col * 64, at, w.head, mine, full + s);
            __syncwarp();
            // The unit's rows follow its first keys, as each tile's place is free.
            if (v == 0 && kb == w.k0 && p.q_tma)
              for (int i = 0; i < 1 + two; ++i) {
                if (uses[i]++ > 0)
                  ok = __all_sync(0xffffffffu, mbar_sleep(qfree + i, (uses[i] - 2) & 1));
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(qfull + i, C::tile);
                __syncwarp();
                if (lane < D / 64)
                  tma_load_3d(smem + i * C::tile + lane * C::half, &p.tq, lane * 64, w.head * p.G,
                              w.u.t0 + (w.u.tile * kUnit + i * kTile) / p.G, qfull + i);
                __syncwarp();
              }
            if (!ok) break;
          }
          if (!ok) break;
        }
      } while (ok && w.next());
      if (lane == 0) {
        todo[scans % kInfo] = -1;
        mbar_arrive(toscan + scans % kInfo);
      }
      if (!ok) {
        if (lane == 0) {
          *given_up = 1;
          record_fault(&g_fault_attn, kFaultAttnWait);
        }
        // Given up: the copies in flight land before the CTA leaves.
        for (int i = max(0, tiles - C::stages); i < tiles; ++i)
          mbar_sleep(full + i % C::stages, (i / C::stages) & 1);
        for (int i = 0; i < 2 && p.q_tma; ++i)
          if (uses[i] > 0) mbar_sleep(qfull + i, (uses[i] - 1) & 1);
      }
      if (lane == 0) {
        // A unit that begins in this part and goes on past it: the CTAs after
        // this one that have a piece of it. (After a wait that ran out the
        // results mean nothing.)
        int *header = p.headers + blockIdx.x * kHeader;
        const int more = any ? w.others() : 0;
        if (more > 0) {
          header[1] = w.u.t0;
          header[2] = w.u.n;
          header[3] = w.head;
          header[4] = w.u.tile;
        }
        header[0] = more;
      }
    } else if (warp == kMmaWarp) {
      // ---- MMAs: the whole warp goes round, one elected lane issues ------------------
      // What decides the way and the operands is taken from lane 0, so that it
      // stays in uniform registers: moving it there for each MMA took as long
      // as an MMA and a half.
      auto uniform = [](uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); };
      const uint32_t tm = uniform(tmem);
      // A negative scale: Q counts negated.
      const uint32_t qk = idesc_bf16(kTile, false) | (p.negative ? 1u << 13 : 0u);
      constexpr uint32_t kPv = idesc_bf16(D, true);
      const uint64_t q_desc = smem_desc_sw128(smem_addr(smem));
      const uint64_t k_desc = smem_desc_sw128(smem_addr(smem + C::off_ring));
      const uint64_t v_desc = smem_desc_rows(smem_addr(smem + C::off_ring), C::half);
      int next = 0, phase = 0, units0 = 0, units1 = 0, blocks0 = 0, blocks1 = 0;
      bool ok = true;
      auto wait = [&](uint64_t *bar, int parity) {
        ok = __all_sync(0xffffffffu, ok && mbar_sleep(bar, parity & 1));
      };
      auto take = [&] {  // the stage of the next tile of keys or values
        wait(full + next, phase);
        const int s = next;
        if (++next == C::stages) {
          next = 0;
          phase ^= 1;
        }
        return s;
      };
      // Issued by the elected lane. S_i = Q_i K^T; last: of the unit.
      auto scores = [&](int i, int s, bool last, bool release) {
        const uint64_t a = q_desc + i * (C::tile >> 4), b = k_desc + s * (C::tile >> 4);
#pragma unroll 1
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t step = (k / 4) * (C::half >> 4) + (k % 4) * 2;
          umma_ss(tm + i * kTile, a + step, b + step, qk, k > 0);
        }
        umma_commit(sfull + i);
        if (last) umma_commit(qfree + i);
        if (release) umma_commit(empty + s);
      };
      // O_i += P_i V.
      auto values = [&](int i, int s, bool fresh, bool release) {
        const uint64_t b = v_desc + s * (C::tile >> 4);
        umma_ts(tm + 2 * kTile + i * kTile, tm + i * kTile, b, kPv, !fresh);
#pragma unroll
        for (int k = 1; k < kTile / 16; ++k)
          umma_ts(tm + 2 * kTile + i * kTile, tm + i * kTile + k * 8, b + k * (2048 >> 4), kPv, 1);
        if (release) umma_commit(empty + s);
      };
      for (int pn = 0; ok; ++pn) {
        const Piece pc = take_piece(pn, ok);
        const bool two = uniform(pc.n * p.G > pc.tile * kUnit + kTile);
        const int n = uniform(pc.k1 - pc.k0);
        if (!ok || uniform(pc.none)) break;
        wait(qfull, units0++);
        int ks = take();
        tc_fence_after();
        if (ok && elect_one()) scores(0, ks, n == 1, !two);
        __syncwarp();
        if (two) {
          wait(qfull + 1, units1++);
          tc_fence_after();
          if (ok && elect_one()) scores(1, ks, n == 1, true);
          __syncwarp();
        }
        // What a block needs besides the weights is waited for ahead of them.
        for (int kb = 0; kb < n && ok; ++kb) {
          const bool more = kb + 1 < n, last = kb + 2 == n;
          const int vs = take();
          if (more) ks = take();
          wait(pfull, blocks0++);
          tc_fence_after();
          if (ok && elect_one()) {
            values(0, vs, kb % kRun == 0, !two);
            if (more)
              scores(0, ks, last, !two);
            else
              umma_commit(ofull);
          }
          __syncwarp();
          if (!two) continue;
          wait(pfull + 1, blocks1++);
          tc_fence_after();
          if (ok && elect_one()) {
            values(1, vs, kb % kRun == 0, true);
            if (more)
              scores(1, ks, last, true);
            else
              umma_commit(ofull + 1);
          }
          __syncwarp();
        }
        if (!uniform(pc.more)) break;
      }
      // Every MMA issued is complete before the tensor memory is released.
      if (elect_one()) umma_commit(done);
      __syncwarp();
      if (!__all_sync(0xffffffffu, mbar_sleep(done, 0)) || !ok)
        if (lane == 0) record_fault(&g_fault_attn, kFaultAttnWait);
    } else {
      // ---- values of masked blocks ----------------------------------------------------
      // A masked value that is not finite would still make 0 * inf: such values
      // become 0 here, before the weights' product with them, and their keys are
      // noted: the rows that do attend one get NaN.
      auto over = [](uint32_t y) { return (y & 0x7F807F80u) + 0x00800080u; };
      bool ok = true;
      for (int n = 0; ok; ++n) {
        ok = __all_sync(0xffffffffu,
                        mbar_sleep_long(toscan + n % kInfo, (n / kInfo) & 1, given_up));
        const int block = ok ? todo[n % kInfo] : -1, t = 2 * block + 1;
        if (block < 0) break;
        ok = __all_sync(0xffffffffu, mbar_sleep(full + t % C::stages, (t / C::stages) & 1));
        if (!ok) break;
        unsigned char *v = smem + C::off_ring + (t % C::stages) * C::tile;
        uint32_t *bad = infos[block % kInfo].bad;
        constexpr int kStep = 32 * kScanWarps;
#pragma unroll 1
        for (int c = (warp - kScanWarp) * 32 + lane; c < C::tile / 16; c += 8 * kStep) {
          uint32_t hit = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint4 x = *reinterpret_cast<const uint4 *>(v + (c + e * kStep) * 16);
            hit |= over(x.x) | over(x.y) | over(x.z) | over(x.w);
          }
          if (!(hit & 0x80008000u)) continue;
#pragma unroll 1
          for (int e = 0; e < 64; ++e) {
            const int at = c + (e / 8) * kStep;
            uint16_t *x = reinterpret_cast<uint16_t *>(v + at * 16) + e % 8;
            if ((*x & 0x7F80u) != 0x7F80u) continue;
            *x = 0;
            const int key = (at / 8) % kTile;
            atomicOr(bad + (key >> 5), 1u << (key & 31));
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(scanned + n % kInfo);
      }
      if (!ok && lane == 0) record_fault(&g_fault_attn, kFaultAttnWait);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    {
      // ---- softmax: a thread per row ------------------------------------------------
      const int i = warp >> 2, r = (warp & 3) * 32 + lane;  // tile, row in it
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t ts = tmem + lanes + i * kTile, to = tmem + lanes + 2 * kTile + i * kTile;
      int blocks = 0, mine = 0, units = 0;  // of the CTA; of this tile
      bool ok = true;
      const int row = i * kTile + r;  // in the unit
      // The unit's rows, where no tensor map describes them: lanes side by side
      // along a row. 16-byte piece c of row r lies at c ^ (r & 7) of the row's 128
      // bytes.
      auto load_q = [&](const Piece &u, int at, int tok) {
        const uint16_t *src = static_cast<const uint16_t *>(p.q.p);
        const uint64_t mine_at =
            at < u.n * p.G
                ? reinterpret_cast<uint64_t>(src + int64_t(u.t0 + tok) * p.q.ts +
                                             int64_t(u.head * p.G + at - tok * p.G) * p.q.hs)
                : 0;
        constexpr int kPieces = D / 8, kAtOnce = 32 / kPieces;  // pieces of a row; rows
        const int c = lane % kPieces;
#pragma unroll 4
        for (int e = 0; e < 32; e += kAtOnce) {
          const int from = e + lane / kPieces, rr = (warp & 3) * 32 + from;
          const uint64_t x = __shfl_sync(0xffffffffu, mine_at, from);
          cp16_or_zero(smem_addr(smem + i * C::tile + (c / 8) * C::half + rr * 128 +
                                 (((c % 8) ^ (rr & 7)) << 4)),
                       x ? reinterpret_cast<const uint16_t *>(x) + c * 8 : src, x != 0);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(qfull + i);
      };
      // The row's place among a piece's results: four columns of all rows, the next
      // four, ..: lanes lie side by side.
      auto part_of = [&](const Piece &u) {
        return p.parts + (int64_t(blockIdx.x) * 2 + (u.k0 == 0)) * (kUnit * (D + 2)) + row * 4;
      };
      for (int pn = 0; ok; ++pn) {
        const Piece pc = take_piece(pn, ok);
        if (!ok || pc.none) break;
        if (i == 1 && pc.n * p.G <= pc.tile * kUnit + kTile) {  // no rows in this tile
          blocks += pc.k1 - pc.k0;
          if (!pc.more) break;
          continue;
        }
        const int at = pc.tile * kUnit + row, tok = at / p.G;
        const bool live = at < pc.n * p.G;
        const int pos = live ? max(pc.len - pc.n + tok, -1) : -1;
        if (!p.q_tma) load_q(pc, at, tok);
        float m = -INFINITY, mc = 0.f, l = 0.f;  // maximum (of scores), times the scale; sum
        float part_mc = 0.f;  // mc when O was last added to part (-inf: nothing attended)
        for (int run = pc.k0; run < pc.k1 && ok; run += kRun) {
          if (run > pc.k0) {
            // (The next scores tell that O is at rest.)
            ok = __all_sync(0xffffffffu, mbar_sleep(sfull + i, mine & 1));
            if (!ok) break;
            tc_fence_after();
            const bool add = run - pc.k0 > kRun;
            const float fac = exp2_fast(part_mc - mc);
            part_mc = m == -INFINITY ? -INFINITY : mc;
            float *part = part_of(pc);
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float o[32];
              tmem_ld32(to + c, o);
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                float4 *x = reinterpret_cast<float4 *>(part + (c + e) * kUnit);
                const float4 y = add ? *x : make_float4(0.f, 0.f, 0.f, 0.f);
                *x = make_float4(fmaf(fac, y.x, o[e]), fmaf(fac, y.y, o[e + 1]),
                                 fmaf(fac, y.z, o[e + 2]), fmaf(fac, y.w, o[e + 3]));
              }
            }
          }
          const int end = min(run + kRun, pc.k1);
          for (int kb = run; kb < end && ok; ++kb, ++blocks, ++mine) {
            // (In this order: a tile that was left out of units is blocks ahead.)
            ok = mbar_sleep(sfull + i, mine & 1) &&
                 mbar_sleep(known + blocks % kInfo, (blocks / kInfo) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            Info &f = infos[blocks % kInfo];
            const int j0 = (pc.block0 + kb) * kTile;
            const uint32_t have = f.pages;
            const int scan = f.scan;
            if (scan >= 0) {
              ok = __all_sync(0xffffffffu,
                              mbar_sleep(scanned + scan % kInfo, (scan / kInfo) & 1));
              if (!ok) break;
              // Through tensor memory and back, in a loop: this way is taken for a
              // block or two of a unit, and as straight code it took longer to fetch
              // than to run.
#pragma unroll 1
              for (int c0 = 0; c0 < kTile; c0 += 32) {
                const uint32_t bad = *static_cast<const volatile uint32_t *>(&f.bad[c0 / 32]);
                const int to = pos - j0 - c0, from = p.window > 0 ? to - p.window + 1 : 0;
                // Bit e: the row attends column c0 + e.
                uint32_t on = to < 0 ? 0u : to >= 31 ? ~0u : (2u << to) - 1u;
                on &= from <= 0 ? ~0u : from >= 32 ? 0u : ~0u << from;
                on &= ((have >> (c0 / 16)) & 1 ? 0xFFFFu : 0u) |
                      ((have >> (c0 / 16)) & 2 ? 0xFFFF0000u : 0u);
                if (__all_sync(0xffffffffu, on == ~0u && bad == 0)) continue;
                float x[32];
                if (__any_sync(0xffffffffu, on)) {
                  tmem_ld32(ts + c0, x);
#pragma unroll
                  for (int e = 0; e < 32; ++e) x[e] = on & (1u << e) ? x[e] : -INFINITY;
                  if (__any_sync(0xffffffffu, bad & on))
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = bad & on & (1u << e) ? NAN : x[e];
                } else {
#pragma unroll
                  for (int e = 0; e < 32; ++e) x[e] = -INFINITY;
                }
                tmem_st32(ts + c0, x);
              }
              tmem_st_wait();
            }
            float s0[32], s1[32], s2[32], s3[32];  // the scores, 32 columns each
            tmem_ld32_async(ts, s0);
            tmem_ld32_async(ts + 32, s1);
            tmem_ld32_async(ts + 64, s2);
            tmem_ld32_async(ts + 96, s3);
            tmem_ld_wait(s0);
            tmem_ld_wait(s1);
            tmem_ld_wait(s2);
            tmem_ld_wait(s3);
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            auto maxima = [&](const float (&v)[32]) {
#pragma unroll
              for (int c = 0; c < 32; c += 8)
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = fmaxf(fmaxf(mx[e], v[c + e]), v[c + 4 + e]);
            };
            maxima(s0);
            maxima(s1);
            maxima(s2);
            maxima(s3);
            const float top_s = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            const float new_m = fmaxf(m, top_s), new_mc = new_m == -INFINITY ? 0.f : new_m * p.scale;
            // (Not for the difference of an infinity with itself.)
            const bool grown = new_m > m && !(new_mc - mc <= kGrow && m != -INFINITY);
            if (__any_sync(0xffffffffu, grown)) {
              const float fac = m == -INFINITY ? 0.f : exp2_fast(grown ? mc - new_mc : 0.f);
              if (grown) {
                m = new_m;
                mc = new_mc;
              }
              l *= fac;
              if (kb > run) {
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                  float o[32];
                  tmem_ld32(to + c, o);
#pragma unroll
                  for (int e = 0; e < 32; ++e) o[e] *= fac;
                  tmem_st32(to + c, o);
                }
              }
            }
            // Weights, rounded to bf16 (2^-8) for the product with the values, whose
            // type it has to be (a second part would be half as many MMAs again, and
            // columns of TMEM that there are not): errors of 0.0021 against 64 bits
            // where fp32 weights have 0.00165, results rounded to bf16. Their sum takes
            // them unrounded.
            uint64_t sum[2] = {0, 0};
            const uint64_t scale2 = pack2(p.scale, p.scale), mc2 = pack2(-mc, -mc);
            auto weights = [&](int c0, const float (&v)[32]) {
              uint32_t x[16];
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                float a, b;
                unpack2(fma2(pack2(v[c], v[c + 1]), scale2, mc2), a, b);
                a = exp2_fast(a);
                b = exp2_fast(b);
                sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], pack2(a, b));
                x[c / 2] = f32x2_to_bf16x2(a, b);
              }
              tmem_st16(ts + c0 / 2, x);
            };
            weights(0, s0);
            weights(32, s1);
            weights(64, s2);
            weights(96, s3);
            float la, lb;
            unpack2(add2(sum[0], sum[1]), la, lb);
            l += la + lb;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(pfull + i);
          }
        }
        if (ok) ok = mbar_sleep(ofull + i, units++ & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        // ---- end of a piece
        const bool whole = pc.k0 == 0 && pc.k1 == pc.blocks;
        if (pc.k1 - pc.k0 > kRun) {  // the earlier runs' sums, added to the last one's
          const float fac = exp2_fast(part_mc - mc);
          const float *part = part_of(pc);
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(to + c, o);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 y = *reinterpret_cast<const float4 *>(part + (c + e) * kUnit);
              o[e] = fmaf(fac, y.x, o[e]);
              o[e + 1] = fmaf(fac, y.y, o[e + 1]);
              o[e + 2] = fmaf(fac, y.z, o[e + 2]);
              o[e + 3] = fmaf(fac, y.w, o[e + 3]);
            }
            tmem_st32(to + c, o);
          }
          tmem_st_wait();
        }
        if (whole) {
          // Four lanes exchange 16-byte pieces of their rows, so that a store
          // covers 64 bytes of each row that it touches: with 16 of each, the
          // stores of a unit took as long as two blocks of keys.
          const uint64_t mine_at =
              live ? reinterpret_cast<uint64_t>(static_cast<uint16_t *>(p.o.p) +
                                                int64_t(pc.t0 + tok) * p.o.ts +
                                                int64_t(pc.head * p.G + at - tok * p.G) * p.o.hs)
                   : 0;
          uint64_t rows[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            rows[e] = __shfl_sync(0xffffffffu, mine_at, (lane & ~3) + e);
          const float inv = m == -INFINITY && l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(to + c, o);
            uint32_t x[16];  // four pieces
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = f32x2_to_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
#pragma unroll
            for (int bit = 1; bit < 4; bit *= 2) {
              // Piece a with the bit clear and a + bit change places across lanes.
              const bool up = lane & bit;
#pragma unroll
              for (int a = 0; a < 4; ++a) {
                if (a & bit) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  uint32_t &lo = x[a * 4 + e], &hi = x[(a + bit) * 4 + e];
                  const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, bit);
                  if (up)
                    lo = got;
                  else
                    hi = got;
                }
              }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (rows[e])
                *reinterpret_cast<uint4 *>(rows[e] + (c + (lane & 3) * 8) * 2) =
                    make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
          }
        } else {
          float *part = part_of(pc);
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(to + c, o);
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4 *>(part + (c + e) * kUnit) =
                  make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
          float *sums = part + kUnit * D - row * 3;
          sums[0] = m;
          sums[kUnit] = l;
        }
        tc_fence_before();
        if (!pc.more) break;
      }
      if (!ok && lane == 0) record_fault(&g_fault_attn, kFaultAttnWait);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

// Joins the pieces of a unit: the one that begins at the end of CTA c's part
// and the continuations at the start of the parts after it. A block per 32
// rows: a lane per row, a warp per four columns at a time.
template <int D>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ AttnTileParams p) {
  constexpr int64_t kPart = kUnit * (D + 2);
  constexpr int kLd = D / 2 + 2;             // words of a row of the result
  constexpr int kMany = 64;                  // pieces at a time
  __shared__ float fac[kMany][32], top[8][32];
  __shared__ uint32_t out_s[32 * kLd];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();
  grid_dependents_launch();
  const int *h = p.headers + blockIdx.x * kHeader;
  const int more = h[0];
  if (more == 0) return;
  const int t0 = h[1], n = h[2], head = h[3], tile = h[4];
  const int row0 = blockIdx.y * 32, row = row0 + lane;
  if (tile * kUnit + row0 >= n * p.G) return;
  const float *first = p.parts + (int64_t(blockIdx.x) * 2 + 1) * kPart;
  const float *rest = p.parts + (int64_t(blockIdx.x) + 1) * 2 * kPart;
  auto piece = [&](int c) { return c == 0 ? first : rest + (c - 1) * 2 * kPart; };
  // (Rows of a second tile that the unit does not have hold anything.)
  const bool live = tile * kUnit + row < n * p.G;
  float m = -INFINITY;
#pragma unroll 8
  for (int c = warp; c <= more; c += 8)
    if (live) m = fmaxf(m, piece(c)[kUnit * D + row]);
  top[warp][lane] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = fmaxf(m, top[w][lane]);
  const float z = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 a[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) a[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c0 = 0; c0 <= more; c0 += kMany) {
    const int cn = min(kMany, more + 1 - c0);
    __syncthreads();
#pragma unroll 8
    for (int c = warp; c < cn; c += 8)
      fac[c][lane] = live ? exp2_fast((piece(c0 + c)[kUnit * D + row] - z) * p.scale) : 0.f;
    __syncthreads();
#pragma unroll 2
    for (int c = 0; c < cn; ++c) {
      const float *x = piece(c0 + c);
      const float f = fac[c][lane];
      if (live) {
        l += f * x[kUnit * D + kUnit + row];
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          const float4 y = *reinterpret_cast<const float4 *>(x + (e * 8 + warp) * 4 * kUnit + row * 4);
          a[e].x += f * y.x;
          a[e].y += f * y.y;
          a[e].z += f * y.z;
          a[e].w += f * y.w;
        }
      }
    }
  }
  const float inv = m == -INFINITY && l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) {
    uint32_t *y = out_s + lane * kLd + (e * 8 + warp) * 2;
    y[0] = f32x2_to_bf16x2(a[e].x * inv, a[e].y * inv);
    y[1] = f32x2_to_bf16x2(a[e].z * inv, a[e].w * inv);
  }
  __syncthreads();
  for (int r = warp; r < 32; r += 8) {
    const int at = tile * kUnit + row0 + r, tok = at / p.G;
    if (at >= n * p.G) break;
    uint32_t *out = reinterpret_cast<uint32_t *>(
        static_cast<uint16_t *>(p.o.p) + int64_t(t0 + tok) * p.o.ts +
        int64_t(head * p.G + at - tok * p.G) * p.o.hs);
#pragma unroll
    for (int c = lane; c < D / 2; c += 32) out[c] = out_s[r * kLd + c];
  }
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// The most units that T rows of n sequences make.
int64_t most_units(const AttnArgs &a) {
  const int64_t G = a.q.n / a.c.heads, few = std::min<int64_t>(a.b.n, a.T);
  return (a.T * G + (kUnit - 1) * few) / kUnit;
}

struct Space {
  int64_t *line, *first;
  int4 *units;
  int *headers;
  float *parts;
  size_t bytes;
};
Space space(unsigned char *ws, const AttnArgs &a) {
  const int64_t most = most_units(a);
  const size_t ctas = std::max(1, sm_count());
  Space s{};
  size_t at = 0;
  auto take = [&](size_t n) {
    unsigned char *p = ws + at;
    at += align256(n);
    return p;
  };
  s.line = reinterpret_cast<int64_t *>(take(24));
  s.headers = reinterpret_cast<int *>(take(ctas * kHeader * 4));
  s.first = reinterpret_cast<int64_t *>(take(size_t(most + 1) * 8));
  s.units = reinterpret_cast<int4 *>(take(size_t(most) * 32));
  s.parts = reinterpret_cast<float *>(take(ctas * 2 * kUnit * (a.c.D + 2) * 4));
  s.bytes = at;
  return s;
}

template <int D>
cudaError_t run(const AttnTileParams &p, bool pdl, cudaStream_t stream) {
  constexpr int kSmem = Cfg<D>::total + 1024;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = ensure_smem_limit(tile_kernel<D>, kSmem, done);
  if (e != cudaSuccess) return e;
  const int ctas = std::max(1, sm_count());
  e = launch_after(plan_kernel, dim3(1), kPlanThreads, 0, pdl, stream, p);
  if (e == cudaSuccess)
    e = launch_after(tile_kernel<D>, dim3(ctas), kThreads, kSmem, pdl, stream, p);
  if (e == cudaSuccess)
    e = launch_after(combine_kernel<D>, dim3(ctas, kUnit / 32), 256, 0, pdl, stream, p);
  return e;
}

}  // namespace

bool tile_path(const AttnArgs &a) {
  if (a.f32) return false;
  // What a tensor map can describe.
  for (int64_t s : {a.c.k.ps, a.c.k.hs, a.c.k.ts, a.c.v.ps, a.c.v.hs, a.c.v.ts})
    if (s * 2 >= int64_t(1) << 40) return false;
  // The streaming kernel reads a sequence's keys for every 16 rows, this one for
  // every 256, at some 12 us more for its plan and its joins: enough rows a
  // sequence, and enough of all heads, are what that takes. Measured with 4 query
  // heads per key head (us, streaming / this): one sequence of 2000 tokens, 512
  // rows of all heads 10 / 21, 1024 rows 20 / 22 (19 with 8 key heads); of 16000,
  // 256 rows 25 / 31, 512 rows 36 / 34; 16 sequences of 2000, 16 rows each of 8
  // key heads 38 / 43, 20 rows 45 / 44; of 16000, 16 rows 172 / 217, 20 rows 319 /
  // 218; 16 of 16000, 32 rows each of one key head 39 / 42, of two 80 / 60.
  const int64_t G = a.q.n / a.c.heads;
  return a.T * G > 16 * std::min<int64_t>(a.b.n, a.T) && a.T * a.q.n > 512;
}

size_t tile_workspace_bytes(const AttnArgs &a) { return space(nullptr, a).bytes; }

cudaError_t launch_attn_tile(const AttnArgs &a, cudaStream_t stream) {
  AttnTileParams p{};
  p.box = 128;
  while (a.c.page_size % p.box) p.box /= 2;
  for (int v = 0; v < 2; ++v) {
    const Pages &pg = v ? a.c.v : a.c.k;
    const uint64_t dims[4] = {uint64_t(a.c.D), uint64_t(a.c.page_size), uint64_t(a.c.heads),
                              uint64_t(a.c.pages)};
    const uint64_t strides[3] = {uint64_t(pg.ts) * 2, uint64_t(pg.hs) * 2, uint64_t(pg.ps) * 2};
    const uint32_t box[4] = {64, uint32_t(p.box), 1, 1};
    const cudaError_t e = make_tmap(v ? &p.tv : &p.tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, pg.p,
                                    dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
  }
  // Rows by TMA where 128 of them are whole tokens, and the strides can be told.
  const int group = a.q.n / a.c.heads;
  const int64_t hs = a.q.n > 1 ? a.q.hs : a.c.D, ts = a.T > 1 ? a.q.ts : a.c.D;
  p.q_tma = kTile % group == 0 && hs > 0 && ts > 0 && hs * 2 < (int64_t(1) << 40) &&
            ts * 2 < (int64_t(1) << 40);
  if (p.q_tma) {
    const uint64_t dims[3] = {uint64_t(a.c.D), uint64_t(a.q.n), uint64_t(a.T)};
    const uint64_t strides[2] = {uint64_t(hs) * 2, uint64_t(ts) * 2};
    const uint32_t box[3] = {64, uint32_t(group), uint32_t(kTile / group)};
    const cudaError_t e = make_tmap(&p.tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.q.p, dims,
                                    strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
  }
  p.q = a.q;
  p.o = a.o;
  p.b = a.b;
  p.pages = static_cast<int>(a.c.pages);
  p.page_size = a.c.page_size;
  p.kv_heads = a.c.heads;
  p.G = a.q.n / a.c.heads;
  p.T = static_cast<int>(a.T);
  p.cap = static_cast<int>(int64_t(a.b.table_pages) * a.c.page_size);
  p.window = window_of(a.window);
  p.scale = static_cast<float>(
      std::min(std::max(std::fabs(static_cast<double>(a.scale)) * M_LOG2E, 1e-37), 3e38));
  p.negative = a.scale < 0.f;
  const Space s = space(a.ws, a);
  p.line = s.line;
  p.first = s.first;
  p.units = s.units;
  p.most = most_units(a);
  p.headers = s.headers;
  p.parts = s.parts;
  return a.c.D == 64 ? run<64>(p, a.pdl, stream) : run<128>(p, a.pdl, stream);
}

cudaError_t attn_take_fault(unsigned int *out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_fault_attn, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_fault_attn, &zero, sizeof zero);
}

}  // namespace mnb
