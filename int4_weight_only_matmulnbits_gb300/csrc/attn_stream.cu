// Attention of new tokens over the pages of a cache: the kernel that streams
// keys and values past 16 query rows at a time (decoding, a few tokens per
// sequence, fp32).
//
//   o_i = sum_j w_ij v_j / sum_j w_ij,  w_ij = exp(scale q_i . k_j),
// over the keys j <= p_i (and j > p_i - window) of row i's position p_i, with
// the running maximum and sum of a softmax: one pass over the keys.
//
// Rows of a sequence are (token, head of the key head's group), numbered token
// first; 16 of them, padded, are the rows of the MMAs, so that a key head's
// keys are read once for its whole group. The keys are cut into blocks of 64,
// and all blocks of all (sequence, key head, 16 rows), of those keys that a window
// reaches from the rows, are shared out evenly in
// one long line: block c of the grid takes the part c of it, wherever that
// begins and ends. So the split follows the lengths that the device arrays
// hold at that moment (a captured graph's too), whatever they are. Pieces of a
// unit that several blocks share are joined by combine_kernel.
//
// A block's warps take 16 of a block's 64 keys each, with a ring of
// asynchronous copies of their own, so that no barrier stands in the loop; the
// warps' sums are joined at the end of a piece.
//
// Few units (a single sequence's decode step): a cluster of 8 or 16 blocks takes
// a unit, an equal share of its keys each, and joins the sums through
// distributed shared memory: one launch instead of two. Decoding one sequence
// of 4097 tokens (8 key heads of 128, bf16) takes 9.0 us this way and 12.7 with
// the line and its joining kernel.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "attn.h"
#include "attn_stream.h"
#include "mnb_common.cuh"
#include "mnb_launch.h"

namespace mnb {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kSplit = 12;        // a block of the grid has sqrt(unit / kSplit) blocks at least
constexpr int kHeader = 8;        // ints of a piece's header
constexpr int kMaxCluster = 16;   // blocks of a cluster

// ROWS query rows per unit: 16 on the tensor cores, 4 (fp32) on the FMA units.
template <int D, bool F32, int ROWS>
struct Cfg {
  static constexpr bool few = ROWS == 4;
  static constexpr int rows = ROWS;
  static constexpr int keys = few ? 8 : 16;     // of a warp's step
  static constexpr int block = kWarps * keys;   // of a block's step
  static constexpr int es = F32 ? 4 : 2;
  static constexpr int row = D * es;            // bytes of a key
  static constexpr int step = 2 * keys * row;   // keys and values of a warp's step
  // 96 KB of copies for two blocks on an SM each, 192 KB where three steps are
  // too large for that.
  static constexpr int per_sm = step * kWarps * 3 <= 98304 ? 2 : 1;
  static constexpr int stages = (per_sm == 2 ? 98304 : 196608) / (kWarps * step);
  static constexpr int ring = kWarps * stages * step;
  static constexpr int ld = D + 4;              // joined: four rows at a time
  static constexpr int joins = (kWarps * 4 * ld + 2 * kWarps * rows) * 4;
  // fp32: the rows of q in bf16 parts, or a step's weights of each warp.
  static constexpr int extra = few ? kWarps * keys * 16 : F32 ? rows * D * 6 : 0;
  static constexpr int smem = ring + joins + extra;
  static_assert(stages >= 3, "copies in flight");
};

__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ float4 lds4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 numbers as three pairs of bf16 numbers each, 24 bits in all: x =
// h + m + l to 2^-25 of it (Henry, Tang, Heinecke, "Leveraging the bfloat16
// Artificial Intelligence Datatype For Higher-Precision Computations", 2019). Of
// the nine products of two such numbers the six
// largest are taken, so a product is within 2^-23 or so. (tf32 pairs cost as
// many tensor instructions and keep 21 bits: scores of 30 then move weights by
// 7e-6.) Infinities, NaN and what is above bf16's largest number become NaN.
__device__ __forceinline__ void split3(float x, float y, uint32_t &h, uint32_t &m, uint32_t &l) {
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(y), "f"(x));
  x -= __uint_as_float(h << 16);
  y -= __uint_as_float(h & 0xFFFF0000u);
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(m) : "f"(y), "f"(x));
  x -= __uint_as_float(m << 16);
  y -= __uint_as_float(m & 0xFFFF0000u);
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(l) : "f"(y), "f"(x));
}
// d += a b from the parts (0: h, 1: m, 2: l), the smallest products first. The
// tensor cores cut off what they add up, relative to the sum so far: the
// products of 16 terms begin a sum of their own, which is added to d with
// rounding. (Added up in d itself, they lost three times as much as fp32 sums
// with rounding do.)
__device__ __forceinline__ void mma_parts(float (&d)[4], const uint32_t (&a)[3][4],
                                          const uint32_t (&b0)[3], const uint32_t (&b1)[3]) {
  float t[4];
  mma_bf16_16816_zero(t, a[2], b0[0], b1[0]);
  mma_bf16_16816(t, a[0], b0[2], b1[2]);
  mma_bf16_16816(t, a[1], b0[1], b1[1]);
  mma_bf16_16816(t, a[1], b0[0], b1[0]);
  mma_bf16_16816(t, a[0], b0[1], b1[1]);
  mma_bf16_16816(t, a[0], b0[0], b1[0]);
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] += t[i];
}

// Bytes 16-byte piece `c` of key `k` lies at in a step's keys or values: pieces
// are swapped so that no two lanes that read together share a bank. bf16:
// ldmatrix reads a piece of eight keys. fp32: the lanes g < 2, t read the
// pieces .. + t of keys g (keys) or the pieces .. + g of keys 2t (values).
template <int D, bool F32>
__device__ __forceinline__ int key_at(int k, int c) {
  return k * (D * (F32 ? 4 : 2)) + ((F32 ? c ^ ((k & 1) << 2) : c ^ (k & 7)) << 4);
}
template <int D, bool F32>
__device__ __forceinline__ int value_at(int k, int c) {
  return k * (D * (F32 ? 4 : 2)) + ((F32 ? c ^ (((k >> 1) & 3) << 1) : c ^ (k & 7)) << 4);
}

// A unit's place in the line of blocks and what it attends.
struct Unit {
  int b, head, tile;      // sequence, key head, 16-row tile
  int t0, n, len, lo;     // the sequence
  int blocks;             // of 64 keys from lo on, up to the tile's last row
  int last;               // position of the tile's last row: no key above it
};

template <typename C>
struct Line {
  const AttnStreamParams &p;
  int lane;
  __device__ __forceinline__ Seq seq(int i) const {
    return load_seq(p.b, i, p.T, p.window);
  }
  __device__ __forceinline__ int tiles(const Seq &s) const {
    return (s.n * static_cast<int>(p.G.d) + C::rows - 1) / C::rows;
  }
  // Places of each unit in the line: the sequence's blocks, or those that a window
  // spans. What a tile's rows do not reach of them, at the unit's end, is skipped.
  __device__ __forceinline__ int blocks(const Seq &s) const {
    const int all = max(1, (min(s.len, p.cap) - s.lo + C::block - 1) / C::block);
    return min(all, p.span);
  }
  __device__ __forceinline__ int64_t work(const Seq &s) const {
    return int64_t(tiles(s)) * p.kv_heads * blocks(s);
  }
  // All blocks of the line, and of the longest unit; every lane takes part, and
  // keeps one of the first 32 sequences in s0.
  __device__ __forceinline__ int64_t total(Seq &s0, int &longest) const {
    s0 = Seq{0, 0, 0, 0};
    if (lane < p.b.n) s0 = seq(lane);
    int64_t w = work(s0);
    longest = s0.n > 0 ? blocks(s0) : 0;
    for (int i = lane + 32; i < p.b.n; i += 32) {
      const Seq s = seq(i);
      w += work(s);
      if (s.n > 0) longest = max(longest, blocks(s));
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
#pragma unroll
    for (int m = 1; m < 32; m *= 2) w += __shfl_xor_sync(0xffffffffu, w, m);
    return w;
  }
  // The unit that holds block x of the line, and the block's number in it.
  __device__ __forceinline__ void start(Unit &u, int &kb, int64_t x, const Seq &s0) const {
    int64_t before = 0;
    for (int i0 = 0; i0 < p.b.n; i0 += 32) {
      Seq s{0, 0, 0, 0};
      if (i0 == 0)
        s = s0;
      else if (i0 + lane < p.b.n)
        s = seq(i0 + lane);
      const int64_t w = work(s);
      int64_t up = w;
#pragma unroll
      for (int m = 1; m < 32; m *= 2) {
        const int64_t o = __shfl_up_sync(0xffffffffu, up, m);
        if (lane >= m) up += o;
      }
      const unsigned past = __ballot_sync(0xffffffffu, before + up > x);
      if (past) {  // (some lane of some round has it: x is below the total)
        const int l = __ffs(past) - 1;
        const int64_t in = x - before - __shfl_sync(0xffffffffu, up - w, l);
        s = Seq{__shfl_sync(0xffffffffu, s.t0, l), __shfl_sync(0xffffffffu, s.n, l),
                __shfl_sync(0xffffffffu, s.len, l), __shfl_sync(0xffffffffu, s.lo, l)};
        u.b = i0 + l;
        const int nb = blocks(s);
        const int unit = static_cast<int>(Share::div(in, nb));
        kb = static_cast<int>(in - int64_t(unit) * nb);
        enter(u, s, unit);
        return;
      }
      before += __shfl_sync(0xffffffffu, up, 31);
    }
  }
  // Unit `unit` of at most 32 sequences; false: there are not as many.
  __device__ __forceinline__ bool pick(Unit &u, int unit) const {
    Seq s{0, 0, 0, 0};
    if (lane < p.b.n) s = seq(lane);
    const int w = tiles(s) * p.kv_heads;
    int up = w;
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
      const int o = __shfl_up_sync(0xffffffffu, up, m);
      if (lane >= m) up += o;
    }
    const unsigned past = __ballot_sync(0xffffffffu, up > unit);
    if (!past) return false;
    const int l = __ffs(past) - 1;
    s = Seq{__shfl_sync(0xffffffffu, s.t0, l), __shfl_sync(0xffffffffu, s.n, l),
            __shfl_sync(0xffffffffu, s.len, l), __shfl_sync(0xffffffffu, s.lo, l)};
    u.b = l;
    enter(u, s, unit - __shfl_sync(0xffffffffu, up - w, l));
    return true;
  }
  // The tiles come first, last, second, last but one, ..: early ones skip most of
  // their places, late ones none, and parts of the line shall be alike. (An fp32
  // prompt of 1024 tokens, 56 / 8 heads: 485 us, 804 with nothing skipped.)
  __device__ __forceinline__ void enter(Unit &u, const Seq &s, int unit) const {
    const int nt = tiles(s);
    u.head = nt == 1 ? unit : unit / nt;
    const int turn = unit - u.head * nt;
    u.tile = turn & 1 ? nt - 1 - turn / 2 : turn / 2;
    u.t0 = s.t0;
    u.n = s.n;
    u.len = s.len;
    u.lo = 0;
    if (p.window > 0)
      u.lo = max(0, max(0, s.len - s.n + p.G.div(u.tile * C::rows)) - p.window + 1) & ~15;
    u.last = max(s.len - s.n + min(s.n - 1, p.G.div(u.tile * C::rows + C::rows - 1)), -1);
    u.blocks = min(blocks(s), max(0, u.last - u.lo) / C::block + 1);
  }
  __device__ __forceinline__ Seq seq_of(const Unit &u) const {
    return Seq{u.t0, u.n, u.len, first_key(u.n, u.len, p.window)};
  }
  // Places of u past its blocks.
  __device__ __forceinline__ int spare(const Unit &u) const {
    return blocks(seq_of(u)) - u.blocks;
  }
  // The unit after u (there is one).
  __device__ __forceinline__ void next(Unit &u) const {
    Seq s = seq_of(u);
    const int nt = tiles(s);
    int unit = u.head * nt + (u.tile < (nt + 1) / 2 ? 2 * u.tile : 2 * (nt - u.tile) - 1) + 1;
    while (unit >= tiles(s) * p.kv_heads) {
      unit = 0;
      s = seq(++u.b);
    }
    enter(u, s, unit);
  }
};

template <int D, bool F32, int ROWS, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, Cfg<D, F32, ROWS>::per_sm)
    stream_kernel(const __grid_constant__ AttnStreamParams p) {
  using C = Cfg<D, F32, ROWS>;
  using E = typename std::conditional<F32, float, uint16_t>::type;
  constexpr int kRows = ROWS, kWarpKeys = C::keys, kBlockKeys = C::block;
  constexpr int kPieces = C::row / 16;            // 16-byte pieces of a key
  constexpr int kKeysAtOnce = 32 / kPieces > 0 ? 32 / kPieces : 1;
  constexpr int kSteps = kWarpKeys / kKeysAtOnce;  // copies per lane, keys or values
  constexpr int kQ = F32 ? 1 : D / 4;              // query registers
  constexpr int kO = C::few ? 1 : D / 8;           // 8-wide column tiles
  constexpr int kPer = D / 32;                     // columns of a lane, joining (few: all along)
  extern __shared__ __align__(128) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  unsigned char *ring = smem + warp * (C::stages * C::step);
  const uint32_t ring_u = smem_addr(ring);
  float *join = reinterpret_cast<float *>(smem + C::ring);  // [warp][4 rows][ld]
  float *join_m = join + kWarps * 4 * C::ld, *join_l = join_m + kWarps * kRows;
  uint4 *qparts = reinterpret_cast<uint4 *>(smem + C::ring + C::joins);  // [d / 16][part][lane]
  float4 *weights_s = reinterpret_cast<float4 *>(smem + C::ring + C::joins) + warp * kWarpKeys;

  grid_dependency_wait();
  grid_dependents_launch();

  const Line<C> line{p, lane};
  Unit fu;
  int fk, slot = 0, rank = 0;
  int64_t x0, x1, total = 0;
  int *header = nullptr;
  if constexpr (CLUSTER) {
    const int which = blockIdx.x / p.cluster;
    rank = blockIdx.x - which * p.cluster;
    if (!line.pick(fu, which)) return;  // (the whole cluster)
    const Share share(fu.blocks, p.cluster);
    x0 = fk = static_cast<int>(share.first(rank));
    x1 = share.first(rank + 1);
  } else {
    Seq s0;
    int longest;
    total = line.total(s0, longest);
    // Of a long unit the pieces take as long to join as to make when a block of the
    // grid has sqrt(unit / kSplit) blocks of the line (16 rows over 16000 keys: 16 us,
    // 30 with a block each, joined by one block; over 2000 9 either way).
    const int least = max(1, static_cast<int>(sqrtf(longest * (1.f / kSplit)) + 0.5f));
    const int parts =
        static_cast<int>(min(int64_t(gridDim.x), (total + least - 1) / least));
    header = p.headers + blockIdx.x * kHeader;
    if (static_cast<int>(blockIdx.x) >= parts) {
      if (threadIdx.x == 0) header[0] = 0;
      return;
    }
    if (threadIdx.x == 0) header[5] = parts;  // for this thread, at the end
    const Share share(total, parts);
    x0 = share.first(blockIdx.x);
    x1 = share.first(blockIdx.x + 1);
    line.start(fu, fk, x0, s0);
    if (fk >= fu.blocks) {  // among places that are skipped
      x0 += line.spare(fu) - (fk - fu.blocks);
      if (x0 >= x1) {
        if (threadIdx.x == 0) header[0] = 0;
        return;
      }
      line.next(fu);
      fk = 0;
    }
  }

  // ---- copies ---------------------------------------------------------------------
  int64_t fx = x0;
  Unit u = fu;
  int kb = fk;
  // Lane l holds the page of this warp's keys in block page0 + l of the unit.
  int page0 = 0, pages = -1;
  auto load_pages = [&](int k0) {
    page0 = k0;
    const int j = fu.lo + min(k0 + lane, fu.blocks) * kBlockKeys + warp * kWarpKeys;
    // The position of the first row that has one.
    const int first = max(fu.len - fu.n + p.G.div(fu.tile * kRows), 0);
    pages = -1;
    if (k0 + lane < fu.blocks && j < min(fu.len, p.cap) && j <= fu.last &&
        (p.window == 0 || j + kWarpKeys > first - p.window + 1)) {
      pages = p.b.table[fu.b * p.b.table_stride + p.page_size.div(j)];
      if (pages < 0 || pages >= p.pages) pages = -1;
    }
  };
  load_pages(fk);
  // Bit s: stage s holds keys that can be attended.
  uint32_t held = 0;
  auto fetch = [&] {
    if (fx < x1) {
      if (fk - page0 >= 32) load_pages(fk);
      const int page = __shfl_sync(0xffffffffu, pages, fk - page0);
      held &= ~(1u << slot);
      if (page >= 0) {
        held |= 1u << slot;
        const int j = fu.lo + fk * kBlockKeys + warp * kWarpKeys;
        const int at = j - p.page_size.div(j) * p.page_size.d, left = min(fu.len, p.cap) - j;
        const int piece = lane % kPieces, first = lane / kPieces;
        const E *k = static_cast<const E *>(p.k.p) + page * p.k.ps + fu.head * p.k.hs +
                     (at + first) * p.k.ts + piece * (16 / C::es);
        const E *v = static_cast<const E *>(p.v.p) + page * p.v.ps + fu.head * p.v.hs +
                     (at + first) * p.v.ts + piece * (16 / C::es);
        const uint32_t dst = ring_u + slot * C::step;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const int key = first + i * kKeysAtOnce;
          cp16_or_zero(dst + key_at<D, F32>(key, piece), k, key < left);
          k += kKeysAtOnce * p.k.ts;
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const int key = first + i * kKeysAtOnce;
          cp16_or_zero(dst + C::step / 2 + value_at<D, F32>(key, piece), v, key < left);
          v += kKeysAtOnce * p.v.ts;
        }
      }
      slot = slot == C::stages - 1 ? 0 : slot + 1;
      ++fx;
      if (++fk == fu.blocks && !CLUSTER) {
        fx += line.spare(fu);
        if (fx < x1) {
          line.next(fu);
          fk = 0;
          load_pages(0);
        }
      }
    }
    cp_commit();
  };
  // ---- the unit's rows ---------------------------------------------------------------
  uint32_t q[kQ];
  float4 qf[C::few ? 4 : 1][C::few ? kPer : 1];
  int pos0 = 0, pos1 = 0;  // positions of the rows g and g + 8, few: lane & 3 (-1: no row)
  auto load_rows = [&] {
    auto row_of = [&](int r, int &pos) -> const E * {
      const int i = u.tile * kRows + r, tok = p.G.div(i);
      if (tok >= u.n) {
        pos = -1;
        return nullptr;
      }
      pos = max(-1, u.len - u.n + tok);
      return static_cast<const E *>(p.q.p) + int64_t(u.t0 + tok) * p.q.ts +
             int64_t((u.head - tok) * static_cast<int>(p.G.d) + i) * p.q.hs;
    };
    if constexpr (C::few) {
      // Lane `sub` of eight has the pieces sub, sub + 8, .. of all four rows.
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        int pos;
        const E *a = row_of(r, pos);
        if (r == (lane & 3)) pos0 = pos;
#pragma unroll
        for (int c = 0; c < kPer; ++c)
          qf[r][c] = a ? *reinterpret_cast<const float4 *>(a + 4 * ((lane & 7) + 8 * c))
                       : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      return;
    }
    const E *a = row_of(g, pos0), *b = row_of(g + 8, pos1);
    if constexpr (F32) {
      // Each warp makes a quarter of the parts, in the order of the MMAs'
      // registers. The k order within 16 elements is the keys': a lane's are 4t
      // to 4t + 3.
      for (int d = warp; d < D / 16; d += kWarps) {
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 x = a ? *reinterpret_cast<const float4 *>(a + 16 * d + 4 * t) : z;
        const float4 y = b ? *reinterpret_cast<const float4 *>(b + 16 * d + 4 * t) : z;
        uint32_t w[3][4];
        split3(x.x, x.y, w[0][0], w[1][0], w[2][0]);
        split3(y.x, y.y, w[0][1], w[1][1], w[2][1]);
        split3(x.z, x.w, w[0][2], w[1][2], w[2][2]);
        split3(y.z, y.w, w[0][3], w[1][3], w[2][3]);
#pragma unroll
        for (int i = 0; i < 3; ++i)
          qparts[(d * 3 + i) * 32 + lane] = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        const int c = 16 * s + 2 * t;
        q[4 * s] = a ? *reinterpret_cast<const uint32_t *>(a + c) : 0u;
        q[4 * s + 1] = b ? *reinterpret_cast<const uint32_t *>(b + c) : 0u;
        q[4 * s + 2] = a ? *reinterpret_cast<const uint32_t *>(a + c + 8) : 0u;
        q[4 * s + 3] = b ? *reinterpret_cast<const uint32_t *>(b + c + 8) : 0u;
      }
    }
  };

  float o[kO][4], m0, m1, l0, l1;
  float acc[C::few ? 4 : 1][kPer];  // few: four rows of a lane's columns
  auto clear = [&] {
#pragma unroll
    for (int r = 0; r < (C::few ? 4 : 1); ++r)
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[r][e] = 0.f;
#pragma unroll
    for (int i = 0; i < kO; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
  };
  // A masked value that is not finite would still make 0 * inf: such values of a
  // step become 0, and the rows that do attend their keys (returned) NaN.
  auto tidy_values = [&](uint32_t vs) {
    unsigned bad = 0;
#pragma unroll 2
    for (int i = 0; i < kSteps; ++i) {
      const int key = lane / kPieces + i * kKeysAtOnce;
      unsigned char *at = ring + (vs - ring_u) + value_at<D, F32>(key, lane % kPieces);
      uint4 w = *reinterpret_cast<uint4 *>(at);
      bool hit = false;
      auto tidy = [&](uint32_t &r) {
        if constexpr (F32) {
          if ((r & 0x7F800000u) == 0x7F800000u) {
            r = 0;
            hit = true;
          }
        } else {
          if ((r & 0x7F80u) == 0x7F80u) {
            r &= 0xFFFF0000u;
            hit = true;
          }
          if ((r & 0x7F800000u) == 0x7F800000u) {
            r &= 0xFFFFu;
            hit = true;
          }
        }
      };
      tidy(w.x);
      tidy(w.y);
      tidy(w.z);
      tidy(w.w);
      if (hit) {
        *reinterpret_cast<uint4 *>(at) = w;
        bad |= 1u << key;
      }
    }
    bad = __reduce_or_sync(0xffffffffu, bad);
    __syncwarp();
    return bad;
  };
  // (Their loads are under way while the first pages are looked up.)
  load_rows();
  for (int i = 0; i < C::stages - 1; ++i) fetch();
  clear();
  int piece0 = kb, cslot = 0;

  for (int64_t x = x0;;) {
    if (!CLUSTER || x < x1) {
      cp_wait<C::stages - 2>();
      __syncwarp();
      const bool there = (held >> cslot) & 1;
      fetch();
      const uint32_t ks = ring_u + cslot * C::step, vs = ks + C::step / 2;
      cslot = cslot == C::stages - 1 ? 0 : cslot + 1;
      const int j0 = u.lo + kb * kBlockKeys + warp * kWarpKeys;
      const int top = u.last, bottom = u.len - u.n + p.G.div(u.tile * kRows);
      const bool masked = j0 + kWarpKeys - 1 > bottom || (p.window > 0 && j0 <= top - p.window);
      if constexpr (C::few) {
        if (there) {
          // Eight lanes per key, four keys at a time: a lane's pieces of a key
          // times those of the four rows; then the lanes add up by halves, so that
          // lane `lane` has the score of row lane & 3 and key 4 (lane >> 2 & 1) +
          // (lane >> 3).
          float s[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
            for (int c = 0; c < kPer; ++c) {
              const float4 k4 = lds4(ks + key_at<D, F32>(4 * i + (lane >> 3), (lane & 7) + 8 * c));
#pragma unroll
              for (int r = 0; r < 4; ++r)
                s[i][r] += qf[r][c].x * k4.x + qf[r][c].y * k4.y + qf[r][c].z * k4.z +
                           qf[r][c].w * k4.w;
            }
          }
          float u4[4], u2[2];
          const bool b2 = lane & 4, b1 = lane & 2, b0 = lane & 1;
#pragma unroll
          for (int r = 0; r < 4; ++r)
            u4[r] = (b2 ? s[1][r] : s[0][r]) +
                    __shfl_xor_sync(0xffffffffu, b2 ? s[0][r] : s[1][r], 4);
#pragma unroll
          for (int r = 0; r < 2; ++r)
            u2[r] = (b1 ? u4[2 + r] : u4[r]) +
                    __shfl_xor_sync(0xffffffffu, b1 ? u4[r] : u4[2 + r], 2);
          float sc = (b0 ? u2[1] : u2[0]) + __shfl_xor_sync(0xffffffffu, b0 ? u2[0] : u2[1], 1);
          if (p.negative) sc = -sc;
          const int key = 4 * ((lane >> 2) & 1) + (lane >> 3), j = j0 + key;
          if (masked) {
            const unsigned bad = tidy_values(vs);
            if (j > pos0 || (p.window > 0 && j <= pos0 - p.window))
              sc = -INFINITY;
            else if ((bad >> key) & 1)
              sc = NAN;
          }
          float n0 = sc;
#pragma unroll
          for (int k = 4; k < 32; k *= 2) n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, k));
          n0 = fmaxf(m0, n0);
          const float z0 = n0 == -INFINITY ? 0.f : n0;
          if (__any_sync(0xffffffffu, n0 != m0)) {
            const float f0 = exp2_fast((m0 - z0) * p.scale);
            m0 = n0;
            l0 *= f0;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float f = __shfl_sync(0xffffffffu, f0, r);
#pragma unroll
              for (int e = 0; e < kPer; ++e) acc[r][e] *= f;
            }
          }
          const float w = exp2_fast((sc - z0) * p.scale);
          l0 += w;
          reinterpret_cast<float *>(weights_s + key)[lane & 3] = w;
          __syncwarp();
          // A lane's columns of every key's values, times the four rows' weights.
#pragma unroll
          for (int k = 0; k < kWarpKeys; ++k) {
            const float4 w4 = weights_s[k];
            float v[kPer];
            const uint32_t at = vs + value_at<D, F32>(k, lane * kPer / 4) + lane * kPer % 4 * 4;
            if constexpr (kPer == 4) {
              const float4 x = lds4(at);
              v[0] = x.x;
              v[1] = x.y;
              v[2] = x.z;
              v[3] = x.w;
            } else {
              asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];"
                           : "=f"(v[0]), "=f"(v[1])
                           : "r"(at)
                           : "memory");
            }
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
              acc[0][e] += w4.x * v[e];
              acc[1][e] += w4.y * v[e];
              acc[2][e] += w4.z * v[e];
              acc[3][e] += w4.w * v[e];
            }
          }
        }
      } else if (there) {
        // ---- scores of 16 rows and 16 keys
        float s[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
        if constexpr (F32) {
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            uint32_t a[3][4];
#pragma unroll
            for (int i = 0; i < 3; ++i) {
              const uint4 w = qparts[(d * 3 + i) * 32 + lane];
              a[i][0] = w.x;
              a[i][1] = w.y;
              a[i][2] = w.z;
              a[i][3] = w.w;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float4 k4 = lds4(ks + key_at<D, F32>(8 * i + g, 4 * d + t));
              uint32_t b0[3], b1[3];
              split3(k4.x, k4.y, b0[0], b0[1], b0[2]);
              split3(k4.z, k4.w, b1[0], b1[1], b1[2]);
              mma_parts(s[i], a, b0, b1);
            }
          }
        } else {
          const int mi = lane >> 3, kr = (mi >> 1) * 8 + (lane & 7);
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            uint32_t k4[4];
            ldsm4(ks + key_at<D, F32>(kr, 2 * d + (mi & 1)), k4);
            const uint32_t a[4] = {q[4 * d], q[4 * d + 1], q[4 * d + 2], q[4 * d + 3]};
            mma_bf16_16816(s[0], a, k4[0], k4[1]);
            mma_bf16_16816(s[1], a, k4[2], k4[3]);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][e] = p.negative ? -s[i][e] : s[i][e];
        // ---- masks, where some row of the tile does not attend some key
        if (masked) {
          const unsigned bad = tidy_values(vs);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = 8 * i + 2 * t + (e & 1), j = j0 + key, pos = e < 2 ? pos0 : pos1;
              if (j > pos || (p.window > 0 && j <= pos - p.window))
                s[i][e] = -INFINITY;
              else if ((bad >> key) & 1)
                s[i][e] = NAN;
            }
        }
        // ---- running maximum and sum. Differences from the maximum are scaled,
        // not scores: the rounding of a large score's product with the scale
        // would move its weight.
        float n0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
        float n1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
        n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, 1));
        n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, 1));
        n0 = fmaxf(m0, fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, 2)));
        n1 = fmaxf(m1, fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, 2)));
        const float z0 = n0 == -INFINITY ? 0.f : n0, z1 = n1 == -INFINITY ? 0.f : n1;
        if (__any_sync(0xffffffffu, n0 != m0 || n1 != m1)) {
          const float f0 = exp2_fast((m0 - z0) * p.scale), f1 = exp2_fast((m1 - z1) * p.scale);
          m0 = n0;
          m1 = n1;
          l0 *= f0;
          l1 *= f1;
#pragma unroll
          for (int i = 0; i < kO; ++i) {
            o[i][0] *= f0;
            o[i][1] *= f0;
            o[i][2] *= f1;
            o[i][3] *= f1;
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          s[i][0] = exp2_fast((s[i][0] - z0) * p.scale);
          s[i][1] = exp2_fast((s[i][1] - z0) * p.scale);
          s[i][2] = exp2_fast((s[i][2] - z1) * p.scale);
          s[i][3] = exp2_fast((s[i][3] - z1) * p.scale);
          l0 += s[i][0] + s[i][1];
          l1 += s[i][2] + s[i][3];
        }
        // ---- weights times values
        if constexpr (F32) {
          uint32_t a[3][4];
          split3(s[0][0], s[0][1], a[0][0], a[1][0], a[2][0]);
          split3(s[0][2], s[0][3], a[0][1], a[1][1], a[2][1]);
          split3(s[1][0], s[1][1], a[0][2], a[1][2], a[2][2]);
          split3(s[1][2], s[1][3], a[0][3], a[1][3], a[2][3]);
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            float v[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int key = 2 * t + (k & 1) + 8 * (k >> 1);
              const float4 w = lds4(vs + value_at<D, F32>(key, 8 * i + g));
              v[k][0] = w.x;
              v[k][1] = w.y;
              v[k][2] = w.z;
              v[k][3] = w.w;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t b0[3], b1[3];
              split3(v[0][e], v[1][e], b0[0], b0[1], b0[2]);
              split3(v[2][e], v[3][e], b1[0], b1[1], b1[2]);
              mma_parts(o[4 * i + e], a, b0, b1);
            }
          }
        } else {
          // Weights are at most 1 and rounded once to bf16, the type of the values
          // that they are multiplied by (an MMA takes one type; a second part of the
          // weights would be a second MMA): 2^-8 of each term, and errors of 0.0017
          // against 64 bits where fp32 weights have 0.00165, results rounded to bf16.
          // Their sum takes them unrounded.
          const uint32_t a[4] = {bf16_bits(s[0][0]) | (bf16_bits(s[0][1]) << 16),
                                 bf16_bits(s[0][2]) | (bf16_bits(s[0][3]) << 16),
                                 bf16_bits(s[1][0]) | (bf16_bits(s[1][1]) << 16),
                                 bf16_bits(s[1][2]) | (bf16_bits(s[1][3]) << 16)};
          const int mi = lane >> 3, vr = (mi & 1) * 8 + (lane & 7);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            uint32_t v4[4];
            ldsm4_t(vs + value_at<D, F32>(vr, 2 * i + (mi >> 1)), v4);
            if constexpr (CLUSTER) {
              mma_bf16_16816(o[2 * i], a, v4[0], v4[1]);
              mma_bf16_16816(o[2 * i + 1], a, v4[2], v4[3]);
            } else {
              // A sum of 16 terms of its own, added with rounding: the tensor cores
              // cut off what they add, relative to the sum so far, and 4 M keys of
              // equal weight in one block came out 0.4 % low. (A cluster's warps have
              // 4096 steps at most, some 2^-12, and one sequence of 4097 tokens takes
              // 0.3 us less without.)
              float x[2][4];
              mma_bf16_16816_zero(x[0], a, v4[0], v4[1]);
              mma_bf16_16816_zero(x[1], a, v4[2], v4[3]);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                o[2 * i][e] += x[0][e];
                o[2 * i + 1][e] += x[1][e];
              }
            }
          }
        }
      }
      __syncwarp();
      ++kb;
      ++x;
      if (kb < u.blocks && x < x1) continue;
    }

    // ---- end of a piece: the warps' sums joined, four rows at a time ---------------
    if constexpr (C::few) {
#pragma unroll
      for (int k = 4; k < 32; k *= 2) l0 += __shfl_xor_sync(0xffffffffu, l0, k);
      if (lane < 4) {
        join_m[warp * kRows + lane] = m0;
        join_l[warp * kRows + lane] = l0;
      }
    } else {
      l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
      if (t == 0) {
        join_m[warp * kRows + g] = m0;
        join_m[warp * kRows + g + 8] = m1;
        join_l[warp * kRows + g] = l0;
        join_l[warp * kRows + g + 8] = l1;
      }
    }
    const bool begins = piece0 == 0, whole = begins && kb == u.blocks;
    const int64_t piece = int64_t(blockIdx.x) * 2 + (begins ? 1 : 0);
    float *part = p.parts + piece * (kRows * (D + 2));
    if constexpr (CLUSTER) {  // into shared memory: the ring's place, which is done with
      part = reinterpret_cast<float *>(smem);
      cp_wait<0>();
      __syncthreads();
    }
    const int live = min(kRows, u.n * static_cast<int>(p.G.d) - u.tile * kRows);
#pragma unroll
    for (int half = 0; half < (C::few ? 1 : 2); ++half) {
#pragma unroll 1
      for (int quad = 0; quad < (C::few ? 4 : 8); quad += 4) {
        if (8 * half + quad >= live) break;
        if constexpr (C::few) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < kPer; ++e)
              join[(warp * 4 + r) * C::ld + lane * kPer + e] = acc[r][e];
        } else if ((g & 4) == quad) {
          float *mine = join + (warp * 4 + (g & 3)) * C::ld;
#pragma unroll
          for (int c = 0; c < kO; ++c) {
            if constexpr (F32) {
              // Column 2t + e of tile 4 i + c is d = 32 i + 8 t + 4 e + c.
              mine[c / 4 * 32 + 8 * t + (c & 3)] = o[c][2 * half];
              mine[c / 4 * 32 + 8 * t + 4 + (c & 3)] = o[c][2 * half + 1];
            } else {
              *reinterpret_cast<float2 *>(mine + 8 * c + 2 * t) =
                  make_float2(o[c][2 * half], o[c][2 * half + 1]);
            }
          }
        }
        __syncthreads();
        // A warp per row, kPer columns a lane.
        const int row = 8 * half + quad + warp;
        float m = -INFINITY, l = 0.f, f[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, join_m[w * kRows + row]);
        const float z = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          f[w] = exp2_fast((join_m[w * kRows + row] - z) * p.scale);
          l += f[w] * join_l[w * kRows + row];
        }
        float a[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) a[e] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
#pragma unroll
          for (int e = 0; e < kPer; e += 2) {
            const float2 v = *reinterpret_cast<const float2 *>(join + (w * 4 + warp) * C::ld +
                                                               lane * kPer + e);
            a[e] += f[w] * v.x;
            a[e + 1] += f[w] * v.y;
          }
        if (CLUSTER || !whole) {
#pragma unroll
          for (int e = 0; e < kPer; e += 2)
            *reinterpret_cast<float2 *>(part + row * D + lane * kPer + e) =
                make_float2(a[e], a[e + 1]);
          if (lane == 0) {
            part[kRows * D + row] = m;
            part[kRows * D + kRows + row] = l;
          }
        } else if (row < live) {
          const int i = u.tile * kRows + row, tok = p.G.div(i);
          E *out = static_cast<E *>(p.o.p) + int64_t(u.t0 + tok) * p.o.ts +
                   int64_t((u.head - tok) * static_cast<int>(p.G.d) + i) * p.o.hs + lane * kPer;
          // No key attended: zeros.
          const float inv = m == -INFINITY && l == 0.f ? 0.f : 1.f / l;
#pragma unroll
          for (int e = 0; e < kPer; e += 2) {
            if constexpr (F32)
              *reinterpret_cast<float2 *>(out + e) = make_float2(a[e] * inv, a[e + 1] * inv);
            else
              *reinterpret_cast<uint32_t *>(out + e) =
                  bf16_bits(a[e] * inv) | (bf16_bits(a[e + 1] * inv) << 16);
          }
        }
        __syncthreads();
      }
    }
    if constexpr (CLUSTER) {
      // Block `rank` joins the rows rank, rank + p.cluster, .. of all blocks, a
      // thread per column; lane r has the maximum and the sum of block r.
      cluster_sync_all();
#pragma unroll 1
      for (int row = rank; row < live; row += p.cluster) {
        const int d = threadIdx.x;
        const bool has = lane < p.cluster;
        const float mr = has ? ld_dsmem_f32(part + kRows * D + row, lane) : -INFINITY;
        float l = has ? ld_dsmem_f32(part + kRows * D + kRows + row, lane) : 0.f;
        float v[kMaxCluster];
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c)
          v[c] = d < D && c < p.cluster ? ld_dsmem_f32(part + row * D + d, c) : 0.f;
        float m = mr;
#pragma unroll
        for (int k = 1; k < 32; k *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
        const float f = exp2_fast((mr - (m == -INFINITY ? 0.f : m)) * p.scale);
        l *= f;
        float a = 0.f;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) a += __shfl_sync(0xffffffffu, f, c) * v[c];
#pragma unroll
        for (int k = 1; k < 32; k *= 2) l += __shfl_xor_sync(0xffffffffu, l, k);
        a *= m == -INFINITY && l == 0.f ? 0.f : 1.f / l;
        const int i = u.tile * kRows + row, tok = p.G.div(i);
        E *out = static_cast<E *>(p.o.p) + int64_t(u.t0 + tok) * p.o.ts +
                 int64_t((u.head - tok) * static_cast<int>(p.G.d) + i) * p.o.hs + d;
        if (d < D) {
          if constexpr (F32)
            *out = a;
          else
            *out = static_cast<uint16_t>(bf16_bits(a));
        }
      }
      cluster_sync_all();  // no block leaves while another reads its memory
      return;
    }
    if (kb == u.blocks) x += line.spare(u);
    if (x >= x1) {
      // A unit that begins here and goes on: the blocks after this one that
      // have a piece of it.
      if (threadIdx.x == 0) {
        int more = 0;
        if (begins && !whole) {
          const int64_t end = x1 + u.blocks - kb;  // first place past the unit's blocks
          more = Share(total, header[5]).owner(end - 1) - static_cast<int>(blockIdx.x);
        }
        header[0] = more;
        header[1] = u.t0;
        header[2] = u.n;
        header[3] = u.head;
        header[4] = u.tile;
      }
      break;
    }
    line.next(u);
    kb = piece0 = 0;
    load_rows();
    clear();
  }
  cp_wait<0>();
}

// Joins the pieces of a unit: the one that begins at the end of block c's part
// and the continuations at the start of the parts after it. Four rows a block
// (a lone unit's pieces are too many for one SM to read: 33 us for 400 of 16 rows,
// 17 so, with fewer pieces), a thread per column of a row, the loads of 32 pieces in flight together, lane c with the
// maximum and the sum of weights of piece c. Bound by latency (a launch, the
// header, the pieces: each the best part of a microsecond), so the code is kept
// short as well: fetching it is part of that.
constexpr int kJoinThreads = 512, kJoinBlocks = 4;
template <int D, bool F32, int ROWS>
__global__ void __launch_bounds__(kJoinThreads)
    combine_kernel(const __grid_constant__ AttnStreamParams p) {
  using E = typename std::conditional<F32, float, uint16_t>::type;
  constexpr int kRows = ROWS;
  constexpr int64_t kPart = kRows * (D + 2);
  const int lane = threadIdx.x & 31, d = threadIdx.x % D;
  grid_dependency_wait();
  grid_dependents_launch();
  const int *h = p.headers + blockIdx.x * kHeader;
  const int more = h[0];
  if (more == 0) return;
  const int t0 = h[1], n = h[2], head = h[3], tile = h[4];
  // Piece 0, and pieces 1, 2, .. two apart from the next block's on.
  const float *parts = p.parts + int64_t(blockIdx.x) * 2 * kPart;
  auto piece = [&](int c) { return parts + (c == 0 ? kPart : c * 2 * kPart); };
#pragma unroll 1
  for (int row = blockIdx.y * (kJoinThreads / D) + threadIdx.x / D; row < kRows;
       row += gridDim.y * (kJoinThreads / D)) {
    const int i = tile * kRows + row, tok = p.G.div(i);
    if (tok >= n) return;
    float m = -INFINITY, l = 0.f, a = 0.f;
#pragma unroll 1
    for (int c0 = 0; c0 <= more; c0 += 32) {
      const bool there = c0 + lane <= more;
      const float *x = piece(there ? c0 + lane : 0) + kRows * D + row;
      const float mc = there ? x[0] : -INFINITY, lc = there ? x[kRows] : 0.f;
      float v[32];
#pragma unroll
      for (int c = 0; c < 32; ++c) v[c] = c0 + c <= more ? piece(c0 + c)[row * D + d] : 0.f;
      float top = mc;
#pragma unroll
      for (int s = 1; s < 32; s *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
      top = fmaxf(top, m);
      const float z = top == -INFINITY ? 0.f : top;
      const float old = exp2_fast((m - z) * p.scale), f = exp2_fast((mc - z) * p.scale);
      m = top;
      a *= old;
      l = l * old + f * lc;
#pragma unroll
      for (int c = 0; c < 32; ++c) a += __shfl_sync(0xffffffffu, f, c) * v[c];
    }
#pragma unroll
    for (int s = 1; s < 32; s *= 2) l += __shfl_xor_sync(0xffffffffu, l, s);
    a *= m == -INFINITY && l == 0.f ? 0.f : 1.f / l;
    E *out = static_cast<E *>(p.o.p) + int64_t(t0 + tok) * p.o.ts +
             int64_t((head - tok) * static_cast<int>(p.G.d) + i) * p.o.hs + d;
    if constexpr (F32)
      *out = a;
    else
      *out = static_cast<uint16_t>(bf16_bits(a));
  }
}

// Blocks of the grid, at most two on an SM.
int grid_blocks(int per_sm) { return std::max(1, sm_count()) * per_sm; }

// Clusters of `kernel` that the current device holds at once (asked once per
// device; 0: none, or the question failed).
template <typename Kernel>
int clusters_at_once(Kernel kernel, const cudaLaunchConfig_t &cfg, std::atomic<int> (&known)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev].load(std::memory_order_acquire);
  if (n) return n - 1;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
          cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  known[dev].store(n + 1, std::memory_order_release);
  return n;
}

template <int D, bool F32, int ROWS>
cudaError_t run(AttnStreamParams p, bool pdl, cudaStream_t stream) {
  using C = Cfg<D, F32, ROWS>;
  constexpr int kRows = ROWS;
  p.span = kMaxPositions;
  // From a multiple of 16 at or below the first row's window to the last row.
  if (p.window > 0)
    p.span = static_cast<int>(
        (int64_t(p.window) + (kRows - 1) / p.G.d + 1 + 15 + C::block - 1) / C::block);
  // The most units that T rows of n sequences make.
  const int64_t few = std::min<int64_t>(p.b.n, p.T);
  const int64_t units =
      (int64_t(p.T) * p.G.d + (kRows - 1) * few) / kRows * p.kv_heads;
  for (int size = kMaxCluster; size >= 8 && p.b.n <= 32 && units <= 64; size /= 2) {
    // Clusters cannot share a long sequence out over all SMs: it has its own
    // units' blocks, some 45 GB/s each, where the line reads at 6500. The line
    // takes 4.3 us more of launch and joining. (The table's width stands for the
    // lengths, which the host does not know: with tables wider than some 53000 tokens,
    // 8 key heads of 128, a short sequence takes the line too.)
    const double bytes = 2.0 * std::min<double>(p.cap, double(p.span) * C::block) * p.kv_heads * C::row;
    const double rate = std::min(6500.0, 45.0 * p.kv_heads * size);
    if (bytes * 1e-3 * (1 / rate - 1 / 6500.0) > 4.3) continue;
    // bf16: sums of the tensor cores stay short (see the product with the values).
    if (!F32 && std::min<double>(p.cap, double(p.span) * C::block) > 4096.0 * C::block * size)
      continue;
    auto *kernel = stream_kernel<D, F32, ROWS, true>;
    static std::atomic<unsigned long long> done{0};
    static std::atomic<int> known[2][64];
    cudaError_t e = ensure_smem_limit(kernel, C::smem, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(units * size));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (clusters_at_once(kernel, cfg, known[size == kMaxCluster]) < units) continue;
    cfg.numAttrs = pdl ? 2 : 1;
    AttnStreamParams q = p;
    q.cluster = size;
    return cudaLaunchKernelEx(&cfg, kernel, q);
  }
  auto *kernel = stream_kernel<D, F32, ROWS, false>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = ensure_smem_limit(kernel, C::smem, done);
  if (e != cudaSuccess) return e;
  const int grid = grid_blocks(C::per_sm);
  e = launch_after(kernel, dim3(grid), kThreads, C::smem, pdl, stream, p);
  if (e != cudaSuccess) return e;
  return launch_after(combine_kernel<D, F32, ROWS>, dim3(grid, kJoinBlocks), kJoinThreads, 0, pdl,
                      stream, p);
}

size_t header_bytes(int grid) { return (size_t(grid) * kHeader * 4 + 255) & ~size_t(255); }

}  // namespace

size_t stream_workspace_bytes(int D) {
  const int grid = grid_blocks(2);
  return header_bytes(grid) + size_t(grid) * 2 * 16 * (D + 2) * 4;
}

cudaError_t launch_attn_stream(const AttnArgs &a, cudaStream_t stream) {
  AttnStreamParams p{};
  p.q = a.q;
  p.o = a.o;
  p.k = a.c.k;
  p.v = a.c.v;
  p.pages = static_cast<int>(a.c.pages);
  p.page_size = FastDiv(a.c.page_size);
  p.kv_heads = a.c.heads;
  p.G = FastDiv(a.q.n / a.c.heads);
  p.b = a.b;
  p.T = static_cast<int>(a.T);
  p.cap = static_cast<int>(int64_t(a.b.table_pages) * a.c.page_size);
  p.window = window_of(a.window);
  // Weights are powers of two, of (score - maximum) * |scale| log2(e).
  // (Kept off 0 and infinity: what a masked score, -inf, is multiplied by.)
  p.scale = static_cast<float>(
      std::min(std::max(std::fabs(static_cast<double>(a.scale)) * M_LOG2E, 1e-37), 3e38));
  p.negative = a.scale < 0.f;
  p.headers = reinterpret_cast<int *>(a.ws);
  p.parts = reinterpret_cast<float *>(a.ws + header_bytes(grid_blocks(2)));
  const bool wide = a.c.D == 128;
  if (!a.f32)
    return wide ? run<128, false, 16>(p, a.pdl, stream) : run<64, false, 16>(p, a.pdl, stream);
  // Four rows a sequence or fewer: fp32 products on the FMA units, some 340
  // instructions for 8 keys, where bf16 parts take 500 for the tensor cores,
  // whose other rows would be empty, and half of the shared memory. Measured
  // with 2 query heads per key head, 8 of those (us, FMA / tensor cores): one
  // sequence of 2049 tokens, 2 rows 9.5 / 14.3, 8 rows 12.3 / 14.6, 16 rows of
  // 8000 37 / 32; 16 sequences of 2049, 4 rows each 48 / 66, 8 rows 72 / 68.
  if (a.T * p.G.d <= std::max<int64_t>(8, 4 * std::min<int64_t>(a.b.n, a.T)))
    return wide ? run<128, true, 4>(p, a.pdl, stream) : run<64, true, 4>(p, a.pdl, stream);
  return wide ? run<128, true, 16>(p, a.pdl, stream) : run<64, true, 16>(p, a.pdl, stream);
}

}  // namespace mnb
