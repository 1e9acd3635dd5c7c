// Host-side launch interfaces of the attention block's kernels: rotary tables,
// norms and rotation of queries and keys, appending to a paged cache and
// attention over its pages. Arguments arrive here already validated by the C
// ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "mnb_common.cuh"

namespace mnb {

constexpr int kMaxHeadDim = 256;  // of norms, rotation and appending
constexpr int kMaxPairs = kMaxHeadDim / 2;

// Rows of heads: element (token, head, d) at token * ts + head * hs + d.
struct Heads {
  void *p;
  int64_t ts, hs;
  int n;
};

// Pages of a cache: element (page, head, token in page, d) at
// page * ps + head * hs + token * ts + d.
struct Pages {
  void *p;
  int64_t ps, hs, ts;
};
struct CacheView {
  Pages k, v;
  int64_t pages;
  int page_size, heads, D;
};
struct BatchView {
  const int32_t *starts, *lengths, *table;
  int64_t table_stride;
  int n, table_pages;
};

struct RopeTableArgs {
  int pairs;
  int64_t first, n;
  double magnitude;
  const double *frequencies;  // HOST
  float *cos, *sin;
  bool pdl;
};
cudaError_t launch_rope_table(const RopeTableArgs &a, cudaStream_t stream);

struct RopeArgs {
  bool f32, append, pdl;
  int64_t T;
  int D;
  Heads q, k, v;    // n = 0: none
  Heads qo, ko;     // ko: not with append
  const float *gq, *gk;
  float eps;
  const float *cos, *sin;  // null: no rotation
  int64_t positions;
  int rot, interleaved;
  const int32_t *pos;  // not with append
  CacheView c;
  BatchView b;
};
cudaError_t launch_rope(const RopeArgs &a, cudaStream_t stream);

struct AttnArgs {
  bool f32, pdl;
  int64_t T;
  Heads q, o;
  CacheView c;
  BatchView b;
  float scale;
  int64_t window;  // 0: none
  unsigned char *ws;
};
size_t attn_workspace_bytes(const AttnArgs &a);
cudaError_t launch_attn(const AttnArgs &a, cudaStream_t stream);

// Division of 0 <= x < 2^31 by a number known at the launch: a product and a
// shift, where the compiler's division takes some 40 instructions.
struct FastDiv {
  uint32_t mul, shift, d;
  FastDiv() = default;
  explicit FastDiv(uint32_t by) : d(by) {
    shift = 0;
    while ((uint64_t(1) << shift) < by) ++shift;  // 2^(shift - 1) < by <= 2^shift
    // ceil(2^(31 + shift) / by) fits 32 bits, and its excess over the quotient,
    // below 1, adds less than x / 2^(31 + shift) < 1 / by to x / by.
    mul = static_cast<uint32_t>(((uint64_t(1) << (31 + shift)) + by - 1) / by);
  }
  __device__ __forceinline__ int div(int x) const {
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(x)) * mul) >>
                            (31 + shift));
  }
};

// `total` blocks of a line shared out over `parts` CTAs: the first total %
// parts of them take one more.
struct Share {
  int64_t q;
  int r;
  __device__ __forceinline__ Share(int64_t total, int parts) {
    if (total < (int64_t(1) << 31)) {  // (64-bit divisions take a microsecond)
      const uint32_t n = static_cast<uint32_t>(total), d = static_cast<uint32_t>(parts);
      q = n / d;
      r = static_cast<int>(n - static_cast<uint32_t>(q) * d);
    } else {
      q = total / parts;
      r = static_cast<int>(total - q * parts);
    }
  }
  __device__ __forceinline__ int64_t first(int c) const { return c * q + min(c, r); }
  // The CTA that has block x.
  __device__ __forceinline__ int owner(int64_t x) const {
    const int64_t head = r * (q + 1);
    return static_cast<int>(x < head ? div(x, q + 1) : r + div(x - head, q));
  }
  static __device__ __forceinline__ int64_t div(int64_t a, int64_t b) {
    if ((a | b) < (int64_t(1) << 31))
      return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
  }
};

// One sequence of a batch as the attention kernels take it: rows t0 .. t0 + n
// of the queries, whose row i stands at position len - n + i; keys from lo on
// (a multiple of 16) are attended by some row, of those that the table holds.
struct Seq {
  int t0, n, len, lo;
};
constexpr int kMaxPositions = 2147483647 - 1024;  // block ends stay within an int
// A window as the kernels take it (0: none): none reaches further than positions.
inline int window_of(int64_t window) {
  return window < kMaxPositions ? static_cast<int>(window) : 0;
}
// The first key, rounded down to a multiple of 16, that some of the rows attends.
__device__ __forceinline__ int first_key(int n, int len, int window) {
  if (window == 0) return 0;
  return static_cast<int>(max(int64_t(0), int64_t(len) - n + 1 - window)) & ~15;
}
// What the device arrays say, brought within the buffers whatever they hold.
__device__ __forceinline__ Seq load_seq(const BatchView &b, int i, int T, int window) {
  Seq s;
  const int a = b.starts[i], z = b.starts[i + 1];
  // The length up to the last row that is here: those past the call's T rows are
  // not, and the ones before them keep their positions.
  const int64_t len = b.lengths[i] - max(int64_t(z) - T, int64_t(0));
  s.t0 = min(max(a, 0), T);
  s.n = max(min(z, T) - s.t0, 0);
  s.len = static_cast<int>(min(max(len, int64_t(0)), int64_t(kMaxPositions)));
  s.lo = first_key(s.n, s.len, window);
  return s;
}

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int block, size_t smem, bool pdl,
                         cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace mnb
