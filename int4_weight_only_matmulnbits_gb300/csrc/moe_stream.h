// Launch interface of the weight-streaming kernel of the expert layer
// (moe_stream.cuh), compiled per number of k steps a scale block spans.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace mnb {

// A run of slots that share an expert: their places in the order of slots.
struct SlotGroup {
  int e, first, cols;
};

enum StreamMode { kStreamProduct = 0, kStreamGateUp = 1, kStreamDown = 2 };

constexpr int kStreamStages = 3;  // ring stages per warp
constexpr int kStreamChunks = 2;  // chunks per stage and tile
constexpr int kStreamCtas = 3;    // CTAs per SM the registers allow

struct StreamMat {
  const uint4 *b;
  const unsigned char *s, *z;
  const float *bias;
};

struct StreamParams {
  int mode;
  StreamMat w[2];  // gate and up, or one matrix twice
  int E, N, N16, K, K64, nb, nbz, bs_log2;
  // Activations, fp32 or bf16: row p / top_k of A for slot p, or row p when
  // per_slot; rows ld elements apart.
  const void *A;
  int a_f32, a_vec;  // a_vec: rows are 16-byte aligned
  int per_slot;
  int64_t ld;
  int P, top_k;
  const uint32_t *tops;  // bits of the largest magnitude of each row
  // Lists.
  const int32_t *offsets, *order, *n_groups;
  const SlotGroup *groups;
  const float *weights;  // [P] (gate and up, down)
  // Outputs: Y [P, N] (product), hidden rows [P, ldh] (gate and up), partials
  // [P, N] (down).
  void *Y;
  int y_f32;
  float *hidden;
  uint32_t *hidden_tops;  // [P], zeros before
  int64_t ldh;
  float *part;
  // Geometry.
  int gt_log2;          // slots per group: 2^gt_log2 <= 8
  int npair;            // tile pairs of an expert
  int ksplit, tpu, tpu_log2, ns;  // warps per pair, pairs per step, steps per group
  int st_tile, st_bytes, st_scale, st_zp;  // stage layout
  int krow;             // staged activation row, in elements
  int off_x, off_sums, off_red, off_ring;
  int early;  // down: weights load ahead of the dependency wait
};

template <int SPB>
cudaError_t launch_stream(const StreamParams &p, bool zp, bool sf32, int terms, int grid,
                          int smem, bool pdl, cudaStream_t stream);

}  // namespace mnb
