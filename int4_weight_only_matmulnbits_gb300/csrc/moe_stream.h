// Launch interface of the weight-streaming kernel of the expert layer
// (moe_stream.cuh), compiled per number of k steps a scale block spans.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace mnb {

enum StreamMode { kStreamProduct = 0, kStreamGateUp = 1, kStreamDown = 2 };

// Slots the kernel lists for itself in shared memory (every CTA builds the
// lists); longer inputs come with lists in global memory.
constexpr int kFewSlots = 256;

struct StreamMat {
  const uint4 *b;
  const unsigned char *s, *z;
  const float *bias;
};

struct StreamParams {
  int mode;
  StreamMat w[2];  // gate and up, or one matrix
  int E, N, N16, K, K64, nb, nbz, bs_log2;
  // Activations: rows of A (row p / top_k, or p when per_slot), or planes of
  // bf16 rows whose sum is the hidden row of slot p (mode down).
  const void *A;
  int a_vec;  // rows of A are 16-byte aligned
  int per_slot;
  int64_t plane;  // elements between planes
  int P, M, top_k;
  // Lists: from logits, from a table of experts, or ready in global memory.
  const void *logits;
  int logits_f32, normalize;
  const int32_t *table;
  const int32_t *offsets, *order;
  const float *weights;  // [P] with the ready lists
  const int32_t *experts;  // [P] with the ready lists (mode down)
  // Outputs: Y [P, N] (product), bf16 planes [P, ldh] (gate and up), fp32
  // partials [P, N] and Y [M, N] (down).
  void *Y;
  int y_f32;
  uint16_t *hidden;
  int ldh, h_planes;
  float *part;
  unsigned *counters;  // [n steps] arrivals per column group; gate and up clears them
  int n_counters;
  // Geometry.
  int gt;               // slots per group (<= 8)
  int ksplit, tpu, ns;  // warps per tile, tiles per step, steps per group
  int kc, st_bytes, st_scale, st_zp;  // chunks per stage; stage layout
  int krow;             // staged activation row, in elements
  int off_lists, off_keys, off_x, off_red, off_ring;
  int early;            // down: the router runs, and weights load, ahead of the dependency wait
};

template <int SPB>
cudaError_t launch_stream(const StreamParams &p, bool zp, bool sf32, int terms, int grid,
                          int smem, bool pdl, cudaStream_t stream);

}  // namespace mnb
