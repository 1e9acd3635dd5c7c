// Launch interface of the expert layer's tensor-core kernel (moe_tile.cu),
// for many slots per expert with bf16 activations.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "moe_stream.h"

namespace mnb {

constexpr int kTileSlots = 192;  // slots per group (columns of an accumulator)
constexpr int kTileBox = 32;     // activation rows per TMA box

// What the kernel needs of a stack's scales and biases.
struct TileScales {
  const float *fac;   // [E * N16 * 16] power of two per row (moe.cu, row_scales_kernel)
  const float *smax;  // [E] largest |scale| (down)
  const float *bmax;  // [E] largest |bias|, or null (down)
};

struct TileParams {
  CUtensorMap tmb;  // activation rows: {64 K64, rows} fp16, box {64, 32}, 128-byte swizzle
  int mode;
  StreamMat w[2];
  TileScales ts[2];
  int N, N16, K64, nb, nbz;
  int ntile;  // column tiles of an expert: 64 columns (gate and up) or 128
  // Lists: slots by expert; places count along the order.
  const int32_t *order, *n_groups;
  const SlotGroup *groups;
  const float *weights;  // [P] by slot (gate and up, down)
  // By place: what undoes the activation row's scale, and that scale's
  // exponent (down).
  const float *unscale;
  const int32_t *shift;
  // Outputs: Y [P, N] bf16 by slot (product); hidden rows [P, ldh] in fp32, by
  // place (gate and up); fp16 partials [P, ldp] and their undo factors, by place
  // (down). ldp is even.
  uint16_t *Y, *part;
  float *hidden;
  int64_t ldh, ldp;
  int y_pairs;  // rows of Y start on 4 bytes
  float *out_unscale;
};

cudaError_t launch_tile(const TileParams &p, bool zp, bool sf32, int bs, bool pdl,
                        cudaStream_t stream);

}  // namespace mnb
