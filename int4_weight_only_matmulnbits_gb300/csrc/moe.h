// Host-side launch interfaces of the mixture-of-experts kernels. Arguments
// arrive here already validated by the C ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace mnb {

// Limits of the router: an expert list and one warp's keys stay in shared
// memory, one lane keeps each choice.
constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxTopK = 32;

struct RouteArgs {
  const void *logits;  // [M, E]
  bool logits_f32;
  int64_t M;
  int E, top_k;
  bool normalize;
  float *weights;    // [M, top_k]
  int32_t *experts;  // [M, top_k]
  int32_t *offsets;  // [E + 1] or null
  int32_t *order;    // [M * top_k] or null
  unsigned char *ws;  // moe_route_workspace_bytes() when order is given
  bool pdl;
};
size_t moe_route_workspace_bytes(int64_t M, int E, int top_k);
cudaError_t launch_moe_route(const RouteArgs &a, cudaStream_t stream);

// A stack of E weights N x K, packed with each expert's rows padded to whole
// 16-row tiles (N16 tiles per expert).
struct ExpertStack {
  const void *b, *s, *z;  // z may be null (every zero point is 8)
  const float *rows;      // [E * 16 N16] row factors, then [E] largest |scale|
  const float *bias;      // [E, N] or null
  int E, N, K, bs;
  bool s_f32;
};

struct ExpertPackArgs {
  const uint8_t *B;
  const void *scales;
  const uint8_t *zp;  // may be null
  int64_t E, N, K;
  int bs;
  bool scale_f32;
  void *packed_b, *packed_scales, *packed_zp;
  float *packed_rows;
};
// Re-layout of a stack; the header is written by the caller's last kernel.
cudaError_t launch_prepack_experts(const ExpertPackArgs &a, cudaStream_t stream);

struct ExpertsArgs {
  const void *A;  // [M, K] or [M, top_k, K]
  bool a_f32, per_slot;
  ExpertStack w;
  const int32_t *experts;  // [M, top_k]
  int64_t M;
  int top_k;
  void *Y;  // [M, top_k, N] in A's dtype
  unsigned char *ws;
  bool pdl;
};
// Host arithmetic on the sizes and types alone (pointers are not looked at).
size_t matmul_experts_workspace_bytes(const ExpertsArgs &a);
cudaError_t launch_matmul_experts(const ExpertsArgs &a, cudaStream_t stream);

struct MoeArgs {
  const void *X;  // [M, H]
  bool a_f32;
  const void *logits;  // [M, E]
  bool logits_f32;
  int64_t M;
  int top_k;
  bool normalize;
  ExpertStack gate, up, down;
  void *Y;  // [M, H]
  unsigned char *ws;
  bool pdl;
};
size_t moe_workspace_bytes(const MoeArgs &a);
cudaError_t launch_moe(const MoeArgs &a, cudaStream_t stream);

// Reads and clears the fault word of the tensor-core kernel.
cudaError_t moe_take_fault(unsigned int *out);

}  // namespace mnb
