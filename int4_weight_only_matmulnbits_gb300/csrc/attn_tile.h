// Parameters of the tensor-core (tcgen05) attention kernel.
#pragma once

#include <cuda.h>

#include "attn.h"

namespace mnb {

struct AttnTileParams {
  CUtensorMap tk, tv;  // pages: 64 columns of `box` tokens
  CUtensorMap tq;      // rows of q: 64 columns of 128 rows (q_tma)
  Heads q, o;
  BatchView b;
  int pages, page_size, box, kv_heads, G;
  int T, cap, window;
  float scale;    // |scale| times log2(e)
  int negative, q_tma;
  int64_t *line;  // [0]: blocks of a key head, [1]: units
  int64_t *first; // [units + 1]: first block of each unit, within a key head
  int4 *units;    // [2 units]: t0, n, len, tile; first block of keys, blocks, sequence
  int64_t most;   // units that there is room for
  int *headers;
  float *parts;
};

bool tile_path(const AttnArgs &a);
size_t tile_workspace_bytes(const AttnArgs &a);
cudaError_t launch_attn_tile(const AttnArgs &a, cudaStream_t stream);
cudaError_t attn_take_fault(unsigned int *out);

}  // namespace mnb
