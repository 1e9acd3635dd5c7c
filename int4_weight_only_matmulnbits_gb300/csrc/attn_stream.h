// Parameters of the attention kernel that streams keys past a few query rows.
#pragma once

#include "attn.h"

namespace mnb {

struct AttnStreamParams {
  Heads q, o;
  Pages k, v;
  BatchView b;
  int pages, kv_heads;
  FastDiv page_size, G;               // G: query heads per key head
  int T, cap;                         // cap: tokens that a row of the table holds
  int window;                         // 0: none
  int span;                           // blocks of keys that the rows of a unit reach in a window
  float scale;                        // |scale| of the scores, times log2(e)
  int negative;                       // the scale is: scores change their sign
  int cluster;                        // blocks of a cluster (one unit each), where they are used
  int *headers;                       // of the pieces that end a block's part
  float *parts;                       // two pieces per block: sums, maxima, sums of weights
};

size_t stream_workspace_bytes(int D);
cudaError_t launch_attn_stream(const AttnArgs &a, cudaStream_t stream);

}  // namespace mnb
