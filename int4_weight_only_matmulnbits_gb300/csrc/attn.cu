// Attention over a paged cache: the choice of the kernel.
#include "attn.h"
#include "attn_stream.h"
#include "attn_tile.h"

namespace mnb {

size_t attn_workspace_bytes(const AttnArgs &a) {
  return tile_path(a) ? tile_workspace_bytes(a) : stream_workspace_bytes(a.c.D);
}

cudaError_t launch_attn(const AttnArgs &a, cudaStream_t stream) {
  return tile_path(a) ? launch_attn_tile(a, stream) : launch_attn_stream(a, stream);
}

}  // namespace mnb
