// Attention over a paged cache: the choice of the kernel.
#include "attn.h"
#include "attn_stream.h"

namespace mnb {

size_t attn_workspace_bytes(const AttnArgs &a) { return stream_workspace_bytes(a.f32, a.c.D); }

cudaError_t launch_attn(const AttnArgs &a, cudaStream_t stream) {
  return launch_attn_stream(a, stream);
}

}  // namespace mnb
