// The expert layer's weight-streaming kernel for scale blocks of 64 codes or more
// (4 k steps of 16 per applied scale).
#include "moe_stream.cuh"

namespace mnb {
template cudaError_t launch_stream<4>(const StreamParams &, bool, bool, int, int, int, bool,
                                       cudaStream_t);
}
