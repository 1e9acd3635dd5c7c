// The expert layer's weight-streaming kernel for scale blocks of 32 codes
// (2 k steps of 16 per applied scale).
#include "moe_stream.cuh"

namespace mnb {
template cudaError_t launch_stream<2>(const StreamParams &, bool, bool, int, int, int, bool,
                                       cudaStream_t);
}
