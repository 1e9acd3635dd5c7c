// The expert layer's weight-streaming kernel for scale blocks of 16 codes
// (1 k step of 16 per applied scale).
#include "moe_stream.cuh"

namespace mnb {
template cudaError_t launch_stream<1>(const StreamParams &, bool, bool, int, int, int, bool,
                                       cudaStream_t);
}
