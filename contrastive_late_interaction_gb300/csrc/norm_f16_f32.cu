// Layer norm and the residual join: fp16 rows beside an fp32 stream.

#include "norm.cuh"

namespace cli {
namespace norm {
template cudaError_t launch_types<__half, float>(const NormLaunch &L, cudaStream_t stream);
}
}  // namespace cli
