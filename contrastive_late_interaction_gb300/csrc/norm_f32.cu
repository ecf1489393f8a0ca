// Layer norm and the residual join: fp32 rows.

#include "norm.cuh"

namespace cli {
namespace norm {
template cudaError_t launch_types<float, float>(const NormLaunch &L, cudaStream_t stream);
}
}  // namespace cli
