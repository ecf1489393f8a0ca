// Layer norm and the residual join: fp16 rows.

#include "norm.cuh"

namespace cli {
namespace norm {
template cudaError_t launch_types<__half, __half>(const NormLaunch &L, cudaStream_t stream);
}
}  // namespace cli
