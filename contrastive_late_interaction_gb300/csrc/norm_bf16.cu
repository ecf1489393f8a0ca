// Layer norm and the residual join: bf16 rows.

#include "norm.cuh"

namespace cli {
namespace norm {
template cudaError_t launch_types<__nv_bfloat16, __nv_bfloat16>(const NormLaunch &L, cudaStream_t stream);
}
}  // namespace cli
