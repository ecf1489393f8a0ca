// Layer norm and the residual join: the call's types.

#include "norm.cuh"

namespace cli {
namespace norm {
extern template cudaError_t launch_types<__nv_bfloat16, __nv_bfloat16>(const NormLaunch &L, cudaStream_t stream);
extern template cudaError_t launch_types<__nv_bfloat16, float>(const NormLaunch &L, cudaStream_t stream);
extern template cudaError_t launch_types<__half, __half>(const NormLaunch &L, cudaStream_t stream);
extern template cudaError_t launch_types<__half, float>(const NormLaunch &L, cudaStream_t stream);
extern template cudaError_t launch_types<float, float>(const NormLaunch &L, cudaStream_t stream);
}  // namespace norm

cudaError_t launch_norm(const NormLaunch &L, cudaStream_t stream) {
    using namespace norm;
    const bool mixed = L.stream_dtype != L.dtype;   // an fp32 stream, then
    if (L.dtype == CLI_BF16)
        return mixed ? launch_types<__nv_bfloat16, float>(L, stream) : launch_types<__nv_bfloat16, __nv_bfloat16>(L, stream);
    if (L.dtype == CLI_F16) return mixed ? launch_types<__half, float>(L, stream) : launch_types<__half, __half>(L, stream);
    return launch_types<float, float>(L, stream);
}

}  // namespace cli
