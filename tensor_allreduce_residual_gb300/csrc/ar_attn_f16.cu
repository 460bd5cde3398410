// ar_attn_f16.cu -- paged attention with __half queries (one translation unit per
// query type so that they compile in parallel).
#include "ar_attn.cuh"

namespace ar {

template cudaError_t launch_attention<__half, __half>(const AttnArgs&, int, int, cudaStream_t);
template cudaError_t launch_attention<__half, __nv_fp8_e4m3>(const AttnArgs&, int, int, cudaStream_t);

}  // namespace ar
