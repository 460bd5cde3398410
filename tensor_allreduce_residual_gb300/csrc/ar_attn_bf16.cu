// ar_attn_bf16.cu -- paged attention with __nv_bfloat16 queries (one translation unit per
// query type so that they compile in parallel).
#include "ar_attn.cuh"

namespace ar {

template cudaError_t launch_attention<__nv_bfloat16, __nv_bfloat16>(const AttnArgs&, int, int, cudaStream_t);
template cudaError_t launch_attention<__nv_bfloat16, __nv_fp8_e4m3>(const AttnArgs&, int, int, cudaStream_t);

}  // namespace ar
