// ar_attn_f32.cu -- paged attention with float queries (one translation unit per
// query type so that they compile in parallel).
#include "ar_attn.cuh"

namespace ar {

template cudaError_t launch_attention<float, float>(const AttnArgs&, int, int, cudaStream_t);

}  // namespace ar
