// ar_tree_bf16.cu -- attention of drafted tokens with __nv_bfloat16 queries (one translation unit per query type so that
// they compile in parallel).
#include "ar_tree_mma.cuh"

namespace ar {

template cudaError_t launch_tree<__nv_bfloat16, __nv_bfloat16>(const TreeArgs&, const TreeMaps&, const TreeShape&, int, int, cudaStream_t);
template cudaError_t launch_tree<__nv_bfloat16, __nv_fp8_e4m3>(const TreeArgs&, const TreeMaps&, const TreeShape&, int, int, cudaStream_t);
template cudaError_t take_tree_wait_timeouts<__nv_bfloat16>(unsigned int*);

}  // namespace ar
