// ar_tree_f16.cu -- attention of drafted tokens with __half queries (one translation unit per query type so that
// they compile in parallel).
#include "ar_tree_mma.cuh"

namespace ar {

template cudaError_t launch_tree<__half, __half>(const TreeArgs&, const TreeMaps&, const TreeShape&, int, int, cudaStream_t);
template cudaError_t launch_tree<__half, __nv_fp8_e4m3>(const TreeArgs&, const TreeMaps&, const TreeShape&, int, int, cudaStream_t);
template cudaError_t take_tree_wait_timeouts<__half>(unsigned int*);

}  // namespace ar
