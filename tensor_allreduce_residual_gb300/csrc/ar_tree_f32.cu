// ar_tree_f32.cu -- attention of drafted tokens with fp32 queries (one translation unit per query type so that they
// compile in parallel).
#include "ar_tree.cuh"

namespace ar {

template <>
cudaError_t launch_tree<float, float>(const TreeArgs& a, const TreeMaps&, const TreeShape& shape, int most, int sms, cudaStream_t s)
{
    return a.head_dim <= 64    ? launch_tree_fma<64>(a, shape, most, sms, s)
           : a.head_dim <= 128 ? launch_tree_fma<128>(a, shape, most, sms, s)
                               : launch_tree_fma<256>(a, shape, most, sms, s);
}

}  // namespace ar
