// The wide kernel (mm_fp8.cuh) of products that end in a bias, a scale and a
// residual, with no activation, relu, relu squared or SwiGLU.
#include "mm_fp8.cuh"

namespace bq {
namespace fp8mm {

cudaError_t launch_wide_simple_end(const CUtensorMap& map_w, const CUtensorMap& map_x, const EndArgs& a, int64_t items,
                                   bool swiglu, cudaStream_t st) {
    if (swiglu)
        return a.residual ? launch_wide<true, END_SIMPLE, true>(map_w, map_x, a, items, st)
                          : launch_wide<true, END_SIMPLE, false>(map_w, map_x, a, items, st);
    return a.residual ? launch_wide<false, END_SIMPLE, true>(map_w, map_x, a, items, st)
                      : launch_wide<false, END_SIMPLE, false>(map_w, map_x, a, items, st);
}

}  // namespace fp8mm
}  // namespace bq
