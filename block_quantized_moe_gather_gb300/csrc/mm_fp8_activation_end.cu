// The wide kernel (mm_fp8.cuh) of products that end in silu, gelu or its tanh form.
// One kernel of all three takes those that have a residual too (a block's last
// projection has no activation): its tiles take 1.6 us longer.
#include "mm_fp8.cuh"

namespace bq {
namespace fp8mm {

cudaError_t launch_wide_activation_end(const CUtensorMap& map_w, const CUtensorMap& map_x, const EndArgs& a, int64_t items,
                                       cudaStream_t st) {
    if (a.residual) return launch_wide<false, END_ANY, true>(map_w, map_x, a, items, st);
    switch (a.act) {
        case BQ_ACT_SILU: return launch_wide<false, END_SILU, false>(map_w, map_x, a, items, st);
        case BQ_ACT_GELU: return launch_wide<false, END_GELU, false>(map_w, map_x, a, items, st);
        default: return launch_wide<false, END_GELU_TANH, false>(map_w, map_x, a, items, st);
    }
}

}  // namespace fp8mm
}  // namespace bq
