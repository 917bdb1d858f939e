// norm_backward_f32_nt.hip -- the norms' backward pass over rows in registers: f32 activations, non-temporal
// loads.
#include "norm_backward.h"

namespace fsdp {
void launch_norm_bwd_rows_f32_nt(const NormBwd& a, float* partial, uint32_t blocks, hipStream_t stream) {
    norm_bwd_rows<float, true>(a, partial, blocks, stream);
}
}  // namespace fsdp
