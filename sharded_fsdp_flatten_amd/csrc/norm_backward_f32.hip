// norm_backward_f32.hip -- the norms' backward pass over rows in registers: f32 activations, cached
// loads.
#include "norm_backward.h"

namespace fsdp {
void launch_norm_bwd_rows_f32(const NormBwd& a, float* partial, uint32_t blocks, hipStream_t stream) {
    norm_bwd_rows<float, false>(a, partial, blocks, stream);
}
}  // namespace fsdp
