// norm_backward_bf16.hip -- the norms' backward pass over rows in registers: bf16 activations, cached
// loads.
#include "norm_backward.h"

namespace fsdp {
void launch_norm_bwd_rows_bf16(const NormBwd& a, float* partial, uint32_t blocks, hipStream_t stream) {
    norm_bwd_rows<uint16_t, false>(a, partial, blocks, stream);
}
}  // namespace fsdp
