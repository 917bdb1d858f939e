// norm_backward_bf16_nt.hip -- the norms' backward pass over rows in registers: bf16 activations, non-temporal
// loads.
#include "norm_backward.h"

namespace fsdp {
void launch_norm_bwd_rows_bf16_nt(const NormBwd& a, float* partial, uint32_t blocks, hipStream_t stream) {
    norm_bwd_rows<uint16_t, true>(a, partial, blocks, stream);
}
}  // namespace fsdp
