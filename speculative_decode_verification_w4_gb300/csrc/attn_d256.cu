// attn_d256.cu -- the attention kernels of head size 256 (see attn.cuh).
#include "attn.cuh"

namespace vw4 {
cudaError_t launch_attn_d256(const AttnParams& p, bool f8, int rows, int* grid, int sms,
                            cudaStream_t s) {
    return attn_dispatch<256>(p, f8, rows, grid, sms, s);
}
}  // namespace vw4
