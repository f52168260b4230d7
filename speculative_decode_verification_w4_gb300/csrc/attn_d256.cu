// attn_d256.cu -- the attention kernels of head size 256 (see attn.cuh, attn_tc.cuh).
#include "attn.cuh"

namespace vw4 {
cudaError_t launch_attn_d256(const AttnParams& p, const AttnMaps& maps, bool f8, int rows, int* grid,
                            int sms, cudaStream_t s) {
    return attn_dispatch<256>(p, maps, f8, rows, grid, sms, s);
}
}  // namespace vw4
