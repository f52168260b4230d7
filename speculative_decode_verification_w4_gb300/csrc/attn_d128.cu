// attn_d128.cu -- the attention kernels of head size 128 (see attn.cuh, attn_tc.cuh).
#include "attn.cuh"

namespace vw4 {
cudaError_t launch_attn_d128(const AttnParams& p, const AttnMaps& maps, bool f8, int rows, int* grid,
                            int sms, cudaStream_t s) {
    return attn_dispatch<128>(p, maps, f8, rows, grid, sms, s);
}
}  // namespace vw4
