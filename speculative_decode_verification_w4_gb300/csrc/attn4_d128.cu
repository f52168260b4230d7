// attn4_d128.cu -- the 4-bit cache's attention kernels of head size 128 (see attn4.cuh).
#include "attn4.cuh"

namespace vw4 {
cudaError_t launch_attn4_d128(const AttnParams& p, const Kv4Blocks& kb, const AttnMaps& maps, int nt,
                            bool large, int* grid, int sms, cudaStream_t s) {
    return attn4_dispatch<128>(p, kb, maps, nt, large, grid, sms, s);
}
}  // namespace vw4
