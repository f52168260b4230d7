// attn4_d64.cu -- the 4-bit cache's attention kernels of head size 64 (see attn4.cuh).
#include "attn4.cuh"

namespace vw4 {
cudaError_t launch_attn4_d64(const AttnParams& p, const Kv4Blocks& kb, const AttnMaps& maps, int nt,
                            bool large, int* grid, int sms, cudaStream_t s) {
    return attn4_dispatch<64>(p, kb, maps, nt, large, grid, sms, s);
}
}  // namespace vw4
