// attn4_tc.cu -- the 4-bit cache's attention kernels of many query rows (see attn4_tc.cuh).
#include "attn4_tc.cuh"

namespace vw4 {
cudaError_t launch_attn4_tc(const AttnParams& p, const Kv4Blocks& kb, const AttnMaps& maps, int D, int rows,
                            int* grid, int sms, cudaStream_t s) {
    switch (rows) {
        case 64:
            return D == 64    ? attn4_tc_launch<64, 64>(p, kb, maps, grid, sms, s)
                   : D == 128 ? attn4_tc_launch<128, 64>(p, kb, maps, grid, sms, s)
                              : attn4_tc_launch<256, 64>(p, kb, maps, grid, sms, s);
        case 128:
            return D == 64    ? attn4_tc_launch<64, 128>(p, kb, maps, grid, sms, s)
                   : D == 128 ? attn4_tc_launch<128, 128>(p, kb, maps, grid, sms, s)
                              : attn4_tc_launch<256, 128>(p, kb, maps, grid, sms, s);
    }
    return cudaErrorInvalidValue;
}
}  // namespace vw4
