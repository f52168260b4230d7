// attn4.cu -- attention over the 4-bit cache: choice of the kernel and workspace.
#include "attn4.cuh"

namespace vw4 {

// Query rows of a block in n-tiles of 8; key heads with more than 64 rows are cut into
// blocks, each reading the keys again (from L2: the blocks of a key head are neighbours in
// the schedule).
constexpr int kAttn4MaxRows = 64;
static int attn4_tiles(int rows) {
    const int n = (rows + 7) / 8;
    return n <= 4 ? n : (n <= 6 ? 6 : 8);
}
constexpr int kAttn4MaxGrid = kAttnMaxGrid64;  // (three blocks an SM at most)
static size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

size_t attn4_workspace_bytes(int B, int rows, int D) {
    const size_t r = 8 * static_cast<size_t>(attn4_tiles(rows < kAttn4MaxRows ? rows : kAttn4MaxRows));
    return align256((static_cast<size_t>(B) + 1) * sizeof(long long)) +
           align256(2u * static_cast<size_t>(kAttn4MaxGrid) * r * (D + 2) * sizeof(float));
}

Attn4Plan attn4_plan(AttnParams& p, int D, void* ws) {
    Attn4Plan plan;
    // blocks of gb heads by tb verify indexes, as even as they get
    const int g_blocks = (p.G + kAttn4MaxRows - 1) / kAttn4MaxRows;
    p.gb = (p.G + g_blocks - 1) / g_blocks;
    const int most = kAttn4MaxRows / p.gb;
    const int t_blocks = (p.R + most - 1) / most;
    p.tb = (p.R + t_blocks - 1) / t_blocks;
    p.blocks_g = (p.G + p.gb - 1) / p.gb;
    p.row_blocks = p.blocks_g * ((p.R + p.tb - 1) / p.tb);
    p.groups = p.Hkv * p.row_blocks;
    plan.nt = attn4_tiles(p.gb * p.tb);
    p.base = static_cast<long long*>(ws);
    p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                         align256((static_cast<size_t>(p.B) + 1) * sizeof(long long)));
    // at most one CTA per tile that the table could hold
    const long long cap = static_cast<long long>(p.max_blocks) * p.page_size;
    plan.tk = attn4_tk(D, plan.nt);
    const long long units = static_cast<long long>(p.B) * p.groups * ((cap + plan.tk - 1) / plan.tk);
    plan.grid = kAttn4MaxGrid;
    if (units < plan.grid) plan.grid = static_cast<int>(units < 1 ? 1 : units);
    p.box_rows = p.page_size < plan.tk ? p.page_size : plan.tk;
    plan.box_bytes = D / 2;
    const long long group = 8 * p.token_stride;
    if (p.head_stride == D / 2 || p.Hkv == 1) {
        p.fold = kFoldBlocks;
    } else if (p.head_stride % group == 0) {
        p.fold = kFoldGroups;
        p.fold_step = static_cast<int>(p.head_stride / group);
    } else {
        p.fold = kFoldNone;
    }
    plan.swizzle = D == 64    ? CU_TENSOR_MAP_SWIZZLE_32B
                   : D == 128 ? CU_TENSOR_MAP_SWIZZLE_64B
                              : CU_TENSOR_MAP_SWIZZLE_128B;
    return plan;
}

cudaError_t launch_attn4(const AttnParams& p, const Kv4Blocks& kb, const AttnMaps& maps,
                         const Attn4Plan& plan, int D, int sms, cudaStream_t s) {
    int grid = plan.grid;
    const cudaError_t e = D == 64    ? launch_attn4_d64(p, kb, maps, plan.nt, &grid, sms, s)
                          : D == 128 ? launch_attn4_d128(p, kb, maps, plan.nt, &grid, sms, s)
                                     : launch_attn4_d256(p, kb, maps, plan.nt, &grid, sms, s);
    if (e != cudaSuccess) return e;
    return launch_attn_join(p, D, 8 * plan.nt, grid, plan.tk, sms, s);
}

}  // namespace vw4
