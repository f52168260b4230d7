// attn4.cu -- attention over the 4-bit cache: choice of the kernel and workspace.
#include "attn4_tc.cuh"

namespace vw4 {

// The 5th-generation tensor cores take their time from the softmax's latency, not from the
// rows: from 33 rows on they are ahead at every head size and length, up to 32 behind or
// even (16 / 32 / 40 / 64 rows, us, mma.sync against tcgen05: 32 sequences of up to 32768
// tokens, 4 key heads of size 128 75 / 106 / 177 / 262 against 109 / 112 / 112 / 117; of size
// 256 135 / 198 / 280 / 426 against 176 / 181 / 182 / 192; 64 windows of 1024, head size 128,
// 24 / 32 / 64 rows 37 / 44 / 87 against 53 / 54 / 57).
constexpr int kAttn4TcFrom = 33;

constexpr int kAttn4Sms = 152;  // (of this GPU)
constexpr int kAttn4MaxGrid = kAttnMaxGrid64;  // (three blocks an SM at most)
static size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

// Query rows of a block; key heads with more are cut into blocks, each reading the keys again
// (from L2: the blocks of a key head are neighbours in the schedule).
struct Attn4Rows {
    bool tc;
    int rows, grid;  // rows of a partial, most CTAs
};
static Attn4Rows attn4_rows(int rows) {
    if (rows >= kAttn4TcFrom) return {true, rows > 64 ? 128 : 64, kAttn4TcGrid};
    return {false, (rows + 7) / 8 * 8, kAttn4MaxGrid};
}

size_t attn4_workspace_bytes(int B, int rows, int D) {
    // (the rows of a block are fewer where a key head's are cut)
    size_t most = 0;
    for (int r = 1; r <= (rows < 128 ? rows : 128); ++r) {
        const Attn4Rows k = attn4_rows(r);
        const size_t n = static_cast<size_t>(k.rows) * k.grid;
        most = n > most ? n : most;
    }
    return align256((static_cast<size_t>(B) + 1) * sizeof(long long)) +
           align256(2u * most * (D + 2) * sizeof(float));
}

Attn4Plan attn4_plan(AttnParams& p, int D, void* ws) {
    Attn4Plan plan;
    // blocks of gb heads by tb verify indexes, as even as they get
    constexpr int max_rows = 128;
    const int g_blocks = (p.G + max_rows - 1) / max_rows;
    p.gb = (p.G + g_blocks - 1) / g_blocks;
    const int most = max_rows / p.gb;
    const int t_blocks = (p.R + most - 1) / most;
    p.tb = (p.R + t_blocks - 1) / t_blocks;
    p.blocks_g = (p.G + p.gb - 1) / p.gb;
    p.row_blocks = p.blocks_g * ((p.R + p.tb - 1) / p.tb);
    p.groups = p.Hkv * p.row_blocks;
    const Attn4Rows k = attn4_rows(p.gb * p.tb);
    plan.tc = k.tc;
    plan.rows = k.rows;
    p.base = static_cast<long long*>(ws);
    p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                         align256((static_cast<size_t>(p.B) + 1) * sizeof(long long)));
    // at most one CTA per tile that the table could hold
    const long long cap = static_cast<long long>(p.max_blocks) * p.page_size;
    const auto units = [&](int tk) {
        return static_cast<long long>(p.B) * p.groups * ((cap + tk - 1) / tk);
    };
    const int nt = k.rows / 8;
    plan.large = !k.tc && (nt == 1 ? units(attn4_tk(D, true)) >= kAttn4Sms : D == 64 && nt == 2);
    plan.tk = k.tc ? attn4_tc_tk(D) : attn4_tk(D, plan.large);
    plan.grid = k.grid;
    const long long most_units = units(plan.tk);
    if (most_units < plan.grid) plan.grid = static_cast<int>(most_units < 1 ? 1 : most_units);
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
    const cudaError_t e = plan.tc   ? launch_attn4_tc(p, kb, maps, D, plan.rows, &grid, sms, s)
                          : D == 64  ? launch_attn4_d64(p, kb, maps, plan.rows / 8, plan.large, &grid, sms, s)
                          : D == 128 ? launch_attn4_d128(p, kb, maps, plan.rows / 8, plan.large, &grid, sms, s)
                                     : launch_attn4_d256(p, kb, maps, plan.rows / 8, plan.large, &grid, sms, s);
    if (e != cudaSuccess) return e;
    return launch_attn_join(p, D, plan.rows, grid, plan.tk, sms, s);
}

}  // namespace vw4
