// attn.cu -- attention of the verify rows: choice of the kernel, workspace,
// and the kernel that joins the partial rows of items split over CTAs.
#include "attn.cuh"

namespace vw4 {

// Query rows of a block: the smallest kernel shape that holds a key head's
// rows; more than 128 (64: e4m3 at head size 256, whose f16 ring leaves no room
// for more queries) are cut into blocks, each reading the keys again (from L2: the
// blocks of a key head are neighbours in the schedule).  17 .. 32 rows as two blocks
// of 16 would read and convert every key twice: e4m3, 24 rows of 256 over a window of
// 1024 took 123 us against 57 (64-row blocks), 32 rows of 128 over 4000 .. 8000 tokens
// 183 against 113, in bf16 243 against 135 (500 .. 1000 tokens: 16.8 against 15.7).
static int attn_rows(int rows, int D, bool f8) {
    return rows <= 16 ? 16 : (rows <= 64 || (D == 256 && f8) ? 64 : 128);
}
// keys of a tile of the kernel for blocks of that many rows
static int attn_tile(int rows, bool f8) { return rows == 16 && !f8 ? 64 : 128; }

static int attn_grid_cap(int D) { return D == 256 ? kAttnMaxGrid256 : kAttnMaxGrid64; }

static size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

size_t attn_workspace_bytes(int B, int rows, int D) {
    const size_t base = align256((static_cast<size_t>(B) + 1) * sizeof(long long));
    return base + align256(2u * static_cast<size_t>(attn_grid_cap(D)) * attn_rows(rows, D, false) * (D + 2) *
                           sizeof(float));
}

constexpr int kJoinThreads = 128;

// Joins the partials of split items, in the order of their tiles, and writes
// the rows of sequences without keys.  One block takes `chunk` rows of an
// item, a warp a row (kJoinRows) or 64 columns of one (kJoinColumns); or its warps
// share the parts of 64 columns of a row (kJoinParts).  The lanes weigh up to 32
// partials at once and then own E columns each; the first U partials' values are on
// their way while the weights are computed (the kernel is a chain of load latencies).
// A kernel of its own: the CTAs of an item are any run of the grid, however long, so no
// cluster holds them, and a last arriving CTA would need tickets that the call clears.  Its
// launch adds 2.6 us to 26.3 for 4 sequences of 8 rows, 24 heads of 256.
constexpr int kJoinRows = 0, kJoinColumns = 1, kJoinParts = 2;

template <int D, int MODE>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnParams p, int rows,
                                                                 int grid, int tk, int chunk) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int item = blockIdx.x, b = item / p.groups, g = item - b * p.groups;
    const int h = g / p.row_blocks;
    const long long T = p.base[p.B], base = p.base[b];
    const int nt = attn_seq(p.seq_lens[b], p.max_blocks * p.page_size, p.R, p.window, p.sinks, tk).nt;
    const long long u = base + static_cast<long long>(g) * nt;
    const int G = attn_ctas(T, grid);
    int c0 = 0, c1 = -1;
    if (nt > 0) {
        c0 = attn_owner(T, G, u);
        c1 = attn_owner(T, G, u + nt - 1);
        if (c0 == c1) return;  // written by the attention kernel
    }
    constexpr bool PARTS = MODE == kJoinParts;
    constexpr int E = MODE == kJoinRows ? D / 32 : 2, U = MODE == kJoinRows ? 8 : 16;
    constexpr int WR = D / (32 * E), W = kJoinThreads / 32;  // warps of a row, of the block
    __shared__ float s_m[PARTS ? W : 1], s_l[PARTS ? W : 1];
    __shared__ float2 s_acc[PARTS ? W : 1][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = (PARTS ? blockIdx.y % WR : warp % WR) * 64 + lane * 2;
    const int per = (c1 - c0 + W) / W;  // a warp's parts of kJoinParts
    const int cs = PARTS ? c0 + warp * per : c0, ce = PARTS ? min(c1, cs + per - 1) : c1;
    const float vs = p.v_scale ? __ldg(p.v_scale + h) : 1.f;
    const size_t slot = static_cast<size_t>(rows) * (D + 2);
    auto part = [&](int c) { return p.partial + static_cast<size_t>(c == c0 ? 2 * c + 1 : 2 * c) * slot; };
    const int r0 = PARTS ? blockIdx.y / WR : blockIdx.y * chunk, r1 = min(r0 + chunk, rows);
    for (int r = PARTS ? r0 : r0 + warp / WR; r < r1; r += PARTS ? 1 : W / WR) {
        const AttnRow row = attn_row(p, g, r);
        if (!row.live) continue;
        float M = -INFINITY, L = 0.f, acc[E] = {};
        for (int cb = cs; cb <= ce; cb += 32) {
            const int n = min(32, ce - cb + 1);
            float v[U][E];
            auto fetch = [&](int k0) {
#pragma unroll
                for (int k = 0; k < U; ++k)
                    if (k0 + k < n) {
                        const float* q = part(cb + k0 + k) + r * D + col;
#pragma unroll
                        for (int e = 0; e < E; e += 2) {
                            const float2 t = *reinterpret_cast<const float2*>(q + e * 32);
                            v[k][e] = t.x;
                            v[k][e + 1] = t.y;
                        }
                    }
            };
            fetch(0);
            float m = -INFINITY, l = 0.f;
            if (lane < n) {
                const float* q = part(cb + lane);
                m = q[rows * D + r];
                l = q[rows * (D + 1) + r];
            }
            float mx = m;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
            mx = fmaxf(mx, M);
            const float old = mx == M ? 1.f : ex2(M - mx);  // (M = -infinity: 0)
            M = mx;
            const float w = lane < n ? (M == -INFINITY ? 1.f : ex2(m - M)) : 0.f;
            float sum = l * w;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
            L = L * old + sum;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] *= old;
            for (int k0 = 0; k0 < n; k0 += U) {
                if (k0 > 0) fetch(k0);
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const float wk = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
                    if (k0 + k < n) {
#pragma unroll
                        for (int e = 0; e < E; ++e) acc[e] = fmaf(v[k][e], wk, acc[e]);
                    }
                }
            }
        }
        if constexpr (PARTS) {  // (one row a block)
            if (lane == 0) s_m[warp] = M, s_l[warp] = L;
            s_acc[warp][lane] = make_float2(acc[0], acc[1]);
            __syncthreads();
            if (warp > 0) return;
            float mx = M;
#pragma unroll
            for (int k = 1; k < W; ++k) mx = fmaxf(mx, s_m[k]);
            M = mx;
            L = acc[0] = acc[1] = 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const float w = mx == -INFINITY ? 1.f : ex2(s_m[k] - mx);
                L = fmaf(s_l[k], w, L);
                acc[0] = fmaf(s_acc[k][lane].x, w, acc[0]);
                acc[1] = fmaf(s_acc[k][lane].y, w, acc[1]);
            }
        }
        const float f = L == 0.f ? 0.f : vs / L;
        const long long orow = static_cast<long long>(b) * p.R + row.i;
        __nv_bfloat16* out = p.out + orow * p.ldo + static_cast<long long>(row.hq) * D;
#pragma unroll
        for (int e = 0; e < E; e += 2)
            *reinterpret_cast<uint32_t*>(out + col + e * 32) = pack2<false>(acc[e] * f, acc[e + 1] * f);
        if (col == 0 && p.lse)
            p.lse[orow * p.Hq + row.hq] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
    }
}

template <int D>
static void (*join_of(int mode))(const AttnParams, int, int, int, int) {
    return mode == kJoinParts     ? attn_join_kernel<D, kJoinParts>
           : mode == kJoinColumns ? attn_join_kernel<D, kJoinColumns>
                                  : attn_join_kernel<D, kJoinRows>;
}

AttnPlan attn_plan(AttnParams& p, int D, bool f8, void* ws) {
    AttnPlan plan;
    const int total = p.R * p.G;
    plan.rows = attn_rows(total, D, f8);
    plan.tk = attn_tile(plan.rows, f8);
    p.gb = p.G < plan.rows ? p.G : plan.rows;
    p.tb = plan.rows / p.gb < p.R ? plan.rows / p.gb : p.R;
    p.blocks_g = (p.G + p.gb - 1) / p.gb;
    p.row_blocks = p.blocks_g * ((p.R + p.tb - 1) / p.tb);
    p.groups = p.Hkv * p.row_blocks;
    p.base = static_cast<long long*>(ws);
    p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                         align256((static_cast<size_t>(p.B) + 1) * sizeof(long long)));
    // at most one CTA per tile that the table could hold
    const long long cap = static_cast<long long>(p.max_blocks) * p.page_size;
    const long long units = static_cast<long long>(p.B) * p.groups * ((cap + plan.tk - 1) / plan.tk);
    plan.grid = attn_grid_cap(D);
    if (units < plan.grid) plan.grid = static_cast<int>(units < 1 ? 1 : units);
    // a box lies inside a page and inside a ring piece of the kernel
    const int piece = plan.rows == 16 ? plan.tk
                      : D == 256      ? (f8 ? 32 : 64)
                      : D == 128 && f8 ? 64
                                       : 128;
    p.box_rows = p.page_size < piece ? p.page_size : piece;
    const int key = D * (f8 ? 1 : 2);
    plan.box_bytes = key < 128 ? key : 128;
    plan.v_blocks = key / plan.box_bytes;
    plan.k_blocks = plan.rows > 16 && D == 256 ? plan.v_blocks / 2 : plan.v_blocks;  // of a piece
    const long long group = 8 * p.token_stride;  // elements
    if (p.head_stride == D || p.Hkv == 1) {
        p.fold = kFoldBlocks;
    } else if (p.head_stride % group == 0) {
        p.fold = kFoldGroups;
        p.fold_step = static_cast<int>(p.head_stride / group);
    } else {
        p.fold = kFoldNone;
    }
    plan.swizzle = key == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    return plan;
}

cudaError_t launch_attn(const AttnParams& p, const AttnMaps& maps, AttnPlan plan, int D, bool f8,
                        int sms, cudaStream_t s) {
    const int rows = plan.rows, tk = plan.tk;
    int grid = plan.grid;
    cudaError_t e = D == 64    ? launch_attn_d64(p, maps, f8, rows, &grid, sms, s)
                    : D == 128 ? launch_attn_d128(p, maps, f8, rows, &grid, sms, s)
                               : launch_attn_d256(p, maps, f8, rows, &grid, sms, s);
    if (e != cudaSuccess) return e;
    return launch_attn_join(p, D, rows, grid, tk, sms, s);
}

cudaError_t launch_attn_join(const AttnParams& p, int D, int rows, int grid, int tk, int sms,
                             cudaStream_t s) {
    // Few rows in many parts: a warp 64 columns, for a row's parts are then asked for at
    // once (8 x 6 rows of 16 items of 256 in ten parts each: 29.2 us a call instead of
    // 31.0, one token of 4 items in nine parts 11.3 instead of 12.3).  Else a warp a row:
    // 256 items of 4 rows in one or two parts 146 us instead of 149, 128 rows of 32 items
    // 40.3 instead of 42.5.  About eight blocks an SM.  From 16 parts on the warps of a
    // block share them (8 rows of one item of 128 over 65536 tokens, in 304 parts: 23.5 us
    // instead of 39.4; 32 rows of 8 items in 19: 30.1 instead of 31.8; with ten parts it
    // took the 48 rows above 33.7 instead of 28.9).
    const int items = p.B * p.groups, used = p.tb * p.gb;
    const long long all = static_cast<long long>(items) * used;
    const bool fine = items <= grid / 4 && all <= 8 * sms;
    const bool parts = fine && items <= grid / 16;
    const int at_once = fine ? kJoinThreads * 2 / D : kJoinThreads / 32;
    int chunk = static_cast<int>((all + 8 * sms - 1) / (8 * sms));
    chunk = chunk < at_once ? at_once : chunk;
    if (chunk > used) chunk = used;
    cudaLaunchConfig_t cfg{};
    if (parts) chunk = 1;
    cfg.gridDim = dim3(items, parts ? used * (D / 64) : (used + chunk - 1) / chunk);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int mode = parts ? kJoinParts : (fine ? kJoinColumns : kJoinRows);
    auto* join = D == 64 ? join_of<64>(mode) : (D == 128 ? join_of<128>(mode) : join_of<256>(mode));
    return cudaLaunchKernelEx(&cfg, join, p, rows, grid, tk, chunk);
}

}  // namespace vw4
