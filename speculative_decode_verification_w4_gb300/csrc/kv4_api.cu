// kv4_api.cu -- entry points of the 4-bit cache, of the pages' bookkeeping and of the
// committed tokens' log probabilities: argument checks and launches.
#include <cmath>

#include "vw4.h"
#include "vw4_internal.cuh"

using namespace vw4;

namespace {

bool misaligned(const void* p, unsigned bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

int shift_of(int n) {
    int s = 0;
    while ((1 << s) < n) ++s;
    return s;
}

bool page_size_ok(int n) { return n >= 8 && n <= 65536 && (n & (n - 1)) == 0; }

vw4_status check_cache(const vw4_kv4_cache& c, int B) {
    if (!c.k_dev || !c.v_dev || !c.k_blocks_dev || !c.v_blocks_dev || !c.block_table_dev)
        return VW4_ERR_INVALID_ARG;
    if (c.reserved != 0 || B < 1 || B > kMaxSeqs || c.Hkv < 1 || c.Hkv > kMaxHeads)
        return VW4_ERR_INVALID_ARG;
    if (c.num_pages < 1 || c.max_blocks < 1 || c.table_stride < c.max_blocks || c.page_size < 1)
        return VW4_ERR_INVALID_ARG;
    const int64_t strides[] = {c.page_stride, c.token_stride, c.head_stride, c.blocks_page_stride,
                               c.blocks_head_stride};
    for (const int64_t s : strides)
        if (s < 0) return VW4_ERR_INVALID_ARG;
    if (c.token_stride == 0 ||
        (c.num_pages > 1 && (c.page_stride == 0 || c.blocks_page_stride == 0)) ||
        (c.Hkv > 1 && (c.head_stride == 0 || c.blocks_head_stride == 0)))
        return VW4_ERR_INVALID_ARG;
    if (c.D != 64 && c.D != 128 && c.D != 256) return VW4_ERR_UNSUPPORTED;
    if (!page_size_ok(c.page_size)) return VW4_ERR_UNSUPPORTED;
    if (static_cast<long long>(c.max_blocks) * c.page_size > (1ll << 30)) return VW4_ERR_INVALID_ARG;
    for (const int64_t s : strides)
        if (s % 16) return VW4_ERR_ALIGN;
    if (misaligned(c.k_dev, 16) || misaligned(c.v_dev, 16) || misaligned(c.k_blocks_dev, 16) ||
        misaligned(c.v_blocks_dev, 16) || misaligned(c.block_table_dev, 4) ||
        misaligned(c.k_scale_dev, 4) || misaligned(c.v_scale_dev, 4))
        return VW4_ERR_ALIGN;
    return VW4_OK;
}

// R rows a sequence of Hq query heads on a cache
vw4_status check_rows(const vw4_kv4_cache& c, int B, int R, int Hq) {
    const vw4_status st = check_cache(c, B);
    if (st != VW4_OK) return st;
    if (R < 1 || R > kMaxVerifyRows || Hq < 1 || Hq > kMaxHeads || Hq % c.Hkv != 0)
        return VW4_ERR_INVALID_ARG;
    return VW4_OK;
}

vw4_status device(int* sms, uint32_t** status) {
    return static_cast<vw4_status>(current_device(sms, status));
}

vw4_status launched(cudaError_t e, const char* what) {
    return e == cudaSuccess ? VW4_OK : static_cast<vw4_status>(report_cuda(e, what));
}

}  // namespace

extern "C" {

VW4_API vw4_status verify_rope_append_kv4(const vw4_append_kv4* a, void* stream) {
    if (!a || !a->x_dev || !a->q_dev || !a->seq_lens_dev) return VW4_ERR_INVALID_ARG;
    const vw4_kv4_cache& c = a->kv;
    vw4_status st = check_rows(c, a->B, a->R, a->Hq);
    if (st != VW4_OK) return st;
    if ((a->x_bf16 != 0 && a->x_bf16 != 1) || (a->adjacent != 0 && a->adjacent != 1))
        return VW4_ERR_INVALID_ARG;
    if (a->rot < 0 || a->rot > c.D || a->rot % 2 || (a->rot > 0 && !a->inv_freq_dev))
        return VW4_ERR_INVALID_ARG;
    if (!(a->eps >= 0.f) || !std::isfinite(a->eps)) return VW4_ERR_INVALID_ARG;
    if (a->ldx < static_cast<int64_t>(a->Hq + 2 * c.Hkv) * c.D ||
        a->ldq < static_cast<int64_t>(a->Hq) * c.D)
        return VW4_ERR_INVALID_ARG;
    if (misaligned(a->x_dev, 16) || misaligned(a->q_dev, 16) || misaligned(a->inv_freq_dev, 8) ||
        misaligned(a->q_norm_dev, 16) || misaligned(a->k_norm_dev, 16) ||
        misaligned(a->seq_lens_dev, 4) || a->ldx % (a->x_bf16 ? 8 : 4) || a->ldq % 8)
        return VW4_ERR_ALIGN;
    int sms = 0;
    uint32_t* status = nullptr;
    st = device(&sms, &status);
    if (st != VW4_OK) return st;
    AppendParams p{};
    p.x = a->x_dev;
    p.x_bf16 = a->x_bf16;
    p.ldx = a->ldx;
    p.inv_freq = a->inv_freq_dev;
    p.q_norm = a->q_norm_dev;
    p.k_norm = a->k_norm_dev;
    p.eps = a->eps;
    p.rot = a->rot;
    p.adjacent = a->adjacent;
    p.q = static_cast<__nv_bfloat16*>(a->q_dev);
    p.ldq = a->ldq;
    p.seq_lens = a->seq_lens_dev;
    p.table = c.block_table_dev;
    p.k = c.k_dev;
    p.v = c.v_dev;
    p.k_scale = c.k_scale_dev;
    p.v_scale = c.v_scale_dev;
    p.status = status;
    p.table_stride = c.table_stride;
    p.page_stride = c.page_stride;
    p.token_stride = c.token_stride;
    p.head_stride = c.head_stride;
    p.B = a->B;
    p.R = a->R;
    p.Hq = a->Hq;
    p.Hkv = c.Hkv;
    p.D = c.D;
    p.page_size = c.page_size;
    p.page_shift = shift_of(c.page_size);
    p.max_blocks = c.max_blocks;
    p.num_pages = c.num_pages;
    p.k_blocks = static_cast<uint8_t*>(c.k_blocks_dev);
    p.v_blocks = static_cast<uint8_t*>(c.v_blocks_dev);
    p.blocks_page_stride = c.blocks_page_stride;
    p.blocks_head_stride = c.blocks_head_stride;
    return launched(launch_append(p, kCacheKv4, sms, static_cast<cudaStream_t>(stream)),
                    "verify_rope_append_kv4 launch");
}

VW4_API vw4_status verify_attn_kv4(const vw4_attn_kv4* a, void* workspace_dev, size_t ws_bytes,
                                   void* stream) {
    if (!a || !a->q_dev || !a->out_dev || !a->seq_lens_dev) return VW4_ERR_INVALID_ARG;
    const vw4_kv4_cache& c = a->kv;
    vw4_status st = check_rows(c, a->B, a->R, a->Hq);
    if (st != VW4_OK) return st;
    if (a->window < 0 || a->sinks < 0 || (a->sinks > 0 && a->window == 0))
        return VW4_ERR_INVALID_ARG;
    if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return VW4_ERR_INVALID_ARG;
    const int64_t width = static_cast<int64_t>(a->Hq) * c.D;
    if (a->ldq < width || a->ldo < width || a->ldo > kMaxOutStride) return VW4_ERR_INVALID_ARG;
    if (misaligned(a->q_dev, 16) || misaligned(a->out_dev, 16) || misaligned(a->lse_dev, 4) ||
        misaligned(a->seq_lens_dev, 4) || a->ldq % 8 || a->ldo % 8)
        return VW4_ERR_ALIGN;
    if (!workspace_dev || ws_bytes < attn4_workspace_bytes(a->B, a->R * (a->Hq / c.Hkv), c.D))
        return VW4_ERR_WORKSPACE;
    if (misaligned(workspace_dev, 256)) return VW4_ERR_ALIGN;
    int sms = 0;
    uint32_t* status = nullptr;
    st = device(&sms, &status);
    if (st != VW4_OK) return st;
    AttnParams p{};
    p.q = static_cast<const __nv_bfloat16*>(a->q_dev);
    p.k = c.k_dev;
    p.v = c.v_dev;
    p.table = c.block_table_dev;
    p.seq_lens = a->seq_lens_dev;
    p.k_scale = c.k_scale_dev;
    p.v_scale = c.v_scale_dev;
    p.out = static_cast<__nv_bfloat16*>(a->out_dev);
    p.lse = a->lse_dev;
    p.status = status;
    p.wait_ns = wait_limit_ns();
    p.ldq = a->ldq;
    p.ldo = a->ldo;
    p.table_stride = c.table_stride;
    p.page_stride = c.page_stride;
    p.token_stride = c.token_stride;
    p.head_stride = c.head_stride;
    p.scale = a->scale;
    p.B = a->B;
    p.R = a->R;
    p.Hq = a->Hq;
    p.Hkv = c.Hkv;
    p.G = a->Hq / c.Hkv;
    // a window or a count of first tokens beyond every length changes nothing
    p.window = a->window < (1 << 30) ? a->window : (1 << 30);
    p.sinks = a->sinks < (1 << 30) ? a->sinks : (1 << 30);
    p.page_size = c.page_size;
    p.page_shift = shift_of(c.page_size);
    p.max_blocks = c.max_blocks;
    p.num_pages = c.num_pages;
    const Attn4Plan plan = attn4_plan(p, c.D, workspace_dev);
    const Kv4Blocks kb{static_cast<const uint8_t*>(c.k_blocks_dev),
                       static_cast<const uint8_t*>(c.v_blocks_dev), c.blocks_page_stride,
                       c.blocks_head_stride};
    AttnMaps maps;
    // strides of dimensions of one element are never used, but must be valid
    const auto valid = [](int64_t v) { return v > 0 ? static_cast<uint64_t>(v) : 16u; };
    const uint64_t Hkv = static_cast<uint64_t>(c.Hkv), pages = static_cast<uint64_t>(c.num_pages);
    const uint64_t page = static_cast<uint64_t>(c.page_size), key = plan.box_bytes;
    const uint64_t token = valid(c.token_stride);
    const uint64_t groups = p.fold == kFoldGroups ? (Hkv - 1) * p.fold_step + page / 8 : page / 8;
    const uint64_t dims5[5] = {key, 8, p.fold == kFoldBlocks ? Hkv : 1, groups, pages};
    const uint64_t strides5[4] = {token, key, 8 * token, valid(c.page_stride)};
    const uint64_t dims4[4] = {key, Hkv, page, pages};
    const uint64_t strides4[3] = {valid(c.head_stride), token, valid(c.page_stride)};
    const uint32_t box5[5] = {static_cast<uint32_t>(key), 8u, 1u, static_cast<uint32_t>(p.box_rows / 8), 1u};
    const uint32_t box4[4] = {static_cast<uint32_t>(key), 1u, 8u, 1u};
    for (int v = 0; v < 2; ++v) {
        CUtensorMap* m = v ? &maps.v : &maps.k;
        const void* base = v ? c.v_dev : c.k_dev;
        st = static_cast<vw4_status>(
            p.fold != kFoldNone ? encode_map(m, false, 5, base, dims5, strides5, box5, plan.swizzle)
                                : encode_map(m, false, 4, base, dims4, strides4, box4, plan.swizzle));
        if (st != VW4_OK) return st;
    }
    const uint64_t qd[3] = {static_cast<uint64_t>(c.D), static_cast<uint64_t>(a->Hq),
                            static_cast<uint64_t>(a->B) * a->R};
    const uint64_t qs[2] = {static_cast<uint64_t>(c.D), static_cast<uint64_t>(a->ldq)};
    const uint32_t qb[3] = {64u, static_cast<uint32_t>(p.gb), static_cast<uint32_t>(p.tb)};
    st = static_cast<vw4_status>(
        encode_map(&maps.q, true, 3, a->q_dev, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B));
    if (st != VW4_OK) return st;
    return launched(launch_attn4(p, kb, maps, plan, c.D, sms, static_cast<cudaStream_t>(stream)),
                    "verify_attn_kv4 launch");
}

VW4_API vw4_status read_kv4(const vw4_read_kv4* a, void* stream) {
    if (!a || !a->seq_lens_dev || !a->k_out_dev || !a->v_out_dev) return VW4_ERR_INVALID_ARG;
    const vw4_kv4_cache& c = a->kv;
    vw4_status st = check_cache(c, a->B);
    if (st != VW4_OK) return st;
    if (a->n < 1 || a->n > (1 << 24) || (a->out_f32 != 0 && a->out_f32 != 1)) return VW4_ERR_INVALID_ARG;
    if (misaligned(a->seq_lens_dev, 4) || misaligned(a->first_dev, 4) ||
        misaligned(a->k_out_dev, 16) || misaligned(a->v_out_dev, 16))
        return VW4_ERR_ALIGN;
    int sms = 0;
    uint32_t* status = nullptr;
    st = device(&sms, &status);
    if (st != VW4_OK) return st;
    Read4Params p{};
    p.k = static_cast<const uint8_t*>(c.k_dev);
    p.v = static_cast<const uint8_t*>(c.v_dev);
    p.blocks = Kv4Blocks{static_cast<const uint8_t*>(c.k_blocks_dev),
                         static_cast<const uint8_t*>(c.v_blocks_dev), c.blocks_page_stride,
                         c.blocks_head_stride};
    p.k_scale = c.k_scale_dev;
    p.v_scale = c.v_scale_dev;
    p.table = c.block_table_dev;
    p.seq_lens = a->seq_lens_dev;
    p.first = a->first_dev;
    p.k_out = a->k_out_dev;
    p.v_out = a->v_out_dev;
    p.status = status;
    p.table_stride = c.table_stride;
    p.page_stride = c.page_stride;
    p.token_stride = c.token_stride;
    p.head_stride = c.head_stride;
    p.B = a->B;
    p.n = a->n;
    p.Hkv = c.Hkv;
    p.D = c.D;
    p.out_f32 = a->out_f32;
    p.page_size = c.page_size;
    p.page_shift = shift_of(c.page_size);
    p.max_blocks = c.max_blocks;
    p.num_pages = c.num_pages;
    return launched(launch_read4(p, sms, static_cast<cudaStream_t>(stream)), "read_kv4 launch");
}

VW4_API vw4_status advance_pages(const vw4_advance* a, void* workspace_dev, size_t ws_bytes,
                                 void* stream) {
    if (!a || !a->block_table_dev || !a->lens_dev || !a->held_dev || !a->free_dev ||
        !a->free_count_dev || !a->lens_out_dev || !a->held_out_dev || !a->free_count_out_dev ||
        !a->seq_lens_dev || !a->row_start_dev)
        return VW4_ERR_INVALID_ARG;
    if (a->B < 1 || a->B > kMaxSeqs || a->R < 0 || a->R > (1 << 20) || a->num_pages < 1 ||
        a->max_blocks < 1 || a->table_stride < a->max_blocks || a->page_size < 1)
        return VW4_ERR_INVALID_ARG;
    if (a->rows_max < 0 || a->rows_max > 2147483647LL) return VW4_ERR_INVALID_ARG;
    if (!page_size_ok(a->page_size)) return VW4_ERR_UNSUPPORTED;
    if (static_cast<long long>(a->max_blocks) * a->page_size > (1ll << 30)) return VW4_ERR_INVALID_ARG;
    const void* ptrs[] = {a->block_table_dev, a->lens_dev, a->accepted_dev, a->ended_dev,
                          a->grow_dev, a->held_dev, a->free_dev, a->free_count_dev,
                          a->lens_out_dev, a->held_out_dev, a->free_count_out_dev,
                          a->seq_lens_dev, a->row_start_dev};
    for (const void* q : ptrs)
        if (misaligned(q, 4)) return VW4_ERR_ALIGN;
    if (misaligned(a->slots_dev, 8)) return VW4_ERR_ALIGN;
    if (!workspace_dev || ws_bytes < advance_workspace_bytes(a->B)) return VW4_ERR_WORKSPACE;
    if (misaligned(workspace_dev, 256)) return VW4_ERR_ALIGN;
    int sms = 0;
    uint32_t* status = nullptr;
    const vw4_status st = device(&sms, &status);
    if (st != VW4_OK) return st;
    AdvanceParams p{};
    p.table = a->block_table_dev;
    p.lens = a->lens_dev;
    p.accepted = a->accepted_dev;
    p.ended = a->ended_dev;
    p.grow = a->grow_dev;
    p.held = a->held_dev;
    p.free_list = a->free_dev;
    p.free_count = a->free_count_dev;
    p.lens_out = a->lens_out_dev;
    p.held_out = a->held_out_dev;
    p.free_count_out = a->free_count_out_dev;
    p.seq_lens = a->seq_lens_dev;
    p.row_start = a->row_start_dev;
    p.slots = reinterpret_cast<long long*>(a->slots_dev);
    p.status = status;
    p.table_stride = a->table_stride;
    p.rows_max = a->rows_max;
    p.B = a->B;
    p.R = a->R;
    p.page_size = a->page_size;
    p.page_shift = shift_of(a->page_size);
    p.num_pages = a->num_pages;
    p.max_blocks = a->max_blocks;
    return launched(launch_advance(p, workspace_dev, sms, static_cast<cudaStream_t>(stream)),
                    "advance_pages launch");
}

VW4_API vw4_status token_logprobs(const vw4_logprobs* a, void* workspace_dev, size_t ws_bytes,
                                  void* stream) {
    if (!a || !a->x_dev) return VW4_ERR_INVALID_ARG;
    if (a->B < 1 || a->B > kMaxSeqs || a->R < 1 || a->R > kMaxVerifyRows || a->V < 1 ||
        a->V > (1 << 24) || a->ldx < a->V)
        return VW4_ERR_INVALID_ARG;
    if (a->top < 0 || a->top > kMaxTop || (a->x_bf16 != 0 && a->x_bf16 != 1)) return VW4_ERR_INVALID_ARG;
    // (beyond 2^126, scale log2(e) is infinite)
    if (!(a->scale > 0.f && a->scale <= 0x1p126f)) return VW4_ERR_INVALID_ARG;
    if ((a->logprob_dev || a->rank_dev) && !a->tokens_dev) return VW4_ERR_INVALID_ARG;
    if (a->top > 0 ? !a->top_ids_dev || !a->top_logprobs_dev : a->top_ids_dev || a->top_logprobs_dev)
        return VW4_ERR_INVALID_ARG;
    const void* ptrs[] = {a->tokens_dev, a->len_dev, a->logprob_dev, a->lse_dev, a->entropy_dev,
                          a->rank_dev, a->top_ids_dev, a->top_logprobs_dev};
    for (const void* q : ptrs)
        if (misaligned(q, 4)) return VW4_ERR_ALIGN;
    if (misaligned(a->x_dev, a->x_bf16 ? 2 : 4)) return VW4_ERR_ALIGN;
    const long long rows = static_cast<long long>(a->B) * a->R;
    if (!workspace_dev || ws_bytes < logprob_workspace_bytes(rows, a->V, a->top))
        return VW4_ERR_WORKSPACE;
    if (misaligned(workspace_dev, 256)) return VW4_ERR_ALIGN;
    int sms = 0;
    uint32_t* status = nullptr;
    const vw4_status st = device(&sms, &status);
    if (st != VW4_OK) return st;
    LogprobParams p{};
    p.x = a->x_dev;
    p.tokens = a->tokens_dev;
    p.len = a->len_dev;
    p.logprob = a->logprob_dev;
    p.lse = a->lse_dev;
    p.entropy = a->entropy_dev;
    p.rank = a->rank_dev;
    p.top_ids = a->top_ids_dev;
    p.top_logprobs = a->top_logprobs_dev;
    p.status = status;
    p.ldx = a->ldx;
    p.scale = a->scale;
    p.B = a->B;
    p.R = a->R;
    p.V = a->V;
    p.top = a->top;
    p.x_bf16 = a->x_bf16;
    return launched(launch_logprobs(p, workspace_dev, sms, static_cast<cudaStream_t>(stream)),
                    "token_logprobs launch");
}

}  // extern "C"
