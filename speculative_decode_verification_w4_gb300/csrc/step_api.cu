// step_api.cu -- entry points between the verify GEMMs of a step (cache append,
// attention, logits processing): argument checks and launches.
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

vw4_status check_cache(const vw4_kv_cache& c, int B, int R, int Hq) {
    if (c.dtype != VW4_KV_BF16 && c.dtype != VW4_KV_E4M3) return VW4_ERR_INVALID_ARG;
    if (!c.k_dev || !c.v_dev || !c.block_table_dev) return VW4_ERR_INVALID_ARG;
    if (B < 1 || B > kMaxSeqs || R < 1 || R > kMaxVerifyRows) return VW4_ERR_INVALID_ARG;
    if (c.Hkv < 1 || Hq < 1 || Hq > kMaxHeads || Hq % c.Hkv != 0) return VW4_ERR_INVALID_ARG;
    if (c.num_pages < 1 || c.max_blocks < 1 || c.table_stride < c.max_blocks)
        return VW4_ERR_INVALID_ARG;
    if (c.page_size < 1 || c.page_stride < 0 || c.token_stride < 0 || c.head_stride < 0)
        return VW4_ERR_INVALID_ARG;
    if (c.token_stride == 0 || (c.num_pages > 1 && c.page_stride == 0) ||
        (c.Hkv > 1 && c.head_stride == 0))
        return VW4_ERR_INVALID_ARG;
    if (c.D != 64 && c.D != 128 && c.D != 256) return VW4_ERR_UNSUPPORTED;
    if (c.page_size < 8 || c.page_size > 65536 || (c.page_size & (c.page_size - 1)))
        return VW4_ERR_UNSUPPORTED;
    if (static_cast<long long>(c.max_blocks) * c.page_size > (1ll << 30)) return VW4_ERR_INVALID_ARG;
    if (c.dtype == VW4_KV_BF16 && (c.k_scale_dev || c.v_scale_dev)) return VW4_ERR_INVALID_ARG;
    const int step = c.dtype == VW4_KV_BF16 ? 8 : 16;  // elements of 16 bytes
    if (misaligned(c.k_dev, 16) || misaligned(c.v_dev, 16) || c.page_stride % step ||
        c.token_stride % step || c.head_stride % step || misaligned(c.block_table_dev, 4) ||
        misaligned(c.k_scale_dev, 4) || misaligned(c.v_scale_dev, 4))
        return VW4_ERR_ALIGN;
    return VW4_OK;
}

}  // namespace

extern "C" {

VW4_API vw4_status verify_rope_append(const vw4_append* a, void* stream) {
    if (!a || !a->x_dev || !a->q_dev || !a->seq_lens_dev) return VW4_ERR_INVALID_ARG;
    vw4_status st = check_cache(a->kv, a->B, a->R, a->Hq);
    if (st != VW4_OK) return st;
    const vw4_kv_cache& c = a->kv;
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
    st = static_cast<vw4_status>(current_device(&sms, &status));
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
    const cudaError_t e =
        launch_append(p, c.dtype == VW4_KV_E4M3 ? kCacheE4m3 : kCacheBf16, sms,
                      static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess)
        return static_cast<vw4_status>(report_cuda(e, "verify_rope_append launch"));
    return VW4_OK;
}

VW4_API vw4_status verify_attn(const vw4_attn* a, void* workspace_dev, size_t ws_bytes,
                               void* stream) {
    if (!a || !a->q_dev || !a->out_dev || !a->seq_lens_dev) return VW4_ERR_INVALID_ARG;
    vw4_status st = check_cache(a->kv, a->B, a->R, a->Hq);
    if (st != VW4_OK) return st;
    const vw4_kv_cache& c = a->kv;
    if (a->window < 0 || a->sinks < 0 || (a->sinks > 0 && a->window == 0))
        return VW4_ERR_INVALID_ARG;
    if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return VW4_ERR_INVALID_ARG;
    const int64_t width = static_cast<int64_t>(a->Hq) * c.D;
    if (a->ldq < width || a->ldo < width || a->ldo > kMaxOutStride) return VW4_ERR_INVALID_ARG;
    if (misaligned(a->q_dev, 16) || misaligned(a->out_dev, 16) || misaligned(a->lse_dev, 4) ||
        misaligned(a->seq_lens_dev, 4) || a->ldq % 8 || a->ldo % 8)
        return VW4_ERR_ALIGN;
    const int rows = a->R * (a->Hq / c.Hkv);
    if (!workspace_dev || ws_bytes < attn_workspace_bytes(a->B, rows, c.D))
        return VW4_ERR_WORKSPACE;
    if (misaligned(workspace_dev, 256)) return VW4_ERR_ALIGN;
    int sms = 0;
    uint32_t* status = nullptr;
    st = static_cast<vw4_status>(current_device(&sms, &status));
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
    const bool f8 = c.dtype == VW4_KV_E4M3;
    const AttnPlan plan = attn_plan(p, c.D, f8, workspace_dev);
    AttnMaps maps;
    {
        // strides of dimensions of one element are never used, but must be valid
        const uint64_t step = f8 ? 16 : 8;
        const auto valid = [step](int64_t v) { return v > 0 ? static_cast<uint64_t>(v) : step; };
        const uint64_t Hkv = static_cast<uint64_t>(c.Hkv), pages = static_cast<uint64_t>(c.num_pages);
        const uint64_t page = static_cast<uint64_t>(c.page_size), block = plan.box_bytes / (f8 ? 1 : 2);
        const uint64_t all = static_cast<uint64_t>(c.D) / block, token = valid(c.token_stride);
        const uint64_t groups = p.fold == kFoldGroups ? (Hkv - 1) * p.fold_step + page / 8 : page / 8;
        const uint64_t dims5[5] = {block, 8, p.fold == kFoldBlocks ? Hkv * all : all, groups, pages};
        const uint64_t strides5[4] = {token, block, 8 * token, valid(c.page_stride)};
        const uint64_t dims4[4] = {static_cast<uint64_t>(c.D), Hkv, page, pages};
        const uint64_t strides4[3] = {valid(c.head_stride), token, valid(c.page_stride)};
        for (int v = 0; v < 2; ++v) {
            const uint32_t box5[5] = {static_cast<uint32_t>(block), 8u,
                                      static_cast<uint32_t>(v ? plan.v_blocks : plan.k_blocks),
                                      static_cast<uint32_t>(p.box_rows / 8), 1u};
            const uint32_t box4[4] = {static_cast<uint32_t>(block), 1u, 8u, 1u};
            CUtensorMap* m = v ? &maps.v : &maps.k;
            const void* base = v ? c.v_dev : c.k_dev;
            st = static_cast<vw4_status>(
                p.fold != kFoldNone ? encode_map(m, !f8, 5, base, dims5, strides5, box5, plan.swizzle)
                                    : encode_map(m, !f8, 4, base, dims4, strides4, box4, plan.swizzle));
            if (st != VW4_OK) return st;
        }
        const uint64_t qd[3] = {static_cast<uint64_t>(c.D), static_cast<uint64_t>(a->Hq),
                                static_cast<uint64_t>(a->B) * a->R};
        const uint64_t qs[2] = {static_cast<uint64_t>(c.D), static_cast<uint64_t>(a->ldq)};
        const uint32_t qb[3] = {64u, static_cast<uint32_t>(p.gb), static_cast<uint32_t>(p.tb)};
        st = static_cast<vw4_status>(
            encode_map(&maps.q, true, 3, a->q_dev, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B));
        if (st != VW4_OK) return st;
    }
    const cudaError_t e =
        launch_attn(p, maps, plan, c.D, f8, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return static_cast<vw4_status>(report_cuda(e, "verify_attn launch"));
    return VW4_OK;
}

VW4_API vw4_status process_logits(const vw4_logits* a, void* stream) {
    if (!a || !a->x_dev || !a->out_dev) return VW4_ERR_INVALID_ARG;
    if (a->B < 1 || a->B > kMaxSeqs || a->R < 1 || a->R > kMaxVerifyRows || a->V < 1 ||
        a->V > (1 << 24))
        return VW4_ERR_INVALID_ARG;
    if (a->ldx < a->V || a->ldo < a->V || (a->out_dev == a->x_dev && a->ldo != a->ldx))
        return VW4_ERR_INVALID_ARG;
    if (a->R > 1 && !a->drafts_dev) return VW4_ERR_INVALID_ARG;
    if (a->history_dev && (a->hist_max < 0 || a->hist_stride < a->hist_max))
        return VW4_ERR_INVALID_ARG;
    if (!a->bias_ids_dev != !a->bias_vals_dev) return VW4_ERR_INVALID_ARG;
    if (a->bias_ids_dev && (a->bias_max < 0 || a->bias_stride < a->bias_max))
        return VW4_ERR_INVALID_ARG;
    if (a->mask_dev && (a->mask_rows < 1 || a->mask_stride < (a->V + 31) / 32))
        return VW4_ERR_INVALID_ARG;
    const void* ptrs[] = {a->x_dev, a->out_dev, a->block_max_dev, a->drafts_dev, a->history_dev,
                          a->hist_len_dev, a->prompt_len_dev, a->repetition_dev, a->presence_dev,
                          a->frequency_dev, a->bias_ids_dev, a->bias_vals_dev, a->bias_len_dev,
                          a->mask_dev, a->mask_index_dev};
    for (const void* q : ptrs)
        if (misaligned(q, 4)) return VW4_ERR_ALIGN;
    int sms = 0;
    uint32_t* status = nullptr;
    const vw4_status st = static_cast<vw4_status>(current_device(&sms, &status));
    if (st != VW4_OK) return st;
    LogitsParams p{};
    p.x = a->x_dev;
    p.out = a->out_dev;
    p.bmax = a->block_max_dev;
    p.drafts = a->drafts_dev;
    p.history = a->history_dev;
    p.hist_len = a->hist_len_dev;
    p.prompt_len = a->prompt_len_dev;
    p.repetition = a->repetition_dev;
    p.presence = a->presence_dev;
    p.frequency = a->frequency_dev;
    p.bias_ids = a->bias_ids_dev;
    p.bias_vals = a->bias_vals_dev;
    p.bias_len = a->bias_len_dev;
    p.mask = a->mask_dev;
    p.mask_index = a->mask_index_dev;
    p.status = status;
    p.ldx = a->ldx;
    p.ldo = a->ldo;
    p.hist_stride = a->hist_stride;
    p.bias_stride = a->bias_stride;
    p.mask_stride = a->mask_stride;
    p.B = a->B;
    p.R = a->R;
    p.V = a->V;
    p.hist_max = a->history_dev ? a->hist_max : 0;
    p.bias_max = a->bias_ids_dev ? a->bias_max : 0;
    p.mask_rows = a->mask_dev ? a->mask_rows : 0;
    const cudaError_t e = launch_logits(p, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return static_cast<vw4_status>(report_cuda(e, "process_logits launch"));
    return VW4_OK;
}

}  // extern "C"
