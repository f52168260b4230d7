// read4.cu -- tokens of a 4-bit paged cache as contiguous rows of keys and values.
//
// value = e2m1(nibble) * e4m3(block scale) * head scale: the product of the first two is
// exact, that with the head's scale rounds to fp32, and to bf16 once more.
//
// One pass: 9/16 of a byte in and 2 bytes out a value, so the writes bound it.  A block
// takes kReadTokens tokens of a sequence at a time, whose page ids it looks up at once; a
// thread takes 8 values (4 bytes of codes, a scale), neighbouring threads neighbouring
// pieces, so that a warp writes 512 bytes in a row; four pieces a thread at a time, so that
// their loads are on their way together.
#include "attn.cuh"

namespace vw4 {

constexpr int kReadThreads = 256;
constexpr int kReadPieces = 4;
constexpr int kReadTokens = 32;

template <int D, bool F32>
__global__ void __launch_bounds__(kReadThreads) read4_kernel(const Read4Params p, int tiles,
                                                             uint32_t inv_per) {
    constexpr int C = D / 8;  // pieces of a head
    __shared__ int s_page[2][kReadTokens];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, is_v = blockIdx.y;
    const uint32_t per = static_cast<uint32_t>(p.Hkv * C);  // pieces of a token
    const uint8_t* src = is_v ? p.v : p.k;
    const uint8_t* blk = is_v ? p.blocks.v : p.blocks.k;
    const float* scales = is_v ? p.v_scale : p.k_scale;
    const long long cap = static_cast<long long>(p.max_blocks) << p.page_shift;
    const long long all = static_cast<long long>(tiles) * p.B;
    int turn = 0;
    for (long long w = blockIdx.x; w < all; w += gridDim.x, turn ^= 1) {
        const int b = static_cast<int>(w / tiles);
        const int t0 = static_cast<int>(w - static_cast<long long>(b) * tiles) * kReadTokens;
        const int nt = min(kReadTokens, p.n - t0);
        const int len = __ldg(p.seq_lens + b);
        const long long pos0 = (p.first ? __ldg(p.first + b) : static_cast<long long>(len) - p.n) + t0;
        if (tid < nt) {
            const long long pos = pos0 + tid;
            int page = -1;
            if (pos >= 0 && pos < len) {
                if (pos < cap)
                    page = __ldg(p.table + static_cast<long long>(b) * p.table_stride +
                                 (pos >> p.page_shift));
                if (page < 0 || page >= p.num_pages) {
                    page = -1;
                    atomicOr(p.status, kStatusBadPage);
                }
            }
            s_page[turn][tid] = page;
        }
        __syncthreads();  // (the other half of s_page is free: all have passed the last one)
        const uint32_t total = per * static_cast<uint32_t>(nt);  // at most 2^18
        const long long out0 = (static_cast<long long>(b) * p.n + t0) * per;
#pragma unroll 1
        for (uint32_t i0 = tid; i0 < total; i0 += kReadThreads * kReadPieces) {
            uint32_t code[kReadPieces];
            float f[kReadPieces];
#pragma unroll
            for (int q = 0; q < kReadPieces; ++q) {
                const uint32_t i = i0 + q * kReadThreads;
                code[q] = 0u;
                f[q] = 0.f;
                if (i >= total) continue;
                const uint32_t t = __umulhi(i, inv_per), r = i - t * per;  // i / per, the rest
                const int page = s_page[turn][t];
                if (page < 0) continue;
                const uint32_t h = r / C, c = r % C;
                const int place = static_cast<int>(pos0 + t) & (p.page_size - 1);
                code[q] = __ldg(reinterpret_cast<const uint32_t*>(
                    src + page * p.page_stride + place * p.token_stride + h * p.head_stride + c * 4));
                const uint32_t s = __ldg(blk + page * p.blocks.page_stride + h * p.blocks.head_stride +
                                         static_cast<long long>(place) * (D / 16) + c / 2);
                const uint32_t s2 = e4m3x2_f16x2(s);
                f[q] = __low2float(*reinterpret_cast<const __half2*>(&s2));
            }
#pragma unroll
            for (int q = 0; q < kReadPieces; ++q) {
                const uint32_t i = i0 + q * kReadThreads;
                if (i >= total) continue;
                const uint32_t h = (i - __umulhi(i, inv_per) * per) / C;
                const float g = scales ? __ldg(scales + h) : 1.f;
                uint32_t e[4];
                e2m1x8_f16(code[q], e);
                float v[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&e[j]));
                    // (a token that is not there: 0 * 0, whatever the head's scale is)
                    v[2 * j] = f[q] == 0.f ? 0.f : (x.x * f[q]) * g;
                    v[2 * j + 1] = f[q] == 0.f ? 0.f : (x.y * f[q]) * g;
                }
                const long long at = (out0 + i) * 8;
                if (F32) {
                    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(is_v ? p.v_out : p.k_out) + at);
                    dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                    dst[1] = make_float4(v[4], v[5], v[6], v[7]);
                } else {
                    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? p.v_out : p.k_out) + at) =
                        make_uint4(pack2<false>(v[0], v[1]), pack2<false>(v[2], v[3]),
                                   pack2<false>(v[4], v[5]), pack2<false>(v[6], v[7]));
                }
            }
        }
    }
}

cudaError_t launch_read4(const Read4Params& p, int sms, cudaStream_t s) {
    const int tiles = (p.n + kReadTokens - 1) / kReadTokens;
    const long long all = static_cast<long long>(tiles) * p.B, most = 8LL * sms;
    // i / per = i * inv >> 32: off by less than 1 / per for i < 2^18 and per <= 2^13
    const uint32_t per = static_cast<uint32_t>(p.Hkv * (p.D / 8));
    const uint32_t inv = static_cast<uint32_t>((0x100000000ull + per - 1) / per);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(all < most ? all : most), 2);
    cfg.blockDim = dim3(kReadThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void (*k)(const Read4Params, int, uint32_t) =
        p.D == 64    ? (p.out_f32 ? read4_kernel<64, true> : read4_kernel<64, false>)
        : p.D == 128 ? (p.out_f32 ? read4_kernel<128, true> : read4_kernel<128, false>)
                     : (p.out_f32 ? read4_kernel<256, true> : read4_kernel<256, false>);
    return cudaLaunchKernelEx(&cfg, k, p, tiles, inv);
}

}  // namespace vw4
