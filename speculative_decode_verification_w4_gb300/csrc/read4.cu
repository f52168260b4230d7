// read4.cu -- tokens of a 4-bit paged cache as contiguous rows of keys and values.
//
// value = e2m1(nibble) * e4m3(block scale) * head scale: the product of the first two is
// exact in f16, that with the head's scale rounds to fp32, and to bf16 once more.
//
// One pass: 9/16 of a byte in and 2 bytes out a value, so the writes bound it.  A thread
// takes 32 values of K or of V (16 bytes of codes, two scales), neighbouring threads
// neighbouring pieces of the output, four pieces a thread at a time, so that their loads
// (page id, codes, scales) are on their way together.
#include "attn.cuh"

namespace vw4 {

constexpr int kReadThreads = 256;
constexpr int kReadPieces = 4;

template <int D, bool F32>
__global__ void __launch_bounds__(kReadThreads) read4_kernel(const Read4Params p) {
    constexpr int C = D / 32;  // pieces of a head
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.y, is_v = blockIdx.z;
    const int per = p.Hkv * C;  // pieces of a token
    const long long total = static_cast<long long>(p.n) * per;
    const int len = __ldg(p.seq_lens + b);
    const long long first = p.first ? __ldg(p.first + b) : static_cast<long long>(len) - p.n;
    const uint8_t* src = is_v ? p.v : p.k;
    const uint8_t* blk = is_v ? p.blocks.v : p.blocks.k;
    const float* scales = is_v ? p.v_scale : p.k_scale;
    const int32_t* table = p.table + static_cast<long long>(b) * p.table_stride;
    const long long cap = static_cast<long long>(p.max_blocks) << p.page_shift;
    bool bad = false;
    const long long step = static_cast<long long>(gridDim.x) * kReadThreads;
    for (long long i0 = static_cast<long long>(blockIdx.x) * kReadThreads + threadIdx.x; i0 < total;
         i0 += step * kReadPieces) {
        int page[kReadPieces], h[kReadPieces], c[kReadPieces];
        long long pos[kReadPieces];
#pragma unroll
        for (int q = 0; q < kReadPieces; ++q) {
            const long long i = i0 + q * step;
            page[q] = -1;
            if (i >= total) continue;
            const uint32_t t = static_cast<uint32_t>(i / per);
            const int r = static_cast<int>(i - static_cast<long long>(t) * per);
            h[q] = r / C;
            c[q] = r % C;
            pos[q] = first + t;
            if (pos[q] >= 0 && pos[q] < len) {
                if (pos[q] < cap) page[q] = __ldg(table + (pos[q] >> p.page_shift));
                if (page[q] < 0 || page[q] >= p.num_pages) {
                    bad = true;
                    page[q] = -1;
                }
            }
        }
        uint4 w[kReadPieces];
        uint16_t s[kReadPieces];
        float g[kReadPieces];
#pragma unroll
        for (int q = 0; q < kReadPieces; ++q) {
            w[q] = make_uint4(0, 0, 0, 0);
            s[q] = 0;
            g[q] = 1.f;
            if (page[q] < 0) continue;
            const int place = static_cast<int>(pos[q]) & (p.page_size - 1);
            w[q] = __ldg(reinterpret_cast<const uint4*>(src + page[q] * p.page_stride +
                                                        place * p.token_stride +
                                                        h[q] * p.head_stride + c[q] * 16));
            s[q] = __ldg(reinterpret_cast<const uint16_t*>(
                blk + page[q] * p.blocks.page_stride + h[q] * p.blocks.head_stride +
                static_cast<long long>(place) * (D / 16) + c[q] * 2));
            if (scales) g[q] = __ldg(scales + h[q]);
        }
#pragma unroll
        for (int q = 0; q < kReadPieces; ++q) {
            const long long i = i0 + q * step;
            if (i >= total) continue;
            const uint32_t sp = e4m3x2_f16x2(s[q]);
            const float2 sf = __half22float2(*reinterpret_cast<const __half2*>(&sp));
            const uint32_t words[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
            float f[32];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t e[4];
                e2m1x8_f16(words[k], e);
                const float sc = k < 2 ? sf.x : sf.y;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&e[j]));
                    // (x * g rounds; a zero of an absent token stays one)
                    f[8 * k + 2 * j] = page[q] < 0 ? 0.f : (v.x * sc) * g[q];
                    f[8 * k + 2 * j + 1] = page[q] < 0 ? 0.f : (v.y * sc) * g[q];
                }
            }
            const long long at = (static_cast<long long>(b) * total + i) * 32;
            if (F32) {
                float4* dst = reinterpret_cast<float4*>(static_cast<float*>(is_v ? p.v_out : p.k_out) + at);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    dst[k] = make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
            } else {
                uint4* dst = reinterpret_cast<uint4*>(
                    static_cast<__nv_bfloat16*>(is_v ? p.v_out : p.k_out) + at);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    dst[k] = make_uint4(pack2<false>(f[8 * k], f[8 * k + 1]),
                                        pack2<false>(f[8 * k + 2], f[8 * k + 3]),
                                        pack2<false>(f[8 * k + 4], f[8 * k + 5]),
                                        pack2<false>(f[8 * k + 6], f[8 * k + 7]));
            }
        }
    }
    if (bad) atomicOr(p.status, kStatusBadPage);
}

cudaError_t launch_read4(const Read4Params& p, int sms, cudaStream_t s) {
    const long long pieces = static_cast<long long>(p.n) * p.Hkv * (p.D / 32);
    const long long want = (pieces + kReadThreads * kReadPieces - 1) / (kReadThreads * kReadPieces);
    const long long most = (16LL * sms + 2 * p.B - 1) / (2 * p.B);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(want < most ? want : most), p.B, 2);
    cfg.blockDim = dim3(kReadThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void (*k)(const Read4Params) =
        p.D == 64    ? (p.out_f32 ? read4_kernel<64, true> : read4_kernel<64, false>)
        : p.D == 128 ? (p.out_f32 ? read4_kernel<128, true> : read4_kernel<128, false>)
                     : (p.out_f32 ? read4_kernel<256, true> : read4_kernel<256, false>);
    return cudaLaunchKernelEx(&cfg, k, p);
}

}  // namespace vw4
