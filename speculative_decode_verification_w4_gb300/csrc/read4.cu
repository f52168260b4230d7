// read4.cu -- tokens of a 4-bit paged cache as contiguous rows of keys and values.
//
// value = e2m1(nibble) * e4m3(block scale) * head scale: the product of the first two is
// exact, that with the head's scale rounds to fp32, and to bf16 once more.
//
// One pass: 9/16 of a byte in and 2 bytes out a value, so the writes bound it: 8192 tokens of 16
// sequences, 8 heads of size 128, 108 us in bf16 (96 at the copy rate) and 282 in fp32 (174; a
// thread's 32 bytes are two stores there).  A block
// takes kReadTokens tokens of a sequence at a time, whose places in the cache it looks up at
// once; a thread takes 8 values (4 bytes of codes, a scale) of the same place of several
// tokens, neighbouring threads neighbouring pieces, so that a warp writes 512 bytes in a
// row and the addresses are a sum; four pieces at a time, so that their loads are on their
// way together.
#include "attn.cuh"

namespace vw4 {

constexpr int kReadThreads = 256;
constexpr int kReadPieces = 4;
constexpr int kReadTokens = 32;

template <int D, bool F32>
__global__ void __launch_bounds__(kReadThreads) read4_kernel(const Read4Params p, int tiles) {
    constexpr int C = D / 8;  // pieces of a head
    __shared__ longlong2 s_at[2][kReadTokens];  // a token's codes and scales (below 0: none)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, is_v = blockIdx.y;
    const int per = p.Hkv * C;  // pieces of a token
    const uint8_t* src = is_v ? p.v : p.k;
    const uint8_t* blk = is_v ? p.blocks.v : p.blocks.k;
    const float* scales = is_v ? p.v_scale : p.k_scale;
    const long long cap = static_cast<long long>(p.max_blocks) << p.page_shift;
    const long long all = static_cast<long long>(tiles) * p.B;
    // a thread's first piece of a token, and the tokens that the block's threads reach at once
    const int at_once = per < kReadThreads ? kReadThreads / per : 1;
    const int t_first = per < kReadThreads ? tid / per : 0;
    const int r_first = per < kReadThreads ? tid - t_first * per : tid;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int turn = 0;
    for (long long w = blockIdx.x; w < all; w += gridDim.x, turn ^= 1) {
        const int b = static_cast<int>(w / tiles);
        const int t0 = static_cast<int>(w - static_cast<long long>(b) * tiles) * kReadTokens;
        const int nt = min(kReadTokens, p.n - t0);
        if (tid < nt) {
            const int len = __ldg(p.seq_lens + b);
            const long long pos = (p.first ? __ldg(p.first + b) : static_cast<long long>(len) - p.n) + t0 + tid;
            longlong2 at = make_longlong2(-1, -1);
            if (pos >= 0 && pos < len) {
                int page = -1;
                if (pos < cap)
                    page = __ldg(p.table + static_cast<long long>(b) * p.table_stride +
                                 (pos >> p.page_shift));
                const int place = static_cast<int>(pos) & (p.page_size - 1);
                if (page >= 0 && page < p.num_pages)
                    at = make_longlong2(page * p.page_stride + place * p.token_stride,
                                        page * p.blocks.page_stride + static_cast<long long>(place) * (D / 16));
                else
                    atomicOr(p.status, kStatusBadPage);
            }
            s_at[turn][tid] = at;
        }
        __syncthreads();  // (the other half of s_at is free: all have passed the last one)
        if (t_first >= at_once) continue;  // (threads of no whole token)
#pragma unroll 1
        for (int r = r_first; r < per; r += kReadThreads) {
            const int h = r / C, c = r % C;
            const uint8_t* s_codes = src + h * p.head_stride + c * 4;
            const uint8_t* s_blocks = blk + h * p.blocks.head_stride + c / 2;
            const float g = scales ? __ldg(scales + h) : 1.f;
            const long long out0 = ((static_cast<long long>(b) * p.n + t0) * per + r) * 8;
#pragma unroll 1
            for (int q0 = t_first; q0 < nt; q0 += at_once * kReadPieces) {
                uint32_t code[kReadPieces], sb[kReadPieces];
#pragma unroll
                for (int q = 0; q < kReadPieces; ++q) {
                    const int t = q0 + q * at_once;
                    code[q] = sb[q] = 0u;
                    if (t >= nt) continue;
                    const longlong2 at = s_at[turn][t];
                    if (at.x < 0) continue;
                    code[q] = __ldg(reinterpret_cast<const uint32_t*>(s_codes + at.x));
                    sb[q] = __ldg(s_blocks + at.y);
                }
#pragma unroll
                for (int q = 0; q < kReadPieces; ++q) {
                    const int t = q0 + q * at_once;
                    if (t >= nt) continue;
                    // (a token that is not there: 0 * 0, whatever the head's scale is)
                    const uint32_t s2 = e4m3x2_f16x2(sb[q]);
                    const float f = __low2float(*reinterpret_cast<const __half2*>(&s2));
                    const float k = sb[q] ? g : 0.f;
                    uint32_t e[4];
                    e2m1x8_f16(code[q], e);
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&e[j]));
                        v[2 * j] = (x.x * f) * k;
                        v[2 * j + 1] = (x.y * f) * k;
                    }
                    const long long at = out0 + static_cast<long long>(t) * per * 8;
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
}

cudaError_t launch_read4(const Read4Params& p, int sms, cudaStream_t s) {
    const int tiles = (p.n + kReadTokens - 1) / kReadTokens;
    const long long all = static_cast<long long>(tiles) * p.B, most = 8LL * sms;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(all < most ? all : most), 2);
    cfg.blockDim = dim3(kReadThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void (*k)(const Read4Params, int) =
        p.D == 64    ? (p.out_f32 ? read4_kernel<64, true> : read4_kernel<64, false>)
        : p.D == 128 ? (p.out_f32 ? read4_kernel<128, true> : read4_kernel<128, false>)
                     : (p.out_f32 ? read4_kernel<256, true> : read4_kernel<256, false>);
    return cudaLaunchKernelEx(&cfg, k, p, tiles);
}

}  // namespace vw4
