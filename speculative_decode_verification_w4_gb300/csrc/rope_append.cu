// rope_append.cu -- from the packed qkv rows of the verify GEMM to rotated
// queries and cache entries: per head an optional RMS norm, the rotation of
// its leading dimensions by the token's position, and the rounding to bf16 or
// (for the cache) to e4m3 of value / scale.
//
// One pass: every value is read once and written once, so the bytes bound it.
// A block takes one token and some of its heads, a warp one head at a time;
// the token's sines and cosines are computed once per block, the angle
// position * inv_freq in 64 bits (in 32 a position of 2^17 would lose 2^-7 of
// a radian), reduced to a fraction of a turn before it is rounded.
#include "attn.cuh"

namespace vw4 {

constexpr int kAppendWarps = 4;
constexpr int kMaxPairs = 128;

template <int D, bool F8>
__global__ void __launch_bounds__(kAppendWarps * 32) append_kernel(const AppendParams p,
                                                                   int heads_per_block) {
    constexpr int E = D / 32;  // consecutive dimensions of a lane
    __shared__ float s_cos[kMaxPairs], s_sin[kMaxPairs];
    __shared__ __align__(16) float s_head[kAppendWarps][D];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int token = blockIdx.x, b = token / p.R, i = token - b * p.R;
    const int pairs = p.rot / 2;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int pos = p.seq_lens[b] - p.R + i;
    for (int j = threadIdx.x; j < pairs; j += kAppendWarps * 32) {
        double turns = static_cast<double>(pos) * p.inv_freq[j] * 0.15915494309189535;
        turns -= rint(turns);
        sincospif(static_cast<float>(2.0 * turns), &s_sin[j], &s_cos[j]);
    }
    // the token's cache slot
    long long slot = -1;
    if (pos >= 0) {
        const int blk = pos >> p.page_shift;
        const int pg = blk < p.max_blocks
                           ? __ldg(p.table + static_cast<long long>(b) * p.table_stride + blk)
                           : -1;
        if (pg >= 0 && pg < p.num_pages)
            slot = static_cast<long long>(pg) * p.page_stride +
                   static_cast<long long>(pos & (p.page_size - 1)) * p.token_stride;
        else if (threadIdx.x == 0)
            atomicOr(p.status, kStatusBadPage);
    }
    __syncthreads();

    const int heads = p.Hq + 2 * p.Hkv;
    const int h_end = min(heads, (static_cast<int>(blockIdx.y) + 1) * heads_per_block);
    const int d0 = lane * E;
    auto load = [&](int h, float* v) {
        const long long at = static_cast<long long>(token) * p.ldx + static_cast<long long>(h) * D + d0;
        if (p.x_bf16) {
            const uint32_t* src = reinterpret_cast<const uint32_t*>(
                static_cast<const __nv_bfloat16*>(p.x) + at);
            uint32_t w[E / 2];
            if (E == 8) *reinterpret_cast<uint4*>(w) = __ldg(reinterpret_cast<const uint4*>(src));
            else if (E == 4) *reinterpret_cast<uint2*>(w) = __ldg(reinterpret_cast<const uint2*>(src));
            else w[0] = __ldg(src);
#pragma unroll
            for (int k = 0; k < E / 2; ++k) {
                v[2 * k] = __uint_as_float(w[k] << 16);
                v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
            }
        } else {
            const float* src = static_cast<const float*>(p.x) + at;
            if (E == 2) {
                *reinterpret_cast<float2*>(v) = __ldg(reinterpret_cast<const float2*>(src));
            } else {
#pragma unroll
                for (int k = 0; k < E; k += 4)
                    *reinterpret_cast<float4*>(v + k) = __ldg(reinterpret_cast<const float4*>(src + k));
            }
        }
    };
    int h = blockIdx.y * heads_per_block + warp;
    __align__(16) float v[8], nx[8];
    if (h < h_end) load(h, v);
    for (; h < h_end; h += kAppendWarps) {
        const bool more = h + kAppendWarps < h_end;
        if (more) load(h + kAppendWarps, nx);
        const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hkv;
        if (is_q || is_k) {
            const float* w = is_q ? p.q_norm : p.k_norm;
            if (w) {
                float ss = 0.f;
#pragma unroll
                for (int k = 0; k < E; ++k) ss = fmaf(v[k], v[k], ss);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float f = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
                for (int k = 0; k < E; ++k) v[k] = v[k] * f * __ldg(w + d0 + k);
            }
            if (pairs > 0 && p.adjacent) {
#pragma unroll
                for (int k = 0; k < E; k += 2) {
                    const int j = (d0 + k) / 2;
                    if (j < pairs) {
                        const float a = v[k], c = v[k + 1];
                        v[k] = a * s_cos[j] - c * s_sin[j];
                        v[k + 1] = c * s_cos[j] + a * s_sin[j];
                    }
                }
            } else if (pairs > 0) {
                __syncwarp();  // the last head's reads are done
#pragma unroll
                for (int k = 0; k < E; ++k) s_head[warp][d0 + k] = v[k];
                __syncwarp();
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const int d = d0 + k;
                    if (d < pairs) v[k] = v[k] * s_cos[d] - s_head[warp][d + pairs] * s_sin[d];
                    else if (d < p.rot)
                        v[k] = v[k] * s_cos[d - pairs] + s_head[warp][d - pairs] * s_sin[d - pairs];
                }
            }
        }
        uint32_t w16[4];
        if (is_q || !F8) {
#pragma unroll
            for (int k = 0; k < E / 2; ++k) w16[k] = pack2<false>(v[2 * k], v[2 * k + 1]);
        }
        void* dst = nullptr;
        const int hk = is_k ? h - p.Hq : h - p.Hq - p.Hkv;
        if (is_q) {
            dst = p.q + static_cast<long long>(token) * p.ldq + static_cast<long long>(h) * D + d0;
        } else if (slot >= 0) {
            const long long at = slot + static_cast<long long>(hk) * p.head_stride + d0;
            uint8_t* base = static_cast<uint8_t*>(is_k ? p.k : p.v);
            dst = base + at * (F8 ? 1 : 2);
        }
        if (dst && (is_q || !F8)) {
            if (E == 8) *static_cast<uint4*>(dst) = make_uint4(w16[0], w16[1], w16[2], w16[3]);
            else if (E == 4) *static_cast<uint2*>(dst) = make_uint2(w16[0], w16[1]);
            else *static_cast<uint32_t*>(dst) = w16[0];
        } else if (dst) {
            const float* sp = is_k ? p.k_scale : p.v_scale;
            const float sc = sp ? __ldg(sp + hk) : 1.f;
            uint16_t w8[4];
#pragma unroll
            for (int k = 0; k < E / 2; ++k)  // nearest, ties to even; beyond 448: 448
                w8[k] = __nv_cvt_float2_to_fp8x2(
                    make_float2(__fdiv_rn(v[2 * k], sc), __fdiv_rn(v[2 * k + 1], sc)),
                    __NV_SATFINITE, __NV_E4M3);
            if (E == 8)
                *static_cast<uint2*>(dst) =
                    make_uint2(w8[0] | (uint32_t(w8[1]) << 16), w8[2] | (uint32_t(w8[3]) << 16));
            else if (E == 4) *static_cast<uint32_t*>(dst) = w8[0] | (uint32_t(w8[1]) << 16);
            else *static_cast<uint16_t*>(dst) = w8[0];
        }
#pragma unroll
        for (int k = 0; k < E; ++k) v[k] = nx[k];
    }
}

cudaError_t launch_append(const AppendParams& p, bool f8, int sms, cudaStream_t s) {
    const int tokens = p.B * p.R, heads = p.Hq + 2 * p.Hkv;
    // one head a warp while that leaves SMs idle; else more heads share a block's angles
    const int want = 8 * sms;
    int per = static_cast<int>((static_cast<long long>(tokens) * heads + want - 1) / want);
    per = (per + kAppendWarps - 1) / kAppendWarps * kAppendWarps;
    if (per < kAppendWarps) per = kAppendWarps;
    if (per > heads) per = heads;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(tokens, (heads + per - 1) / per);
    cfg.blockDim = dim3(kAppendWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void (*k)(const AppendParams, int);
    if (p.D == 64) k = f8 ? append_kernel<64, true> : append_kernel<64, false>;
    else if (p.D == 128) k = f8 ? append_kernel<128, true> : append_kernel<128, false>;
    else k = f8 ? append_kernel<256, true> : append_kernel<256, false>;
    return cudaLaunchKernelEx(&cfg, k, p, per);
}

}  // namespace vw4
