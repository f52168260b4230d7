// rope_append.cu -- from the packed qkv rows of the verify GEMM to rotated
// queries and cache entries: per head an optional RMS norm, the rotation of
// its leading dimensions by the token's position, and the rounding to bf16 or
// (for the cache) to e4m3 of value / scale.
//
// One pass: every value is read once and written once, so the bytes bound it: 2304
// tokens of 32 heads of 256 (fp32 in, bf16 and e4m3 out) take 23 us, 70 % of the copy
// rate; 8 such tokens 2.3 us, which is launch and load latency.
// A block takes one token and some of its heads, a warp one head at a time;
// the token's sines and cosines are computed once per block, the angle
// position * inv_freq in 64 bits (in 32 a position of 2^17 would lose 2^-7 of
// a radian), reduced to a fraction of a turn before it is rounded.
//
// A lane holds two units of D / 64 neighbouring dimensions.  For the planes
// (j, j + rot/2) they are the two units that turn together, so that a rotation
// needs no exchange (through shared memory it was bound by bank conflicts: 72 us
// for 256 x 9 tokens of 32 heads of 256, against 16 for the bytes).
#include <type_traits>

#include "attn.cuh"

namespace vw4 {

constexpr int kAppendWarps = 4;
constexpr int kMaxPairs = 128;

template <int U>
__device__ __forceinline__ void load_unit(const float* p, float* v) {
    if (U == 4) *reinterpret_cast<float4*>(v) = __ldg(reinterpret_cast<const float4*>(p));
    else if (U == 2) *reinterpret_cast<float2*>(v) = __ldg(reinterpret_cast<const float2*>(p));
    else v[0] = __ldg(p);
}
template <int U>
__device__ __forceinline__ void load_unit(const __nv_bfloat16* p, float* v) {
    if (U == 4) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
        v[0] = __uint_as_float(w.x << 16);
        v[1] = __uint_as_float(w.x & 0xffff0000u);
        v[2] = __uint_as_float(w.y << 16);
        v[3] = __uint_as_float(w.y & 0xffff0000u);
    } else if (U == 2) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p));
        v[0] = __uint_as_float(w << 16);
        v[1] = __uint_as_float(w & 0xffff0000u);
    } else {
        v[0] = __bfloat162float(p[0]);
    }
}
template <int U>
__device__ __forceinline__ void store_unit(__nv_bfloat16* p, const float* v) {
    if (U == 4) *reinterpret_cast<uint2*>(p) = make_uint2(pack2<false>(v[0], v[1]), pack2<false>(v[2], v[3]));
    else if (U == 2) *reinterpret_cast<uint32_t*>(p) = pack2<false>(v[0], v[1]);
    else p[0] = __float2bfloat16(v[0]);
}
// nearest, ties to even; beyond 448: 448
template <int U>
__device__ __forceinline__ void store_unit(uint8_t* p, const float* v) {
    if (U == 1) {
        p[0] = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
        return;
    }
    uint32_t w = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
    if (U == 2) {
        *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w);
    } else {
        w |= static_cast<uint32_t>(
                 __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3)) << 16;
        *reinterpret_cast<uint32_t*>(p) = w;
    }
}

template <int D, bool F8, bool XBF16>
__global__ void __launch_bounds__(kAppendWarps * 32) append_kernel(const AppendParams p,
                                                                   int heads_per_block) {
    constexpr int U = D / 64;  // dimensions of a unit; a lane has two
    using X = std::conditional_t<XBF16, __nv_bfloat16, float>;
    using C = std::conditional_t<F8, uint8_t, __nv_bfloat16>;
    __shared__ __align__(16) float s_cos[kMaxPairs], s_sin[kMaxPairs];
    __shared__ __align__(16) float s_head[kAppendWarps][D];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int token = blockIdx.x, b = token / p.R, i = token - b * p.R;
    const int pairs = p.rot / 2;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int heads = p.Hq + 2 * p.Hkv;
    const int h_end = min(heads, (static_cast<int>(blockIdx.y) + 1) * heads_per_block);
    // the lane's units: lanes below P hold a pair of units that turn together, the others
    // two neighbouring units of the rest
    const bool split = pairs > 0 && !p.adjacent && pairs % U == 0;
    const int P = split ? pairs / U : 0;
    const int d0 = (lane < P ? lane : 2 * lane) * U, d1 = lane < P ? d0 + pairs : d0 + U;
    const X* x = static_cast<const X*>(p.x) + static_cast<long long>(token) * p.ldx;
    auto load = [&](int h, float* v) {
        load_unit<U>(x + static_cast<long long>(h) * D + d0, v);
        load_unit<U>(x + static_cast<long long>(h) * D + d1, v + U);
    };
    int h = blockIdx.y * heads_per_block + warp;
    __align__(16) float v[2 * U], nx[2 * U];
    if (h < h_end) load(h, v);  // on its way while the angles are computed
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
    __align__(16) float cs[U], sn[U];  // of the lane's planes
#pragma unroll
    for (int k = 0; k < U; ++k) {
        cs[k] = lane < P ? s_cos[d0 + k] : 1.f;
        sn[k] = lane < P ? s_sin[d0 + k] : 0.f;
    }

    for (; h < h_end; h += kAppendWarps) {
        if (h + kAppendWarps < h_end) load(h + kAppendWarps, nx);
        const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hkv;
        if (is_q || is_k) {
            const float* w = is_q ? p.q_norm : p.k_norm;
            if (w) {
                float ss = 0.f;
#pragma unroll
                for (int k = 0; k < 2 * U; ++k) ss = fmaf(v[k], v[k], ss);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float f = rsqrtf(ss * (1.f / D) + p.eps);
                __align__(16) float g[2 * U];
                load_unit<U>(w + d0, g);
                load_unit<U>(w + d1, g + U);
#pragma unroll
                for (int k = 0; k < 2 * U; ++k) v[k] = v[k] * f * g[k];
            }
            if (split) {
                if (lane < P) {
#pragma unroll
                    for (int k = 0; k < U; ++k) {
                        const float a = v[k], c = v[U + k];
                        v[k] = a * cs[k] - c * sn[k];
                        v[U + k] = c * cs[k] + a * sn[k];
                    }
                }
            } else if (pairs > 0 && p.adjacent) {
                // (the lane's dimensions are 2 U neighbours)
#pragma unroll
                for (int k = 0; k < 2 * U; k += 2) {
                    const int j = (d0 + k) / 2;
                    if (j < pairs) {
                        const float a = v[k], c = v[k + 1];
                        v[k] = a * s_cos[j] - c * s_sin[j];
                        v[k + 1] = c * s_cos[j] + a * s_sin[j];
                    }
                }
            } else if (pairs > 0) {
                // planes that do not fall into whole units
                __syncwarp();  // the last head's reads are done
#pragma unroll
                for (int k = 0; k < 2 * U; ++k) s_head[warp][d0 + k] = v[k];
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 2 * U; ++k) {
                    const int d = d0 + k;
                    if (d < pairs) v[k] = v[k] * s_cos[d] - s_head[warp][d + pairs] * s_sin[d];
                    else if (d < p.rot)
                        v[k] = v[k] * s_cos[d - pairs] + s_head[warp][d - pairs] * s_sin[d - pairs];
                }
            }
        }
        if (is_q) {
            __nv_bfloat16* dst = p.q + static_cast<long long>(token) * p.ldq + static_cast<long long>(h) * D;
            store_unit<U>(dst + d0, v);
            store_unit<U>(dst + d1, v + U);
        } else if (slot >= 0) {
            const int hk = is_k ? h - p.Hq : h - p.Hq - p.Hkv;
            C* dst = static_cast<C*>(is_k ? p.k : p.v) + slot + static_cast<long long>(hk) * p.head_stride;
            if (F8) {
                const float* sp = is_k ? p.k_scale : p.v_scale;
                float sc = sp ? __ldg(sp + hk) : 1.f;
                if (sc == 0.f) sc = INFINITY;  // zeros: what such a head reads back
#pragma unroll
                for (int k = 0; k < 2 * U; ++k) v[k] = __fdiv_rn(v[k], sc);
            }
            store_unit<U>(dst + d0, v);
            store_unit<U>(dst + d1, v + U);
        }
#pragma unroll
        for (int k = 0; k < 2 * U; ++k) v[k] = nx[k];
    }
}

template <int D>
static void (*append_of(bool f8, bool bf16))(const AppendParams, int) {
    if (f8) return bf16 ? append_kernel<D, true, true> : append_kernel<D, true, false>;
    return bf16 ? append_kernel<D, false, true> : append_kernel<D, false, false>;
}

cudaError_t launch_append(const AppendParams& p, bool f8, int sms, cudaStream_t s) {
    const int tokens = p.B * p.R, heads = p.Hq + 2 * p.Hkv;
    // one head a warp while that leaves SMs idle; else more heads share a block's angles
    // (a 64-bit product and a sine and cosine for each of up to 128 planes).  Sixteen
    // blocks an SM: 1800 tokens of 80 heads of 256 take 36.8 us, 42.7 with eight, whose
    // last wave is half empty; 2304 tokens of 32 heads, 128 planes, 23.2 with either, 24.8
    // with 32.
    const int want = 16 * sms;
    int per = static_cast<int>((static_cast<long long>(tokens) * heads + want - 1) / want);
    per = (per + kAppendWarps - 1) / kAppendWarps * kAppendWarps;
    if (per < kAppendWarps) per = kAppendWarps;
    // even blocks: 80 heads as 40 and 40, not 60 and 20
    const int shares = (heads + per - 1) / per;
    per = ((heads + shares - 1) / shares + kAppendWarps - 1) / kAppendWarps * kAppendWarps;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(tokens, (heads + per - 1) / per);
    cfg.blockDim = dim3(kAppendWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const bool bf16 = p.x_bf16 != 0;
    void (*k)(const AppendParams, int) = p.D == 64    ? append_of<64>(f8, bf16)
                                         : p.D == 128 ? append_of<128>(f8, bf16)
                                                      : append_of<256>(f8, bf16);
    return cudaLaunchKernelEx(&cfg, k, p, per);
}

}  // namespace vw4
