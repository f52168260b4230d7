// rope_append.cu -- from the packed qkv rows of the verify GEMM to rotated
// queries and cache entries: per head an optional RMS norm, the rotation of
// its leading dimensions by the token's position, and the rounding to bf16 or
// (for the cache) to e4m3 of value / scale or to nvfp4.
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
__device__ __forceinline__ void put_unit(float* p, const float* v) {  // (p aligned to the unit)
    if (U == 4) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else if (U == 2) *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    else p[0] = v[0];
}
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

// ---------------------------------------------------------------- 4-bit caches
// A head's D values in their order, D / 32 to a lane, so that 512 / D lanes hold the 16
// values of a block.  t = y / g, block scale s = e4m3(max |t| / 6), codes e2m1(t / s).
//
// The codes are to be those of the 64-bit formula, but 64-bit arithmetic has 1/64 of the
// rate of 32-bit.  So 32 bits give t / s and how far it may be off, and both ends of that
// range are rounded: where they agree, so does everything between (rounding is
// monotone).  Where they do not, |y| is compared with border * s * |g|: a fused product
// and sum of 32 bits has the exact sign where y itself is exact; else (about six heads of
// keys in a thousand) y is taken again in 64 bits, the head's norm by the warp, the value
// by its lane.
//
// kValueError bounds the error of a key against |a| + |c| of its plane, or |y| of a value
// that is normed and not turned: the norm's sum of squares 13 roundings of 2^-24,
// halved by the root, rsqrtf two steps, the two factors and the mean one each: 2^-20.2;
// angle, sine and cosine 2^-22.2, products and sum 2^-23: below 2^-19.
constexpr float kValueError = 1.9073486328125e-6f;  // 2^-19
constexpr float kDivError = 2.384185791015625e-7f;  // 2^-22, of a product with a reciprocal

// The norm's factor of a key head in 64 bits (the whole warp; 1 without a norm).
template <int D, class X>
__device__ __noinline__ double kv4_norm(const AppendParams& p, const X* x) {
    if (!p.k_norm) return 1.0;
    double ss = 0.0;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
        const double v = static_cast<double>(static_cast<float>(x[(threadIdx.x & 31) * (D / 32) + k]));
        ss = fma(v, v, ss);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    return rsqrt(ss / D + static_cast<double>(p.eps));
}
// Dimension d of a key in 64 bits.
template <int D, class X>
__device__ __noinline__ double kv4_key(const AppendParams& p, const X* x, int d, double f, int pos) {
    auto at = [&](int k) {
        const double y = static_cast<double>(static_cast<float>(x[k]));
        return p.k_norm ? y * f * static_cast<double>(p.k_norm[k]) : y;
    };
    const double y = at(d);
    if (d >= p.rot) return y;
    const int half = p.rot / 2, j = p.adjacent ? d >> 1 : (d < half ? d : d - half);
    const bool second = p.adjacent ? d & 1 : d >= half;
    const double c = at(p.adjacent ? d ^ 1 : (second ? d - half : d + half));
    double turns = static_cast<double>(pos) * p.inv_freq[j] * 0.15915494309189535, sn, cs;
    turns -= rint(turns);
    sincospi(2.0 * turns, &sn, &cs);
    return second ? y * cs + c * sn : y * cs - c * sn;
}

__device__ __forceinline__ uint32_t e4m3_byte(float v) {
    return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float e4m3_value(uint32_t b) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b), __NV_E4M3)));
}
// two codes, sign and magnitude, and what a magnitude stands for
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
    uint16_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tmov.b16 %0, {t, 0};\n\t}"
        : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float e2m1_value(uint32_t c) {
    return c < 4 ? 0.5f * static_cast<float>(c) : (c & 1 ? 1.5f : 1.f) * (c < 6 ? 2.f : 4.f);
}

// What the quick way below does not take, all of it by quotients: infinities, NaN, heads whose
// squares overflow or vanish, head scales of 0 or so small that their reciprocal or a quotient
// overflows.
// (Codes, block scale) of the lane.
template <int D, class X>
__device__ __noinline__ uint2 kv4_special(const AppendParams& p, const X* x, const float* head,
                                          bool is_k, int pos, float g) {
    constexpr int N = D / 32, GL = 16 / N;
    const int lane = threadIdx.x & 31;
    const double f = is_k ? kv4_norm<D, X>(p, x) : 1.0;
    double t[N], m = 0.0;
    bool nan = false;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int d = lane * N + k;
        const double y = is_k ? kv4_key<D, X>(p, x, d, f, pos) : head[d];
        t[k] = g == 0.f ? (isnan(y) ? y : 0.0) : y / static_cast<double>(g);
        nan |= isnan(t[k]);
        t[k] = fmin(fmax(t[k], -2688.0), 2688.0);
        m = fmax(m, fabs(t[k]));
    }
    unsigned bad = nan;
#pragma unroll
    for (int o = 1; o < GL; o <<= 1) {
        m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
        bad |= __shfl_xor_sync(0xffffffffu, bad, o);
    }
    uint32_t sb = 0u;
    while (sb < 0x7Eu) {
        const double mid = 3.0 * (static_cast<double>(e4m3_value(sb)) + e4m3_value(sb + 1));
        if (m < mid || (m == mid && !(sb & 1u))) break;
        ++sb;
    }
    const double s = e4m3_value(sb);
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        uint32_t c = 0;
        while (sb && c < 7u) {
            const double mid = 0.5 * (static_cast<double>(e2m1_value(c)) + e2m1_value(c + 1)) * s;
            if (fabs(t[k]) < mid || (fabs(t[k]) == mid && !(c & 1u))) break;
            ++c;
        }
        w |= (c | (sb && t[k] < 0.0 ? 8u : 0u)) << (4 * k);
    }
    return make_uint2(w, bad ? 0x7Fu : sb);
}

// The head's values from shared memory to the cache.  offs: what they may be off by (keys), or
// null: exact.  t / s is y times a product of reciprocals: off by less than 2^-21 of itself.
template <int D, class X>
__device__ __forceinline__ void store_kv4(const AppendParams& p, const X* x, const float* head,
                                          const float* offs, bool is_k, int hk, int pos,
                                          long long at, long long bat, int lane) {
    constexpr int N = D / 32, GL = 16 / N;  // values of a lane, lanes of a block
    const float* sp = is_k ? p.k_scale : p.v_scale;
    const float g = sp ? __ldg(sp + hk) : 1.f;
    const float rg = __fdiv_rn(1.f, g), ag = fabsf(g), ar = fabsf(rg);
    __align__(16) float y[N], of[N];
#pragma unroll
    for (int k = 0; k < N; k += 2) {
        *reinterpret_cast<float2*>(y + k) = *reinterpret_cast<const float2*>(head + lane * N + k);
        *reinterpret_cast<float2*>(of + k) =
            offs ? *reinterpret_cast<const float2*>(offs + lane * N + k) : make_float2(0.f, 0.f);
    }
    uint32_t largest = 0u;  // bits of the largest magnitude: a NaN's are above all
    float off = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        largest = max(largest, __float_as_uint(y[k]) & 0x7fffffffu);
        off = fmaxf(off, of[k]);
    }
#pragma unroll
    for (int o = 1; o < GL; o <<= 1) {
        largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, o));
        if (offs) off = fmaxf(off, __shfl_xor_sync(0xffffffffu, off, o));
    }
    const float m = __uint_as_float(largest);
    uint32_t w = 0, sb;
    // (quotients as well: what follows has no room for an infinity)
    if (__any_sync(0xffffffffu, !(ar > 1e-30f && ar < 1e30f && m + off < 1e30f && (m + off) * ar < 1e30f))) {
        const uint2 r = kv4_special<D, X>(p, x, head, is_k, pos, g);
        w = r.x;
        sb = r.y;
    } else {
        const float e = fmaf(off, ar, m * ar * kDivError);
        // (the bound may be above the block's values: those of a key's partners go into it)
        sb = e4m3_byte(fmaxf(0.f, m * ar - e) * (1.f / 6.f) * (1.f - kDivError));
        const uint32_t sb1 = e4m3_byte((m * ar + e) * (1.f / 6.f) * (1.f + kDivError));
        double f = 0.0;
        bool have_f = false;
        if (__any_sync(0xffffffffu, sb != sb1)) {
            double top = m;
            if (offs) {
                f = kv4_norm<D, X>(p, x);
                have_f = true;
                top = 0.0;
#pragma unroll 1
                for (int k = 0; k < N; ++k) {
                    const float v = head[lane * N + k];
                    if (sb != sb1 && fabsf(v) + 2.f * off >= m)
                        top = fmax(top, fabs(kv4_key<D, X>(p, x, lane * N + k, f, pos)));
                }
#pragma unroll
                for (int o = 1; o < GL; o <<= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
            }
            while (sb < sb1) {
                const double mid = 3.0 * (static_cast<double>(e4m3_value(sb)) + e4m3_value(sb + 1)) * ag;
                if (top < mid || (top == mid && !(sb & 1u))) break;
                ++sb;
            }
        }
        const float s = e4m3_value(sb), rs = sb ? __frcp_rn(s) : 0.f, c1 = rg * rs, c2 = ar * rs;
        uint32_t unsure = 0;
#pragma unroll
        for (int k = 0; k < N; k += 2) {
            float q[2], d[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                q[j] = y[k + j] * c1;
                d[j] = fmaf(of[k + j], c2, fabsf(q[j]) * (2.f * kDivError));
            }
            const uint32_t a = e2m1_pair(q[0] - d[0], q[1] - d[1]);
            const uint32_t c = e2m1_pair(q[0] + d[0], q[1] + d[1]);
            unsure |= (a ^ c) << (4 * k);
            w |= a << (4 * k);
        }
        if (sb == 0u) w = unsure = 0u;
        if (__any_sync(0xffffffffu, unsure != 0u)) {
            if (offs && !have_f) f = kv4_norm<D, X>(p, x);
#pragma unroll 1
            for (int k = 0; k < N; ++k) {
                if (((unsure >> (4 * k)) & 15u) == 0u) continue;
                // the codes that the range reaches, from the least magnitude on
                const float v = head[lane * N + k], mag = fabsf(v), o = offs ? offs[lane * N + k] : 0.f;
                const double v64 = offs ? kv4_key<D, X>(p, x, lane * N + k, f, pos) : 0.0;
                const float least = mag * c2 - fmaf(o, c2, mag * c2 * (2.f * kDivError));
                uint32_t c = least > 0.f ? e2m1_pair(least, 0.f) & 7u : 0u;
                while (sb && c < 7u) {
                    const float mid = 0.5f * (e2m1_value(c) + e2m1_value(c + 1)) * s;  // few bits
                    const bool low = offs ? fabs(v64) < static_cast<double>(mid) * ag : fmaf(mid, ag, -mag) > 0.f;
                    const bool tie = offs ? fabs(v64) == static_cast<double>(mid) * ag : fmaf(mid, ag, -mag) == 0.f;
                    if (low || (tie && !(c & 1u))) break;
                    ++c;
                }
                // (a zero has no sign)
                const bool minus = offs ? v64 != 0.0 && (v64 < 0.0) != (g < 0.f)
                                        : v != 0.f && (v < 0.f) != (g < 0.f);
                w = (w & ~(15u << (4 * k))) | (c | (minus ? 8u : 0u)) << (4 * k);
            }
        }
    }
    uint8_t* dst = static_cast<uint8_t*>(is_k ? p.k : p.v) + at + lane * (N / 2);
    if (N == 8) *reinterpret_cast<uint32_t*>(dst) = w;
    else if (N == 4) *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(w);
    else *dst = static_cast<uint8_t>(w);
    uint8_t* bl = is_k ? p.k_blocks : p.v_blocks;
    if (lane % GL == 0) bl[bat + lane / GL] = static_cast<uint8_t>(sb);
}

// A block's heads, from first on: any (kHeadsAny), queries, or keys and values.
constexpr int kHeadsAny = 0, kHeadsQ = 1, kHeadsKv = 2;

// AHEAD: how many heads of a warp are on their way while one is turned.
template <int D, int KIND, bool XBF16, int PART, int AHEAD>
__device__ __forceinline__ void append_block(const AppendParams& p, int first, int heads_per_block) {
    constexpr bool F8 = KIND == kCacheE4m3, KV4 = KIND == kCacheKv4;
    constexpr int U = D / 64;  // dimensions of a unit; a lane has two
    using X = std::conditional_t<XBF16, __nv_bfloat16, float>;
    using C = std::conditional_t<KIND == kCacheBf16, __nv_bfloat16, uint8_t>;
    __shared__ __align__(16) float s_cos[kMaxPairs], s_sin[kMaxPairs];
    __shared__ __align__(16) float s_head[kAppendWarps][D];
    constexpr bool OFF = KV4 && PART != kHeadsQ;
    __shared__ __align__(16) float s_off[OFF ? kAppendWarps : 1][OFF ? D : 1];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int token = blockIdx.x, b = token / p.R, i = token - b * p.R;
    const int pairs = p.rot / 2;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int heads = PART == kHeadsQ ? p.Hq : p.Hq + 2 * p.Hkv;
    const int h_end = min(heads, first + heads_per_block);
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
    int h = first + warp;
    __align__(16) float v[2 * U], nx[AHEAD][2 * U];
    if (h < h_end) load(h, v);  // on its way while the angles are computed
#pragma unroll
    for (int q = 0; q + 1 < AHEAD; ++q)
        if (h + (q + 1) * kAppendWarps < h_end) load(h + (q + 1) * kAppendWarps, nx[q]);
    const int pos = p.seq_lens[b] - p.R + i;
    for (int j = threadIdx.x; j < pairs; j += kAppendWarps * 32) {
        double turns = static_cast<double>(pos) * p.inv_freq[j] * 0.15915494309189535;
        turns -= rint(turns);
        sincospif(static_cast<float>(2.0 * turns), &s_sin[j], &s_cos[j]);
    }
    // the token's cache slot
    long long slot = -1, bslot = 0;
    if (PART != kHeadsQ && pos >= 0) {
        const int blk = pos >> p.page_shift;
        const int pg = blk < p.max_blocks
                           ? __ldg(p.table + static_cast<long long>(b) * p.table_stride + blk)
                           : -1;
        if (pg >= 0 && pg < p.num_pages) {
            slot = static_cast<long long>(pg) * p.page_stride +
                   static_cast<long long>(pos & (p.page_size - 1)) * p.token_stride;
            if (KV4)
                bslot = static_cast<long long>(pg) * p.blocks_page_stride +
                        static_cast<long long>(pos & (p.page_size - 1)) * (D / 16);
        } else if (threadIdx.x == 0)
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
        if (h + AHEAD * kAppendWarps < h_end) load(h + AHEAD * kAppendWarps, nx[AHEAD - 1]);
        const bool is_q = PART == kHeadsQ || (PART == kHeadsAny && h < p.Hq);
        const bool is_k = !is_q && h < p.Hq + p.Hkv;
        float off[KV4 ? 2 * U : 1];  // 4-bit keys: what a value may be off by
        bool wide = false;           // and whether 32 bits say nothing of it
        if (KV4) {
#pragma unroll
            for (int k = 0; k < 2 * U; ++k) off[KV4 ? k : 0] = 0.f;
        }
        if (is_q || is_k) {
            const float* w = is_q ? p.q_norm : p.k_norm;
            if (w) {
                float ss = 0.f;
#pragma unroll
                for (int k = 0; k < 2 * U; ++k) ss = fmaf(v[k], v[k], ss);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float mean = ss * (1.f / D) + p.eps, f = rsqrtf(mean);
                __align__(16) float g[2 * U];
                load_unit<U>(w + d0, g);
                load_unit<U>(w + d1, g + U);
#pragma unroll
                for (int k = 0; k < 2 * U; ++k) v[k] = v[k] * f * g[k];
                if (KV4 && is_k) {
#pragma unroll
                    for (int k = 0; k < 2 * U; ++k) off[KV4 ? k : 0] = fabsf(v[k]);
                    // squares that leave the range of 32 bits: the head is taken in 64
                    wide = !(mean > 1e-30f && mean < 1e30f);
                }
            }
            if (split) {
                if (lane < P) {
#pragma unroll
                    for (int k = 0; k < U; ++k) {
                        const float a = v[k], c = v[U + k];
                        if (KV4) off[KV4 ? k : 0] = off[KV4 ? U + k : 0] = fabsf(a) + fabsf(c);
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
                        if (KV4) off[KV4 ? k : 0] = off[KV4 ? k + 1 : 0] = fabsf(a) + fabsf(c);
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
                    if (KV4 && d < p.rot)
                        off[KV4 ? k : 0] =
                            fabsf(v[k]) + fabsf(s_head[warp][d < pairs ? d + pairs : d - pairs]);
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
        } else if (KV4 && PART != kHeadsQ) {
            if (slot >= 0) {  // (the same for the warp)
                __syncwarp();  // the last head's reads are done
                float* offs = s_off[OFF ? warp : 0];
#pragma unroll
                for (int k = 0; k < 2 * U; ++k) off[KV4 ? k : 0] = wide ? INFINITY : off[KV4 ? k : 0] * kValueError;
                put_unit<U>(s_head[warp] + d0, v);
                put_unit<U>(s_head[warp] + d1, v + U);
                if (is_k) {
                    put_unit<U>(offs + d0, off);
                    put_unit<U>(offs + d1, off + (KV4 ? U : 0));
                }
                __syncwarp();
                const int hk = is_k ? h - p.Hq : h - p.Hq - p.Hkv;
                store_kv4<D, X>(p, x + static_cast<long long>(h) * D, s_head[warp],
                                is_k && (p.k_norm || p.rot > 0) ? offs : nullptr, is_k, hk, pos,
                                slot + static_cast<long long>(hk) * p.head_stride,
                                bslot + static_cast<long long>(hk) * p.blocks_head_stride, lane);
            }
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
        for (int k = 0; k < 2 * U; ++k) {
            v[k] = nx[0][k];
#pragma unroll
            for (int q = 0; q + 1 < AHEAD; ++q) nx[q][k] = nx[q + 1][k];
        }
    }
}

template <int D, int KIND, bool XBF16>
__global__ void __launch_bounds__(kAppendWarps * 32) append_kernel(const AppendParams p,
                                                                   int heads_per_block) {
    append_block<D, KIND, XBF16, kHeadsAny, 1>(p, blockIdx.y * heads_per_block, heads_per_block);
}
// Queries and the others in blocks of their own: the registers that rounding to 4 bits takes
// would be spilled in the queries' loop (2304 tokens of 32 heads of 256, with the rows read
// back: 54 us together, 40 apart).  Keys and values first: a head that is done again has the
// queries to hide behind (47 us last).  Alone the kernel takes 31 us of fp32 rows (15.7 at the copy
// rate) and 32 of bf16 (10.1), 28 and 29 without a rotation: both blocks of a token compute its
// angles.  No unit is above 59 % (issue slots); its warps wait for rows and for shared memory.
template <int D, bool XBF16>
__global__ void __launch_bounds__(kAppendWarps * 32, 7) append_kv4_kernel(const AppendParams p,
                                                                          int heads_per_block) {
    const int kv_blocks = (2 * p.Hkv + heads_per_block - 1) / heads_per_block, y = blockIdx.y;
    if (y < kv_blocks)
        append_block<D, kCacheKv4, XBF16, kHeadsKv, 1>(p, p.Hq + y * heads_per_block, heads_per_block);
    else
        append_block<D, kCacheKv4, XBF16, kHeadsQ, 2>(p, (y - kv_blocks) * heads_per_block, heads_per_block);
}

template <int D>
static void (*append_of(int kind, bool bf16))(const AppendParams, int) {
    if (kind == kCacheKv4)
        return bf16 ? append_kv4_kernel<D, true> : append_kv4_kernel<D, false>;
    if (kind == kCacheE4m3)
        return bf16 ? append_kernel<D, kCacheE4m3, true> : append_kernel<D, kCacheE4m3, false>;
    return bf16 ? append_kernel<D, kCacheBf16, true> : append_kernel<D, kCacheBf16, false>;
}

cudaError_t launch_append(const AppendParams& p, int kind, int sms, cudaStream_t s) {
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
    cfg.gridDim = dim3(tokens, kind == kCacheKv4 ? (p.Hq + per - 1) / per + (2 * p.Hkv + per - 1) / per
                                                 : (heads + per - 1) / per);
    cfg.blockDim = dim3(kAppendWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const bool bf16 = p.x_bf16 != 0;
    void (*k)(const AppendParams, int) = p.D == 64    ? append_of<64>(kind, bf16)
                                         : p.D == 128 ? append_of<128>(kind, bf16)
                                                      : append_of<256>(kind, bf16);
    return cudaLaunchKernelEx(&cfg, k, p, per);
}

}  // namespace vw4
