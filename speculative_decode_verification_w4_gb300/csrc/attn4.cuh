// attn4.cuh -- attention of the verify rows over a paged cache in 4 bits (nvfp4), as a
// template over the head size and the number of query rows, instantiated per head size in
// attn4_d*.cu.  The work schedule, the page loads and the join of split items are those of
// the other cache types (attn.cuh).
//
// Mathematics.  S = Q K^T, P = exp(S - max), O = P V with a running maximum and sum over
// tiles of 128 keys, all transposed: keys, then dimensions are the rows of the matrix
// instructions and the query rows their columns, eight to an instruction, so that the
// converted cache values are the operand that is made once and the query rows cost little
// where they are few.  K^T and V become f16 in registers, exactly: e2m1 times its block's
// e4m3 scale has six significant bits.
//
// A tile.  Each of eight warps takes 16 keys for S = K Q^T (32 dimensions of 8 keys are a
// register of codes a lane), forms P against the block's common reference, and leaves it in
// shared memory; beside it, the warps leave V's scales as f16, token by token.  After the
// barrier each warp takes 32 dimensions of V for O = V^T P^T (of all keys at head size 256,
// of a half or a quarter below), so nothing is converted twice however many query rows there
// are, and S of the next tile runs in the same phase: one barrier a tile.
//
// The reference that the weights use is the running maximum, followed lazily: only where a
// score exceeds it by 2^5 do the warps meet for the true maximum, rescale and form P again
// (the first tile of an item; rarely later).  Weights are at most 2^14 in f16, and reach
// down to 2^-33 of the largest (f16 ends at 2^-24).
#pragma once
#include "attn.cuh"

namespace vw4 {

constexpr float kTail4 = 9.f;     // weights carry 2^9
constexpr float kLazy4 = 5.f;     // (log2) of the reference
constexpr int kAttn4Tk = 128;

#ifdef __CUDACC__
template <int D, int NT>
struct Attn4Shape {
    static constexpr int kWarps = 8;
    static constexpr int kThreads = (kWarps + 2) * 32;
    static constexpr int kTK = kAttn4Tk;
    static constexpr int kRows = 8 * NT;
    static constexpr int kKB = D / 2;                 // bytes of a key's codes
    static constexpr int kNB = D / 16;                // and of its scales
    static constexpr int kTile = kTK * kKB;
    static constexpr int kSTile = kTK * kNB;
    static constexpr int kStage = 2 * kTile + 2 * kSTile;  // K, V, scales of K, of V
    static constexpr int kSlices = D / 32;            // slices of V's dimensions
    static constexpr int kParts = kWarps / kSlices;   // parts of its keys
    static constexpr int kQ = kRows * D * 2;
    static constexpr int kQBlk = kRows * 128;
    static constexpr int kP = NT * kTK * 16;          // weights: f16 [n-tile][key][8]
    static constexpr int kVRow = (kTK + 16) * 2;      // V's scales: f16 [block][token]
    static constexpr int kVS = kNB * kVRow;
    static constexpr int kX = (kParts - 1) * kSlices * 1024;  // an n-tile's outputs of the other parts
    static constexpr int kStages = D == 64 ? 6 : (D == 128 ? 4 : (NT <= 2 ? 2 : 3));
    static constexpr int kOffQ = kStages * kStage;
    static constexpr int kOffP = kOffQ + 2 * kQ;
    static constexpr int kOffV = kOffP + 2 * kP;
    static constexpr int kOffX = kOffV + 2 * kVS;
    static constexpr int kOffML = kOffX + kX;          // float [2][warps][rows]: maxima, sums
    static constexpr int kOffRow = kOffML + 2 * kWarps * kRows * 4;  // [4][rows], see below
    static constexpr int kSmem = kOffRow + 4 * kRows * 4 + 1024;
    static_assert(kStage % 1024 == 0 && kQ % 1024 == 0 && kVS % 16 == 0, "alignment");
    static_assert(kSmem <= 225 * 1024, "shared memory");
    __device__ static __forceinline__ uint32_t at(int key, int chunk) {  // 16 bytes of a key's codes
        const int x = kKB == 128 ? key & 7 : (kKB == 64 ? (key >> 1) & 3 : (key >> 2) & 1);
        return static_cast<uint32_t>(key * kKB + ((chunk ^ x) << 4));
    }
    __device__ static __forceinline__ uint32_t q_at(int row, int chunk) {  // 16 bytes of a query
        return static_cast<uint32_t>((chunk >> 3) * kQBlk + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
    }
};

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <int D, int NT, int MINB>
__global__ void __launch_bounds__(Attn4Shape<D, NT>::kThreads, MINB)
    attn4_kernel(const AttnParams p, const Kv4Blocks kb, const __grid_constant__ AttnMaps maps) {
    using S = Attn4Shape<D, NT>;
    constexpr int TK = S::kTK, NST = S::kStages, NB = S::kNB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ __align__(8) uint64_t b_full[NST], b_empty[NST], b_qe[2];
    __shared__ AttnUnit s_unit[kUnitRing];
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, lane = tid & 31, wk = tid >> 5;
    const uint32_t sm = smem_u32(smem);
    float* s_m = reinterpret_cast<float*>(smem + S::kOffML);
    float* s_l = s_m + S::kWarps * S::kRows;
    float* s_rs = reinterpret_cast<float*>(smem + S::kOffRow);      // a query row's scale
    int* s_pos = reinterpret_cast<int*>(s_rs + S::kRows);           // its position (dead: -1)
    int* s_out = s_pos + S::kRows;                                  // verify index << 16 | head (dead: -1)
    uint32_t* s_nan = reinterpret_cast<uint32_t*>(s_out + S::kRows);  // its blocks that a NaN reached

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == S::kWarps * 32) {
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
        tma_prefetch_desc(&maps.q);
    }
    if (tid == 0) {
        for (int k = 0; k < NST; ++k) {
            mbar_init(&b_full[k], 2);
            mbar_init(&b_empty[k], 1);
        }
        mbar_init(&b_qe[0], 1);
        mbar_init(&b_qe[1], 1);
        fence_barrier_init();
        s_abort = 0;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int cap = p.max_blocks * p.page_size;
    const AttnSpan span = attn_span<S::kThreads>(p, cap, TK);
    const int n_units = static_cast<int>(span.u1 - span.u0);
    if (n_units == 0) return;
    auto wait = [&](uint64_t* bar, int phase) {  // the same answer in every lane
        const bool ok = mbar_wait_bounded(bar, phase & 1, p.wait_ns, &s_abort);
        if (!ok) {
            s_abort = 1;
            atomicOr(p.status, kStatusWaitTimeout);
        }
        return __all_sync(0xffffffffu, ok) != 0;
    };

    if (wk >= S::kWarps) {
        // ------------------------------------------------------- producers
        const bool keys = wk == S::kWarps;  // else values
        const uint8_t* blocks = keys ? kb.k : kb.v;
        const uint64_t policy = policy_evict_normal();
        AttnWalk<TK> w;
        w.begin(p, span, cap, lane);
        int u = 0;
        for (; u < n_units; ++u) {
            const int st = u % NST;
            const AttnUnit d = w.unit(p);
            const AttnTile t = w.tile(p);
            if (u + 1 < n_units) w.next(p, lane);
            if (u >= NST && !wait(&b_empty[st], u / NST - 1)) break;
            const bool q = keys && (d.flags & kUnitFirst);
            if (q && d.seg >= 2 && !wait(&b_qe[d.seg & 1], (d.seg >> 1) - 1)) break;
            const uint32_t box = static_cast<uint32_t>(t.box_rows * NB);  // bytes of a box's scales
            uint8_t* sdst = smem + st * S::kStage + 2 * S::kTile + (keys ? 0 : S::kSTile) + lane * box;
            const bool there = t.page >= 0 && t.page < p.num_pages;
            if (t.page == p.num_pages) {  // no such page: zeros
                for (uint32_t c = 0; c < box; c += 16)
                    *reinterpret_cast<uint4*>(sdst + c) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
            }
            const uint32_t bytes = t.template bytes<TK, 1, S::kKB>(0, lane) +
                                   __popc(__ballot_sync(0xffffffffu, there)) * box;
            __syncwarp();
            if (lane == 0) {
                if (keys) s_unit[u % kUnitRing] = d;
                mbar_arrive_expect_tx(&b_full[st], bytes + (q ? attn_q_bytes(p, D) : 0u));
                if (q)
                    attn_load_q<D>(p, &maps.q, sm + S::kOffQ + (d.seg & 1) * S::kQ, S::kQBlk, d,
                                   &b_full[st]);
            }
            __syncwarp();
            t.template load<TK, 1, 1, S::kKB, 1>(p, keys ? &maps.k : &maps.v,
                                                 sm + st * S::kStage + (keys ? 0 : S::kTile),
                                                 &b_full[st], 0, 0, lane);
            if (there)
                bulk_load(sdst, blocks + t.page * kb.page_stride + t.h * kb.head_stride +
                                    static_cast<long long>((t.start + lane * t.box_rows) &
                                                           (p.page_size - 1)) * NB,
                          box, &b_full[st], policy);
            __syncwarp();
        }
        // copies in flight land before the block ends
        if (u < n_units) {
            for (int k = u > NST ? u - NST : 0; k < u; ++k)
                mbar_wait_bounded(&b_full[k % NST], (k / NST) & 1, p.wait_ns, nullptr);
        }
        return;
    }

    // ---- the eight warps.  Every path between two meetings has the same number of them in
    // all warps: a wait that ran out makes a warp skip its work, and the next meeting ends
    // the block's.
    bool dead = false;
    auto meet = [&](bool flag) {  // the threads of the eight warps; any of the flags
        uint32_t r;
        asm volatile(
            "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\t"
            "barrier.cta.red.or.pred b, 1, 256, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
            : "=r"(r) : "r"(static_cast<uint32_t>(flag)) : "memory");
        return r != 0;
    };
    float o[2][NT][4];       // rows: dimensions 4 u + 2 i, + 1 of the slice; columns: query rows
    float l[NT][2], ref[NT][2], c2[NT][2];
    const int t4 = lane & 3, u8 = lane >> 2, lm = lane >> 3, lr = lane & 7;
    const int key0 = wk * 16;                          // of the warp's keys
    const int slice = wk % S::kSlices, part = wk / S::kSlices;
    const int blk = 2 * slice + (lane >> 4);           // scale block of the lane's dimensions

    // O += V^T P^T of unit u
    auto values = [&](int u) {
        const uint32_t vS = sm + (u % NST) * S::kStage + S::kTile;
        const uint32_t pS = sm + S::kOffP + (u & 1) * S::kP;
        const uint8_t* sc = smem + S::kOffV + (u & 1) * S::kVS + blk * S::kVRow;
#pragma unroll
        for (int k = 0; k < TK / S::kParts; k += 32) {
            const int key = part * (TK / S::kParts) + k;
            uint32_t x[4], e[4][4];
            ldsm4t(x, vS + S::at(key + lr + 8 * lm, slice));
            // a register: two tokens x four dimensions; to pairs of tokens, scaled
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const uint32_t s = *reinterpret_cast<const uint32_t*>(sc + (key + 8 * m + 2 * t4) * 2);
                uint32_t h[4];
                e2m1x8_f16(x[m], h);
                e[m][0] = mul_f16x2(__byte_perm(h[0], h[2], 0x5410), s);
                e[m][1] = mul_f16x2(__byte_perm(h[0], h[2], 0x7632), s);
                e[m][2] = mul_f16x2(__byte_perm(h[1], h[3], 0x5410), s);
                e[m][3] = mul_f16x2(__byte_perm(h[1], h[3], 0x7632), s);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint32_t b[4];
                ldsm4t(b, pS + n * (TK * 16) + (key + lr + 8 * lm) * 16);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t a[4] = {e[2 * h][2 * i], e[2 * h][2 * i + 1],
                                               e[2 * h + 1][2 * i], e[2 * h + 1][2 * i + 1]};
                        mma16816<true>(o[i][n], a, b[2 * h], b[2 * h + 1]);
                    }
            }
        }
    };

    for (int u = 0; u < n_units; ++u) {
        // ---- a part of an item: its queries
        dead |= !wait(&b_full[u % NST], u / NST);
        AttnUnit td = s_unit[u % kUnitRing];
        const int qslot = td.seg & 1;
        const uint32_t qs = sm + S::kOffQ + qslot * S::kQ;
        const int h = td.g / p.row_blocks;
        float ks = 1.f, vs = 1.f;
        if (!dead) {
            ks = p.k_scale ? __ldg(p.k_scale + h) : 1.f;
            vs = p.v_scale ? __ldg(p.v_scale + h) : 1.f;
            // bf16 -> f16 under a power of two per row that puts its largest magnitude into
            // [2^14, 2^15), with the sign of the head's scale: exact for every value down to
            // 2^-31 of it.  Within 32 dimensions the order is that of the codes' registers.
            for (int r = wk; r < S::kRows; r += S::kWarps) {
                const AttnRow ar = attn_row(p, td.g, r);
                uint32_t* row = reinterpret_cast<uint32_t*>(smem + S::kOffQ + qslot * S::kQ);
                float v[D / 32];
                float mx = 0.f;
#pragma unroll
                for (int k = 0; k < D / 64; ++k) {
                    const int e = lane + 32 * k;  // pair of dimensions 2e, 2e + 1
                    const uint32_t x = ar.live ? row[(S::q_at(r, e >> 2) >> 2) + (e & 3)] : 0u;
                    v[2 * k] = __uint_as_float(x << 16);
                    v[2 * k + 1] = __uint_as_float(x & 0xffff0000u);
                    mx = fmaxf(mx, fmaxf(fabsf(v[2 * k]), fabsf(v[2 * k + 1])));
                }
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
                const int ex = static_cast<int>(__float_as_uint(mx) >> 23);
                int sh = ex == 0 || ex == 255 ? 0 : 127 + 14 - ex;
                sh = max(-126, min(126, sh));
                const float up = copysignf(__uint_as_float(static_cast<uint32_t>(127 + sh) << 23), ks);
                if (lane == 0) {
                    s_rs[r] = __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
                    s_pos[r] = ar.live ? td.p0 + ar.i : -1;
                    s_out[r] = ar.live ? ar.i << 16 | ar.hq : -1;
                    s_nan[r] = 0u;
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < D / 64; ++k) {
                    const int e = lane + 32 * k, s = (e & ~15) | ((e & 3) << 2) | ((e >> 2) & 3);
                    row[(S::q_at(r, s >> 2) >> 2) + (s & 3)] = pack2<true>(v[2 * k] * up, v[2 * k + 1] * up);
                }
            }
            fence_async_smem();  // (a later load will write there)
        }
        if (meet(dead)) return;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                l[n][k] = 0.f;
                ref[n][k] = -INFINITY;
                c2[n][k] = p.scale * kLog2e * fabsf(ks) * s_rs[n * 8 + t4 * 2 + k];
                if (c2[n][k] < kMinFactor) c2[n][k] = kMinFactor;  // (NaN stays)
                o[0][n][2 * k] = o[0][n][2 * k + 1] = o[1][n][2 * k] = o[1][n][2 * k + 1] = 0.f;
            }
        }
        for (const int first = u;; ++u) {
            if (u > first) {
                dead |= !wait(&b_full[u % NST], u / NST);
                if (!dead) td = s_unit[u % kUnitRing];
            }
            const bool edge = td.flags & kUnitEdge;
            uint8_t* stage = smem + (u % NST) * S::kStage;
            float s[NT][4];
            float sum[NT][2];
            // weights against the reference, to shared memory; true where a score is too far
            // above it
            auto weights = [&] {
                bool grew = false;
                uint8_t* dst = smem + S::kOffP + (u & 1) * S::kP + (key0 + u8) * 16 + t4 * 4;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float w[4];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float r = ref[n][k] == -INFINITY ? 0.f : ref[n][k];
                        grew |= fmaxf(s[n][k], s[n][k + 2]) * c2[n][k] > ref[n][k] + kLazy4;
                        w[k] = ex2(fmaf(s[n][k], c2[n][k], kTail4 - r));
                        w[k + 2] = ex2(fmaf(s[n][k + 2], c2[n][k], kTail4 - r));
                        sum[n][k] = w[k] + w[k + 2];
                    }
                    *reinterpret_cast<uint32_t*>(dst + n * (TK * 16)) = pack2<true>(w[0], w[1]);
                    *reinterpret_cast<uint32_t*>(dst + n * (TK * 16) + 128) = pack2<true>(w[2], w[3]);
                }
                return grew;
            };
            bool grew = false;
            if (!dead) {
                // ---- V's scales to f16, token by token
                {
                    constexpr int PER = NB / 2;  // bytes of a thread
                    const int token = tid >> 1, b0 = (tid & 1) * PER;
                    const uint8_t* src = stage + 2 * S::kTile + S::kSTile + token * NB + b0;
                    uint32_t w[PER > 4 ? 2 : 1];
                    if (PER == 2) w[0] = *reinterpret_cast<const uint16_t*>(src);
                    else if (PER == 4) w[0] = *reinterpret_cast<const uint32_t*>(src);
                    else {
                        w[0] = *reinterpret_cast<const uint32_t*>(src);
                        w[PER > 4 ? 1 : 0] = *reinterpret_cast<const uint32_t*>(src + 4);
                    }
                    if (edge) {
                        const int j = td.start + token;
                        if (!key_some(j, td.len, td.p0, p.window, p.sinks)) {
                            // no row sees it: zeros, whatever the cache holds there
#pragma unroll
                            for (int k = 0; k < (PER > 4 ? 2 : 1); ++k) w[k] = 0u;
                        } else if (!key_all(j, td.len, td.p0, p.window, p.sinks)) {
                            // NaN scales must not reach rows that do not see the key through a
                            // weight of zero: noted for the others, and taken out
#pragma unroll 1
                            for (int k = 0; k < PER; ++k) {
                                uint32_t& wk4 = w[PER > 4 && k >= 4 ? 1 : 0];
                                const int at = 8 * (k & 3);
                                if (((wk4 >> at) & 0x7fu) != 0x7fu) continue;
                                wk4 &= ~(0xffu << at);
#pragma unroll 1
                                for (int r = 0; r < S::kRows; ++r)
                                    if (s_out[r] >= 0 && key_seen(j, s_pos[r], p.window, p.sinks))
                                        atomicOr(&s_nan[r], 1u << (b0 + k));
                            }
                        }
                    }
                    uint8_t* dst = smem + S::kOffV + (u & 1) * S::kVS + b0 * S::kVRow + token * 2;
#pragma unroll
                    for (int k = 0; k < PER; k += 2) {
                        const uint32_t f = e4m3x2_f16x2(w[k / 4] >> (8 * (k & 3)));
                        *reinterpret_cast<uint16_t*>(dst + k * S::kVRow) = static_cast<uint16_t>(f);
                        *reinterpret_cast<uint16_t*>(dst + (k + 1) * S::kVRow) =
                            static_cast<uint16_t>(f >> 16);
                    }
                }
                // ---- S = K Q^T of the warp's keys
                const uint32_t kS = sm + (u % NST) * S::kStage;
                uint32_t sk[2][D / 64];  // scales of two 32-dimension chunks, of keys u8 and u8 + 8
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint8_t* src = stage + 2 * S::kTile + (key0 + u8 + 8 * k) * NB;
                    const uint32_t sel = t4 & 2 ? 0x7531u : 0x6420u;
                    if constexpr (NB == 4) {
                        sk[k][0] = e4m3x2_f16x2(
                            __byte_perm(*reinterpret_cast<const uint32_t*>(src), 0, sel & 0x3333u));
                    } else if constexpr (NB == 8) {
                        const uint2 w = *reinterpret_cast<const uint2*>(src);
                        const uint32_t b = __byte_perm(w.x, w.y, sel);
                        sk[k][0] = e4m3x2_f16x2(b);
                        sk[k][1] = e4m3x2_f16x2(b >> 16);
                    } else {
                        const uint4 w = *reinterpret_cast<const uint4*>(src);
                        const uint32_t b = __byte_perm(w.x, w.y, sel), c = __byte_perm(w.z, w.w, sel);
                        sk[k][0] = e4m3x2_f16x2(b);
                        sk[k][1] = e4m3x2_f16x2(b >> 16);
                        sk[k][2] = e4m3x2_f16x2(c);
                        sk[k][3] = e4m3x2_f16x2(c >> 16);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
                for (int c = 0; c < D / 32; c += 2) {
                    uint32_t w[4];
                    ldsm4(w, kS + S::at(key0 + lr + (lm & 1) * 8, c + (lm >> 1)));
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t x[4], y[4];
                        e2m1x8_f16(w[2 * e], x);
                        e2m1x8_f16(w[2 * e + 1], y);
                        const uint32_t sx = __byte_perm(sk[0][c / 2], 0, e ? 0x3232 : 0x1010);
                        const uint32_t sy = __byte_perm(sk[1][c / 2], 0, e ? 0x3232 : 0x1010);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            x[k] = mul_f16x2(x[k], sx);
                            y[k] = mul_f16x2(y[k], sy);
                        }
                        const uint32_t a0[4] = {x[0], y[0], x[1], y[1]}, a1[4] = {x[2], y[2], x[3], y[3]};
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            uint32_t b[4];
                            ldsm4(b, qs + S::q_at(n * 8 + lr, (c + e) * 4 + lm));
                            mma16816<true>(s[n], a0, b[0], b[1]);
                            mma16816<true>(s[n], a1, b[2], b[3]);
                        }
                    }
                }
                if (edge) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int pos = s_pos[n * 8 + t4 * 2 + k], j = td.start + key0 + u8;
                            if (!key_seen(j, pos, p.window, p.sinks)) s[n][k] = -INFINITY;
                            if (!key_seen(j + 8, pos, p.window, p.sinks)) s[n][k + 2] = -INFINITY;
                        }
                }
                grew = weights();
                if (u > first) values(u - 1);
            }
            if (meet(grew || dead)) {
                if (meet(dead)) return;
                // ---- the true maximum of the rows, and the weights again
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float mx = fmaxf(s[n][k], s[n][k + 2]);
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1)
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                        if (lane < 4) s_m[wk * S::kRows + n * 8 + t4 * 2 + k] = mx * c2[n][k];
                    }
                meet(false);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float mx = ref[n][k];
#pragma unroll
                        for (int w = 0; w < S::kWarps; ++w)
                            mx = fmaxf(mx, s_m[w * S::kRows + n * 8 + t4 * 2 + k]);
                        const float f = mx == ref[n][k] ? 1.f : ex2(ref[n][k] - mx);
                        ref[n][k] = mx;
                        l[n][k] *= f;
                        o[0][n][k] *= f;
                        o[0][n][k + 2] *= f;
                        o[1][n][k] *= f;
                        o[1][n][k + 2] *= f;
                    }
                weights();
                meet(false);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                l[n][0] += sum[n][0];
                l[n][1] += sum[n][1];
            }
            if (u > first && tid == 0) mbar_arrive(&b_empty[(u - 1) % NST]);
            if (td.flags & kUnitLast) break;
        }
        values(u);
        // ---- end of the part: join the warps, write out
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float x = l[n][k];
#pragma unroll
                for (int q = 4; q < 32; q <<= 1) x += __shfl_xor_sync(0xffffffffu, x, q);
                if (lane < 4) s_l[wk * S::kRows + n * 8 + t4 * 2 + k] = x;
            }
        float* po = nullptr;  // partial rows [rows][D], then m [rows], l [rows]
        if (td.slot >= 0) po = p.partial + static_cast<long long>(td.slot) * S::kRows * (D + 2);
        float4* xb = reinterpret_cast<float4*>(smem + S::kOffX);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float4 v[2] = {make_float4(o[0][n][0], o[0][n][2], o[1][n][0], o[1][n][2]),
                           make_float4(o[0][n][1], o[0][n][3], o[1][n][1], o[1][n][3])};
            if (S::kParts > 1 && part > 0) {
                xb[(wk - S::kSlices) * 64 + lane] = v[0];
                xb[(wk - S::kSlices) * 64 + 32 + lane] = v[1];
            }
            if (S::kParts > 1 || n == 0) meet(false);  // (n = 0: s_l too)
            if (part == 0) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
#pragma unroll
                    for (int q = 1; q < S::kParts; ++q) {
                        const float4 a = xb[(slice + (q - 1) * S::kSlices) * 64 + 32 * k + lane];
                        v[k].x += a.x;
                        v[k].y += a.y;
                        v[k].z += a.z;
                        v[k].w += a.w;
                    }
                    const int r = n * 8 + t4 * 2 + k, to = s_out[r];
                    if (to < 0) continue;
                    if ((s_nan[r] >> blk) & 1u) v[k] = make_float4(NAN, NAN, NAN, NAN);
                    float L = 0.f;
#pragma unroll
                    for (int w = 0; w < S::kWarps; ++w) L += s_l[w * S::kRows + r];
                    const float M = ref[n][k] == -INFINITY ? -INFINITY : ref[n][k] - kTail4;
                    const int col = slice * 32 + u8 * 4;
                    if (td.slot >= 0) {
                        *reinterpret_cast<float4*>(po + r * D + col) = v[k];
                        if (col == 0) {
                            po[S::kRows * D + r] = M;
                            po[S::kRows * (D + 1) + r] = L;
                        }
                    } else {
                        const long long orow = static_cast<long long>(td.b) * p.R + (to >> 16);
                        const int hq = to & 0xffff;
                        const float f = L == 0.f ? 0.f : vs / L;
                        *reinterpret_cast<uint2*>(p.out + orow * p.ldo + static_cast<long long>(hq) * D + col) =
                            make_uint2(pack2<false>(v[k].x * f, v[k].y * f),
                                       pack2<false>(v[k].z * f, v[k].w * f));
                        if (col == 0 && p.lse)
                            p.lse[orow * p.Hq + hq] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
                    }
                }
            }
            if (S::kParts > 1 || n == NT - 1) meet(false);
        }
        if (tid == 0) {
            mbar_arrive(&b_empty[u % NST]);
            mbar_arrive(&b_qe[qslot]);
        }
    }
}

template <int D, int NT>
cudaError_t attn4_launch(const AttnParams& p, const Kv4Blocks& kb, const AttnMaps& maps, int* grid,
                         int sms, cudaStream_t s) {
    using S = Attn4Shape<D, NT>;
    constexpr int kMinBlocks = S::kSmem <= 113 * 1024 && NT <= 3 ? 2 : 1;
    static std::atomic<unsigned long long> once;
    static std::atomic<int> occ;
    auto* kernel = attn4_kernel<D, NT, kMinBlocks>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (!bit || !(once.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        int n = 0;
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, S::kThreads, S::kSmem);
        if (e != cudaSuccess) return e;
        occ.store(n < 1 ? 1 : n);
        once.fetch_or(bit, std::memory_order_acq_rel);
    }
    const int resident = sms * occ.load();
    if (*grid > resident) *grid = resident;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(*grid);
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, kb, maps);
}

template <int D>
cudaError_t attn4_dispatch(const AttnParams& p, const Kv4Blocks& kb, const AttnMaps& maps, int nt,
                           int* grid, int sms, cudaStream_t s) {
    switch (nt) {
        case 1: return attn4_launch<D, 1>(p, kb, maps, grid, sms, s);
        case 2: return attn4_launch<D, 2>(p, kb, maps, grid, sms, s);
        case 3: return attn4_launch<D, 3>(p, kb, maps, grid, sms, s);
        case 4: return attn4_launch<D, 4>(p, kb, maps, grid, sms, s);
        case 6: return attn4_launch<D, 6>(p, kb, maps, grid, sms, s);
        case 8: return attn4_launch<D, 8>(p, kb, maps, grid, sms, s);
    }
    return cudaErrorInvalidValue;
}
#endif  // __CUDACC__

}  // namespace vw4
