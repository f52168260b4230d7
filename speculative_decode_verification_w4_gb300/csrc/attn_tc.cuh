// attn_tc.cuh -- the attention of more than 16 query rows of a key head on the
// 5th-generation tensor cores: the same units, partials and results as
// attn_kernel (attn.cuh).
//
// One CTA per SM, warps with roles.  A producer warp loads K and V tiles (TMA)
// into a ring of half stages (K, V, K, V, ...) in the 128-byte swizzled layout
// the tensor cores read; one thread issues S = Q K^T (both operands in shared
// memory) and O += P V (P in tensor memory, V contiguous along N); the softmax
// warps own one query row a thread, so the softmax has no shuffles and S and P
// never pass through shared memory.  S has two buffers: Q K^T of the next tile
// runs under the softmax of this one; P overwrites the front of its S.
//
// The last role differs by the cache's type.  bf16: four warps pass each V tile
// on; at the edges (keys that not every row sees) they clean it first.  e4m3:
// tiles arrive raw in a ring of their own and eight warps turn them into f16
// (exact), the queries into f16 under a power of two per row; both cleaned the
// same way.
//
// The running maximum that the exponents use follows the true one lazily: O is
// rescaled only when a row's maximum grew by more than 2^8 (its weights are
// then at most 2^8, harmless in bf16, f16 and the fp32 sum).
#pragma once
#include "attn.cuh"

namespace vw4 {
#ifdef __CUDACC__

template <int D, bool F8, int ROWS>
struct AttnTcShape {
    static constexpr int kTK = D == 256 ? 64 : 128;  // keys of a tile
    static constexpr int kHalf = kTK * D * 2;        // K or V of a tile, 16-bit operands
    static constexpr int kBlk = kTK * 128;           // 64 dimensions of it
    static constexpr int kQ = ROWS * D * 2;
    static constexpr int kQBlk = ROWS * 128;
    static constexpr int kNQ = D == 256 && ROWS == 128 ? 1 : 2;
    static constexpr int kRaw = kTK * D;             // e4m3 half before conversion
    static constexpr int kNR = !F8 ? 0 : (D == 64 ? 8 : 4);
    static constexpr int kNS = F8 ? (D == 64 ? 4 : 3)
                                  : (D == 64 ? 8 : (D == 128 && ROWS == 64 ? 6 : 5));
    static constexpr int kAuxWarps = F8 ? 8 : 4;     // converters, or cleaners
    static constexpr int kThreads = (6 + kAuxWarps) * 32;
    static constexpr int kOffSlots = kNQ * kQ;
    static constexpr int kOffRaw = kOffSlots + kNS * kHalf;
    static constexpr int kSmem = kOffRaw + kNR * kRaw + 1024;  // and alignment
    // the products read 128 rows of Q whatever ROWS is: what follows must be there
    static_assert(kOffRaw >= (kNQ - 1) * kQ + (D / 64 - 1) * kQBlk + 128 * 128, "Q reads");
    static_assert(kSmem + 2048 <= 227 * 1024 && kSmem > 114 * 1024, "one CTA per SM");
    static constexpr uint32_t kColO = 0, kColS = D;  // tensor memory columns
    static_assert(D + 2 * kTK <= 512, "tensor memory");
    __device__ static __forceinline__ uint32_t at(int row, int chunk) {  // 16 bytes of an operand row
        return static_cast<uint32_t>((chunk >> 3) * kBlk + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
    }
};

constexpr float kLazy = 8.f;

// The V halves are the odd ones: of a ring of ns slots, an even ns gives a slot
// only halves of one kind (every ns-th half), an odd ns one V in two rounds.
__host__ __device__ constexpr int attn_v_phase(int h, int ns) {
    return ns % 2 == 0 ? h / ns : h / (2 * ns);
}

template <int D, bool F8, int ROWS>
__global__ void __launch_bounds__(AttnTcShape<D, F8, ROWS>::kThreads, 1)
    attn_tc_kernel(const AttnParams p, const __grid_constant__ AttnMaps maps) {
    using S = AttnTcShape<D, F8, ROWS>;
    constexpr int TK = S::kTK, NS = S::kNS, NR = F8 ? S::kNR : 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    __shared__ volatile int s_odd[8];  // seg + 1: the part's values lost infinities or NaN
    __shared__ AttnUnit s_unit[kUnitRing];
    // loaded (bf16) or converted (e4m3) halves, their release, cleaned V halves (bf16)
    __shared__ __align__(8) uint64_t b_full[NS], b_empty[NS], b_clean[NS];
    __shared__ __align__(8) uint64_t b_raw[NR], b_raw_empty[NR];
    __shared__ __align__(8) uint64_t b_s[2], b_p[2], b_pv, b_q[2], b_qc[2], b_qe[2], b_o, b_end;
    __shared__ float s_rs[F8 ? 2 : 1][F8 ? ROWS : 1];  // 1 / row scale of f16 queries
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row_warps = (p.tb * p.gb + 31) / 32;     // softmax warps with rows

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 4) {
        tmem_alloc<512>(&s_tmem);
        if (lane == 0) {
            for (int k = 0; k < NS; ++k) {
                mbar_init(&b_full[k], F8 ? S::kAuxWarps : 1);
                mbar_init(&b_empty[k], 1);
                mbar_init(&b_clean[k], S::kAuxWarps);
            }
            for (int k = 0; k < NR; ++k) {
                mbar_init(&b_raw[k], 1);
                mbar_init(&b_raw_empty[k], S::kAuxWarps);
            }
            for (int k = 0; k < 2; ++k) {
                mbar_init(&b_s[k], 1);
                mbar_init(&b_p[k], row_warps);
                mbar_init(&b_q[k], 1);
                mbar_init(&b_qc[k], S::kAuxWarps);
                mbar_init(&b_qe[k], 1);
            }
            mbar_init(&b_pv, 1);
            mbar_init(&b_o, row_warps);
            mbar_init(&b_end, 1);
            fence_barrier_init();
            s_abort = 0;
            for (int k = 0; k < 8; ++k) s_odd[k] = 0;
        }
        tc_fence_before();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int cap = p.max_blocks * p.page_size;
    const AttnSpan span = attn_span<S::kThreads>(p, cap, TK);
    tc_fence_after();
    const int n_units = static_cast<int>(span.u1 - span.u0);
    const uint32_t sm = smem_u32(smem), tmem = s_tmem;
    auto wait = [&](uint64_t* bar, int phase) {
        if (mbar_wait_bounded(bar, phase & 1, p.wait_ns, &s_abort)) return true;
        s_abort = 1;
        atomicOr(p.status, kStatusWaitTimeout);
        return false;
    };
    // (the same answer in every lane: what follows is executed by whole warps)
    auto warp_wait = [&](uint64_t* bar, int phase) {
        return __all_sync(0xffffffffu, wait(bar, phase)) != 0;
    };

    if (n_units > 0 && warp == 5) {
        // -------------------------------------------------------- producer
        constexpr int NB = F8 ? 1 : D / 64, BOXB = F8 ? D : 128;  // boxes across a key
        constexpr int NL = F8 ? NR : NS;                          // ring that is loaded
        uint64_t* full = F8 ? b_raw : b_full;
        uint64_t* empty = F8 ? b_raw_empty : b_empty;
        AttnWalk<TK> w;
        w.begin(p, span, cap, lane);
        int hl = 0;  // halves loaded
        bool ok = true;
        int q_loads = 0;
        for (int u = 0; u < n_units; ++u) {
            const AttnUnit d = w.unit(p);
            const uint32_t bytes = w.template bytes<NB, BOXB>();
            if (d.flags & kUnitFirst) {
                const int qs = d.seg % S::kNQ;
                ok = d.seg < S::kNQ || warp_wait(&b_qe[qs], d.seg / S::kNQ - 1);
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&b_q[qs], attn_q_bytes(p, D));
                    attn_load_q<D>(p, &maps.q, sm + qs * S::kQ, S::kQBlk, d, &b_q[qs]);
                }
                ++q_loads;
                __syncwarp();
            }
            if (lane == 0) s_unit[u % kUnitRing] = d;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                const int st = hl % NL;
                ok = hl < NL || warp_wait(&empty[st], hl / NL - 1);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&full[st], bytes);
                __syncwarp();
                w.template load<NB, BOXB, F8 ? 1 : 2>(
                    p, half ? &maps.v : &maps.k,
                    sm + (F8 ? S::kOffRaw + st * S::kRaw : S::kOffSlots + st * S::kHalf), &full[st], lane);
                ++hl;
            }
            if (!ok) break;
            if (u + 1 < n_units) w.next(p, lane);
        }
        if (!ok) {  // copies in flight land before the block ends
            for (int k = hl > NL ? hl - NL : 0; k < hl; ++k)
                mbar_wait_bounded(&full[k % NL], (k / NL) & 1, p.wait_ns, nullptr);
            for (int k = q_loads > S::kNQ ? q_loads - S::kNQ : 0; k < q_loads; ++k)
                mbar_wait_bounded(&b_q[k % S::kNQ], (k / S::kNQ) & 1, p.wait_ns, nullptr);
        }
    } else if (n_units > 0 && warp >= 6) {
        // ----------------------------------------- cleaners or converters
        const int at = tid - 192;
        constexpr int N = S::kAuxWarps * 32;
        for (int u = 0; u < n_units; ++u) {
            if (!F8) {
                const int hv = 2 * u + 1, st = hv % NS;
                if (!warp_wait(&b_full[st], hv / NS)) break;
                const AttnUnit d = s_unit[u % kUnitRing];
                if (d.flags & kUnitEdge) {
                    // Values that no row sees become zeros; infinities and NaN of values
                    // that only some rows see too (0 times them must not reach the other
                    // rows): the end of the part gives them to the rows that see them.
                    bool odd = false;
#pragma unroll 1
                    for (int c = at; c < TK * (D / 8); c += N) {
                        const int row = c / (D / 8), j = d.start + row;
                        if (key_all(j, d.len, d.p0, p.window, p.sinks)) continue;
                        uint4* q = reinterpret_cast<uint4*>(smem + S::kOffSlots + st * S::kHalf +
                                                            S::at(row, c % (D / 8)));
                        if (!key_some(j, d.len, d.p0, p.window, p.sinks)) {
                            *q = make_uint4(0, 0, 0, 0);
                            continue;
                        }
                        const uint4 v = *q;
                        uint32_t w[4] = {v.x, v.y, v.z, v.w};
                        bool hit = false;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if ((w[e] & 0x7F80u) == 0x7F80u) w[e] &= 0xffff0000u, hit = true;
                            if ((w[e] & 0x7F800000u) == 0x7F800000u) w[e] &= 0xffffu, hit = true;
                        }
                        if (hit) *q = make_uint4(w[0], w[1], w[2], w[3]);
                        odd |= hit;
                    }
                    if (odd) s_odd[d.seg & 7] = d.seg + 1;
                    fence_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&b_clean[st]);
                continue;
            }
            bool ok = true;
#pragma unroll 1
            for (int half = 0; half < 2 && ok; ++half) {
                const int hh = 2 * u + half, st = hh % NS, sr = hh % NR;
                ok = warp_wait(&b_raw[sr], hh / NR);
                if (!ok) break;
                const AttnUnit d = s_unit[u % kUnitRing];
                if (half == 0 && (d.flags & kUnitFirst)) {
                    // The queries become f16 under a power of two per row that puts the
                    // row's largest magnitude into [2^14, 2^15): exact for every value
                    // down to 2^-31 of it.
                    const int qs = d.seg % S::kNQ;
                    ok = warp_wait(&b_q[qs], d.seg / S::kNQ);
                    if (!ok) break;
                    for (int r = warp - 6; r < p.tb * p.gb; r += S::kAuxWarps) {
                        uint32_t x[D / 64];
                        float mx = 0.f;
#pragma unroll
                        for (int k = 0; k < D / 64; ++k) {
                            // 64 dimensions: word `lane` of the 128-byte row of block k
                            const uint32_t o = qs * S::kQ + k * S::kQBlk + r * 128 +
                                               (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4;
                            x[k] = *reinterpret_cast<const uint32_t*>(smem + o);
                            mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(x[k] << 16)),
                                                 fabsf(__uint_as_float(x[k] & 0xffff0000u))));
                        }
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1)
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                        const int ex = static_cast<int>(__float_as_uint(mx) >> 23);
                        int sh = ex == 0 || ex == 255 ? 0 : 127 + 14 - ex;
                        sh = max(-126, min(126, sh));
                        const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
                        if (lane == 0)
                            s_rs[F8 ? qs : 0][F8 ? r : 0] =
                                __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
#pragma unroll
                        for (int k = 0; k < D / 64; ++k) {
                            const uint32_t o = qs * S::kQ + k * S::kQBlk + r * 128 +
                                               (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4;
                            *reinterpret_cast<uint32_t*>(smem + o) =
                                pack2<true>(__uint_as_float(x[k] << 16) * up,
                                            __uint_as_float(x[k] & 0xffff0000u) * up);
                        }
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&b_qc[qs]);
                }
                ok = hh < NS || warp_wait(&b_empty[st], hh / NS - 1);
                if (!ok) break;
                const uint8_t* src = smem + S::kOffRaw + sr * S::kRaw;
                uint8_t* dst = smem + S::kOffSlots + st * S::kHalf;
                const bool clean = half == 1 && (d.flags & kUnitEdge);
                bool odd = false;
                constexpr int CH = D / 16;
#pragma unroll 4
                for (int i = 0; i < TK * CH / N; ++i) {
                    const int c = at + i * N, row = c / CH, ch = c % CH;
                    const uint4 v = *reinterpret_cast<const uint4*>(src + c * 16);
                    uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    if (clean) {  // (as above)
                        const int j = d.start + row;
                        if (!key_some(j, d.len, d.p0, p.window, p.sinks)) {
                            w[0] = w[1] = w[2] = w[3] = 0u;
                        } else if (!key_all(j, d.len, d.p0, p.window, p.sinks)) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
#pragma unroll
                                for (int q = 0; q < 32; q += 8)
                                    if (((w[e] >> q) & 0x7Fu) == 0x7Fu) {
                                        w[e] &= ~(0xFFu << q);
                                        odd = true;
                                    }
                        }
                    }
                    uint32_t f[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        f[2 * e] = e4m3x2_f16x2(w[e]);
                        f[2 * e + 1] = e4m3x2_f16x2(w[e] >> 16);
                    }
                    // lanes of neighbouring 64-dimension blocks write their two chunks in
                    // opposite order: eight lanes then cover all banks
                    const int flip = (ch >> 2) & 1;
                    uint4 a = make_uint4(f[0], f[1], f[2], f[3]), b = make_uint4(f[4], f[5], f[6], f[7]);
                    *reinterpret_cast<uint4*>(dst + S::at(row, 2 * ch + flip)) = flip ? b : a;
                    *reinterpret_cast<uint4*>(dst + S::at(row, 2 * ch + 1 - flip)) = flip ? a : b;
                }
                if (odd) s_odd[d.seg & 7] = d.seg + 1;
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&b_full[st]);
                    mbar_arrive(&b_raw_empty[sr]);
                }
            }
            if (!ok) break;
        }
    } else if (n_units > 0 && warp == 4) {
        // ----------------------------------------------- the tensor cores
        if (lane == 0) {
            constexpr uint32_t iS = tc_idesc(!F8, 128, TK, false), iO = tc_idesc(!F8, 128, D, true);
            int fl[2] = {0, 0}, seg = 0;
            auto scores = [&](int u) {
                const int hk = 2 * u;
                if (!wait(&b_full[hk % NS], hk / NS)) return false;
                const AttnUnit* d = &s_unit[u % kUnitRing];
                fl[u & 1] = d->flags;
                seg = d->seg;
                const int qs = seg % S::kNQ;
                if ((d->flags & kUnitFirst) && !wait(F8 ? &b_qc[qs] : &b_q[qs], seg / S::kNQ))
                    return false;
                tc_fence_after();
                const uint32_t q = sm + qs * S::kQ;
                const uint32_t k = sm + S::kOffSlots + (hk % NS) * S::kHalf;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    tc_mma_ss(tmem + S::kColS + (u & 1) * TK,
                              tc_desc(q + (ks >> 2) * S::kQBlk + (ks & 3) * 32, 16, 1024),
                              tc_desc(k + (ks >> 2) * S::kBlk + (ks & 3) * 32, 16, 1024), iS, ks > 0);
                tc_commit(&b_s[u & 1]);
                tc_commit(&b_empty[hk % NS]);
                if (d->flags & kUnitLast) tc_commit(&b_qe[qs]);
                return true;
            };
            bool ok = scores(0);
            int parts = -1;
            for (int u = 0; u < n_units && ok; ++u) {
                const bool first = fl[u & 1] & kUnitFirst;
                if (u + 1 < n_units) ok = scores(u + 1);
                if (first && ++parts > 0) ok = ok && wait(&b_o, parts - 1);  // O has been read
                const int hv = 2 * u + 1;
                ok = ok && wait(&b_p[u & 1], u >> 1) &&
                     wait(F8 ? &b_full[hv % NS] : &b_clean[hv % NS],
                          F8 ? hv / NS : attn_v_phase(hv, NS));
                if (!ok) break;
                tc_fence_after();
                const uint32_t v = sm + S::kOffSlots + (hv % NS) * S::kHalf;
#pragma unroll
                for (int ks = 0; ks < TK / 16; ++ks)
                    tc_mma_ts(tmem + S::kColO, tmem + S::kColS + (u & 1) * TK + ks * 8,
                              tc_desc(v + ks * 2048, S::kBlk, 1024), iO, !(first && ks == 0));
                tc_commit(&b_empty[hv % NS]);
                tc_commit(&b_pv);
            }
            // everything issued is complete before the tensor memory is given back
            tc_commit(&b_end);
            mbar_wait_bounded(&b_end, 0, p.wait_ns, nullptr);
        }
        __syncwarp();
    } else if (n_units > 0 && warp < row_warps) {
        // ---------------------------------------------------------- softmax
        const int r = tid;  // row of the block = lane of tensor memory
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
        const uint32_t tO = tmem + lanes + S::kColO;
        float m = -INFINITY, l = 0.f, c2 = 1.f;
        int pr = -1, seg_start = 0;
        AttnRow row{};
        for (int u = 0; u < n_units; ++u) {
            if (!warp_wait(&b_s[u & 1], u >> 1)) break;
            tc_fence_after();
            const AttnUnit td = s_unit[u % kUnitRing];
            const int h = td.g / p.row_blocks;
            const bool first = td.flags & kUnitFirst, edge = td.flags & kUnitEdge;
            if (first) {
                seg_start = td.start;
                row = attn_row(p, td.g, r);
                pr = row.live ? td.p0 + row.i : -1;
                c2 = p.scale * kLog2e;
                if (F8) {
                    if (p.k_scale) c2 *= __ldg(p.k_scale + h);
                    c2 *= s_rs[F8 ? td.seg % S::kNQ : 0][F8 ? min(r, ROWS - 1) : 0];
                }
                l = 0.f;
            }
            const uint32_t tS = tmem + lanes + S::kColS + (u & 1) * TK;
            uint32_t x[64];
            float mx = -INFINITY;
            auto masked = [&](int c) {  // 64 columns of the row from column c
                tmem_ld64(x, tS + c);
                if (edge) {
#pragma unroll
                    for (int k = 0; k < 64; ++k)
                        if (!key_seen(td.start + c + k, pr, p.window, p.sinks)) x[k] = 0xff800000u;
                }
            };
#pragma unroll
            for (int c = TK - 64; c >= 0; c -= 64) {
                masked(c);
#pragma unroll
                for (int k = 0; k < 64; k += 2)
                    mx = fmaxf(mx, fmaxf(__uint_as_float(x[k]), __uint_as_float(x[k + 1])));
            }
            bool grow = false;
            float corr = 1.f;
            if (first) {
                m = mx;
            } else if ((mx - m) * c2 > kLazy) {
                // (m = -infinity: O and l are zeros still)
                if (m != -INFINITY) {
                    corr = ex2((m - mx) * c2);
                    grow = true;
                }
                l *= corr;
                m = mx;
            }
            if (__any_sync(0xffffffffu, grow)) {
                if (!warp_wait(&b_pv, u - 1)) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t y[32];
                    tmem_ld32(y, tO + c);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        y[k] = __float_as_uint(__uint_as_float(y[k]) * corr);
                    tmem_st32(tO + c, y);
                }
            }
            const float mc = m == -INFINITY ? 0.f : m * c2;
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int c = 0; c < TK; c += 64) {
                if (c > 0) masked(c);
                uint32_t y[32];
#pragma unroll
                for (int k = 0; k < 64; k += 2) {
                    const float a = ex2(fmaf(__uint_as_float(x[k]), c2, -mc));
                    const float b = ex2(fmaf(__uint_as_float(x[k + 1]), c2, -mc));
                    s0 += a;
                    s1 += b;
                    y[k / 2] = pack2<F8>(a, b);
                }
                tmem_st32(tS + c / 2, y);
            }
            l += s0 + s1;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b_p[u & 1]);
            if (!(td.flags & kUnitLast)) continue;

            // ---- end of the segment
            if (!warp_wait(&b_pv, u)) break;
            tc_fence_after();
            const bool live = row.live, odd = s_odd[td.seg & 7] == td.seg + 1;
            const float mm = m == -INFINITY ? -INFINITY : mc;
            const float vs = F8 && p.v_scale ? __ldg(p.v_scale + h) : 1.f;
            const float f = td.slot >= 0 ? 1.f : (l == 0.f ? 0.f : vs / l);
            const long long orow = static_cast<long long>(td.b) * p.R + row.i;
            __nv_bfloat16* out = p.out + orow * p.ldo + static_cast<long long>(row.hq) * D;
            float* po = p.partial + static_cast<long long>(td.slot < 0 ? 0 : td.slot) * ROWS * (D + 2);
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t y[32];
                __syncwarp();
                tmem_ld32(y, tO + c);
                if (odd && live) {
                    // infinities and NaN of values that this row sees and others do not
                    auto give = [&](int j0, int j1) {
#pragma unroll 1
                        for (int j = max(j0, seg_start); j <= min(j1, td.start + TK - 1); ++j) {
                            const int pg = p.table[static_cast<long long>(td.b) * p.table_stride +
                                                   (j >> p.page_shift)];
                            if (pg < 0 || pg >= p.num_pages || !key_seen(j, pr, p.window, p.sinks))
                                continue;
                            const long long at = static_cast<long long>(pg) * p.page_stride +
                                                 static_cast<long long>(j & (p.page_size - 1)) *
                                                     p.token_stride +
                                                 static_cast<long long>(h) * p.head_stride + c;
                            // (loops: rare, and y keeps constant indexes)
#pragma unroll
                            for (int k = 0; k < 32; ++k) {
                                float vv;
                                if (F8)
                                    vv = (static_cast<const uint8_t*>(p.v)[at + k] & 0x7F) == 0x7F ? NAN : 0.f;
                                else
                                    vv = __bfloat162float(static_cast<const __nv_bfloat16*>(p.v)[at + k]);
                                if (!isfinite(vv))
                                    y[k] = __float_as_uint(__uint_as_float(y[k]) + vv);
                            }
                        }
                    };
                    // the ends of the rows' windows, then the verify rows themselves
                    if (p.window > 0)
                        give(max(0, td.p0 - p.window + 1), min(td.p0, td.len - 1 - p.window));
                    give(max(0, td.p0 + 1), td.len - 1);
                }
                if (live && td.slot >= 0) {
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        *reinterpret_cast<uint4*>(po + r * D + c + k) =
                            make_uint4(y[k], y[k + 1], y[k + 2], y[k + 3]);
                } else if (live) {
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack2<false>(__uint_as_float(y[k + 2 * e]) * f,
                                                __uint_as_float(y[k + 2 * e + 1]) * f);
                        *reinterpret_cast<uint4*>(out + c + k) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            __syncwarp();
            tc_fence_before();
            if (live) {
                if (td.slot >= 0) {
                    po[ROWS * D + r] = mm;
                    po[ROWS * (D + 1) + r] = l;
                } else if (p.lse) {
                    p.lse[orow * p.Hq + row.hq] = l == 0.f ? -INFINITY : (mm + log2f(l)) * kLn2;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&b_o);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc<512>(tmem);
    }
}

#endif  // __CUDACC__
}  // namespace vw4
