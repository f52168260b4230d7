// attn_tc.cuh -- the attention of more than 16 query rows of a key head on the
// 5th-generation tensor cores: the same units, partials and results as
// attn_kernel (attn.cuh).
//
// One CTA per SM, warps with roles.  A producer warp loads K and V tiles (TMA)
// into a ring of half stages (K, V, K, V, ...) in the 128-byte swizzled layout
// the tensor cores read; one thread issues S = Q K^T and O += P V, whichever
// has its operands first, with Q and P in tensor memory (a product of 64 or
// 128 keys that also read Q from shared memory was bound by those reads); the
// softmax warps own one query row a thread, so the softmax has no shuffles and
// S and P never pass through shared memory.  S has two buffers: Q K^T of the
// next tile runs under the softmax of this one; P overwrites the front of its S.
//
// The last role brings an item's queries into tensor memory and differs by the
// cache's type.  bf16: four warps pass each V tile on; at the edges (keys that
// not every row sees) they clean it first.  e4m3: tiles arrive raw in a ring of
// their own, four warps turn K and four V into f16 (exact), cleaned the same
// way, and the queries into f16 under a power of two per row.
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
    static constexpr int kRaw = kTK * D;             // e4m3 half before conversion
    static constexpr int kNR = !F8 ? 0 : (D == 64 ? 8 : 5);
    static constexpr int kNS = F8 ? 4 : (D == 64 ? 8 : 6);
    static constexpr int kAuxWarps = F8 ? 8 : 4;     // converters, or cleaners
    static constexpr int kThreads = (6 + kAuxWarps) * 32;
    static constexpr int kOffRaw = kNS * kHalf;
    static constexpr int kOffStage = kOffRaw + kNR * kRaw;  // 4 KB a softmax warp, for the output
    static constexpr int kSmem = kOffStage + 4 * 4096 + 1024;  // and alignment
    static_assert(kSmem + 2048 <= 227 * 1024 && kSmem > 114 * 1024, "one CTA per SM");
    // tensor memory columns: O, two S, the queries (two 16-bit values a column)
    static constexpr uint32_t kColO = 0, kColS = D, kColQ = D + 2 * kTK;
    static constexpr int kNQ = D == 256 ? 1 : 2;
    static_assert(D + 2 * kTK + kNQ * D / 2 <= 512, "tensor memory");
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
    __shared__ __align__(8) uint64_t b_s[2], b_p[2], b_pv, b_q[2], b_qe[2], b_part[8], b_o, b_end;
    // log2 of the row scales of f16 queries, by part: the queries of part n + 4 wait for
    // the last products of part n + 2 or later, whose scores wait for reads of part n
    __shared__ int8_t s_rs[F8 ? 4 : 1][F8 ? ROWS : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row_warps = (p.tb * p.gb + 31) / 32;     // softmax warps with rows

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 160) {
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
    }
    if (warp == 4) {
        tmem_alloc<512>(&s_tmem);
        if (lane == 0) {
            for (int k = 0; k < NS; ++k) {
                mbar_init(&b_full[k], F8 ? 4 : 1);
                mbar_init(&b_empty[k], 1);
                mbar_init(&b_clean[k], 4);
            }
            for (int k = 0; k < NR; ++k) {
                mbar_init(&b_raw[k], 1);
                mbar_init(&b_raw_empty[k], 4);
            }
            for (int k = 0; k < 2; ++k) {
                mbar_init(&b_s[k], 1);
                mbar_init(&b_p[k], row_warps);
                mbar_init(&b_q[k], row_warps);
                mbar_init(&b_qe[k], 1);
            }
            for (int k = 0; k < 8; ++k) mbar_init(&b_part[k], 1);
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

    // An item's queries into tensor memory: one row a thread of four warps.  For an
    // e4m3 cache they become f16 under a power of two per row that puts the row's
    // largest magnitude into [2^14, 2^15): exact for every value down to 2^-31 of it
    // (bf16 has 8 significant bits, f16 11 and subnormals).
    auto queries = [&](const AttnUnit& d, int qw) {
        const int qs = d.seg % S::kNQ, r = qw * 32 + lane;
        const AttnRow row = attn_row(p, d.g, r);
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + (static_cast<long long>(d.b) * p.R + row.i) * p.ldq + static_cast<long long>(row.hq) * D);
        uint4 v[D == 256 ? 16 : D / 8];  // half a row of 256, else a row
        constexpr int NV = D == 256 ? 16 : D / 8;
        float up = 1.f;
        auto get = [&](int from) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                v[k] = row.live ? __ldg(src + from + k) : make_uint4(0, 0, 0, 0);
        };
        if (F8) {
            uint32_t mx = 0;  // largest magnitude, as bits
#pragma unroll 1
            for (int from = 0; from < D / 8; from += NV) {
                get(from);
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mx = max(mx, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
                }
            }
            const int ex = static_cast<int>(mx >> 7);
            int sh = ex == 0 || ex == 255 ? 0 : 127 + 14 - ex;
            sh = max(-126, min(126, sh));
            up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
            if (r < ROWS)
                s_rs[F8 ? d.seg & 3 : 0][F8 ? r : 0] = static_cast<int8_t>(sh);
        } else {
            get(0);
        }
        if (d.seg >= S::kNQ && !warp_wait(&b_qe[qs], d.seg / S::kNQ - 1)) return false;
        tc_fence_after();
#pragma unroll 1
        for (int from = 0; from < D / 8; from += NV) {
            if (F8 || from > 0) get(from);
#pragma unroll
            for (int c = 0; c < NV; c += 8) {
                uint32_t y[32];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint4 t = v[c + k];
                    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[4 * k + e] = F8 ? pack2<true>(__uint_as_float(w[e] << 16) * up,
                                                        __uint_as_float(w[e] & 0xffff0000u) * up)
                                          : w[e];
                }
                tmem_st32(tmem + (static_cast<uint32_t>(qw * 32) << 16) + S::kColQ + qs * (D / 2) +
                              (from + c) * 4, y);
            }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_q[qs]);
        return true;
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
        for (int u = 0; u < n_units; ++u) {
            const AttnUnit d = w.unit(p);
            const uint32_t bytes = w.template bytes<NB, BOXB>();
            if (lane == 0) {
                s_unit[u % kUnitRing] = d;
                if (d.flags & kUnitFirst) mbar_arrive(&b_part[d.seg & 7]);  // its queries may be read
            }
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                const int st = hl % NL;
                ok = hl < NL || warp_wait(&empty[st], hl / NL - 1);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&full[st], bytes);
                __syncwarp();
                w.template load<NB, BOXB, F8 ? 1 : 2>(
                    p, half ? &maps.v : &maps.k,
                    sm + (F8 ? S::kOffRaw + st * S::kRaw : st * S::kHalf), &full[st], lane);
                ++hl;
            }
            if (!ok) break;
            if (u + 1 < n_units) w.next(p, lane);
        }
        if (!ok) {  // copies in flight land before the block ends
            for (int k = hl > NL ? hl - NL : 0; k < hl; ++k)
                mbar_wait_bounded(&full[k % NL], (k / NL) & 1, p.wait_ns, nullptr);
        }
    } else if (n_units > 0 && warp >= 6) {
        // ----------------------------------------- cleaners or converters
        // Four warps a group; group 0 also brings the queries (its warps reach all
        // lanes of tensor memory: 32 (warp % 4) ..).  e4m3: group 0 has K, group 1 V.
        constexpr int N = 128;
        const int group = (warp - 6) >> 2, at = (tid - 192) & 127, half = F8 ? group : 1;
        const int qw = warp & 3;
        bool first = true;
        int parts = 0;
        for (int u = 0; u < n_units; ++u) {
            const int hh = 2 * u + half, st = hh % NS, sr = hh % NR;
            if (first) {
                if (group == 0 && qw < row_warps) {
                    if (!warp_wait(&b_part[parts & 7], parts >> 3)) break;
                    const AttnUnit d = s_unit[u % kUnitRing];
                    if (!queries(d, qw)) break;
                }
                ++parts;
            }
            if (!warp_wait(F8 ? &b_raw[sr] : &b_full[st], F8 ? hh / NR : hh / NS)) break;
            const AttnUnit d = s_unit[u % kUnitRing];
            first = d.flags & kUnitLast;  // (of the next unit)
            const bool clean = half == 1 && (d.flags & kUnitEdge);
            if (!F8) {
                if (clean) {
                    // Values that no row sees become zeros; infinities and NaN of values
                    // that only some rows see too (0 times them must not reach the other
                    // rows): the end of the part gives them to the rows that see them.
                    bool odd = false;
#pragma unroll 1
                    for (int c = at; c < TK * (D / 8); c += N) {
                        const int row = c / (D / 8), j = d.start + row;
                        if (key_all(j, d.len, d.p0, p.window, p.sinks)) continue;
                        uint4* q = reinterpret_cast<uint4*>(smem + st * S::kHalf + S::at(row, c % (D / 8)));
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
            } else {
                if (hh >= NS && !warp_wait(&b_empty[st], hh / NS - 1)) break;
                const uint8_t* src = smem + S::kOffRaw + sr * S::kRaw;
                uint8_t* dst = smem + st * S::kHalf;
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
        }
    } else if (n_units > 0 && warp == 4) {
        // ----------------------------------------------- the tensor cores
        if (lane == 0) {
            constexpr uint32_t iS = tc_idesc(!F8, 128, TK, false), iO = tc_idesc(!F8, 128, D, true);
            int fl[2] = {0, 0}, parts = 0;
            int qk = 0, pv = 0;   // next tile of either product
            bool k_in = false;    // the next K tile has arrived (its unit is known)
            uint64_t t0 = 0;
            while (pv < n_units) {
                // S of tile qk takes the buffer of tile qk - 2, whose P has been read
                if (qk < n_units && qk <= pv + 1) {
                    const int hk = 2 * qk;
                    k_in = k_in || mbar_test(&b_full[hk % NS], (hk / NS) & 1);
                    const AttnUnit* d = &s_unit[qk % kUnitRing];
                    const int seg = k_in ? d->seg : 0, qs = seg % S::kNQ;
                    if (k_in && (!(d->flags & kUnitFirst) || mbar_test(&b_q[qs], (seg / S::kNQ) & 1))) {
                        tc_fence_after();
                        const uint32_t k = sm + (hk % NS) * S::kHalf;
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks)
                            tc_mma_ts(tmem + S::kColS + (qk & 1) * TK,
                                      tmem + S::kColQ + qs * (D / 2) + ks * 8,
                                      tc_desc(k + (ks >> 2) * S::kBlk + (ks & 3) * 32, 16, 1024), iS,
                                      ks > 0);
                        tc_commit(&b_s[qk & 1]);
                        tc_commit(&b_empty[hk % NS]);
                        if (d->flags & kUnitLast) tc_commit(&b_qe[qs]);
                        fl[qk & 1] = d->flags;
                        ++qk;
                        k_in = false;
                        t0 = 0;
                        continue;
                    }
                }
                if (pv < qk) {
                    const int hv = 2 * pv + 1;
                    const bool first = fl[pv & 1] & kUnitFirst;
                    if (mbar_test(&b_p[pv & 1], (pv >> 1) & 1) &&
                        mbar_test(F8 ? &b_full[hv % NS] : &b_clean[hv % NS],
                                  (F8 ? hv / NS : attn_v_phase(hv, NS)) & 1) &&
                        (!first || parts == 0 || mbar_test(&b_o, (parts - 1) & 1))) {  // O was read
                        tc_fence_after();
                        const uint32_t v = sm + (hv % NS) * S::kHalf;
#pragma unroll
                        for (int ks = 0; ks < TK / 16; ++ks)
                            tc_mma_ts(tmem + S::kColO, tmem + S::kColS + (pv & 1) * TK + ks * 8,
                                      tc_desc(v + ks * 2048, S::kBlk, 1024), iO, !(first && ks == 0));
                        tc_commit(&b_empty[hv % NS]);
                        tc_commit(&b_pv);
                        parts += first;
                        ++pv;
                        t0 = 0;
                        continue;
                    }
                }
                if (s_abort) break;
                const uint64_t now = globaltimer_ns();
                if (t0 == 0) t0 = now;
                if (now - t0 > p.wait_ns) {
                    s_abort = 1;
                    atomicOr(p.status, kStatusWaitTimeout);
                    break;
                }
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
                    c2 *= __uint_as_float(
                        static_cast<uint32_t>(127 - s_rs[F8 ? td.seg & 3 : 0][F8 ? min(r, ROWS - 1) : 0]) << 23);
                }
                l = 0.f;
            }
            const uint32_t tS = tmem + lanes + S::kColS + (u & 1) * TK;
            uint32_t x[64];
            float mx = -INFINITY;
            auto masked = [&](int c) {  // 64 columns of the row from column c
                tmem_ld64(x, tS + c);
                if (edge) {
                    // seen: k <= hi and (k > lo or k < sk)
                    const int hi = pr - td.start - c;
                    if (p.window == 0) {
#pragma unroll
                        for (int k = 0; k < 64; ++k)
                            if (k > hi) x[k] = 0xff800000u;
                    } else {
                        const int lo = hi - p.window, sk = p.sinks - td.start - c;
#pragma unroll
                        for (int k = 0; k < 64; ++k)
                            if (k > hi || (k <= lo && k >= sk)) x[k] = 0xff800000u;
                    }
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
            // A wait names a phase by its parity, so the one before it must be known to be
            // over: S of tile u was committed after the product of tile u - 2.
            if ((u > 0 && !warp_wait(&b_pv, u - 1)) || !warp_wait(&b_pv, u)) break;
            tc_fence_after();
            const bool live = row.live, odd = s_odd[td.seg & 7] == td.seg + 1;
            const float mm = m == -INFINITY ? -INFINITY : mc;
            const float vs = F8 && p.v_scale ? __ldg(p.v_scale + h) : 1.f;
            const float f = td.slot >= 0 ? 1.f : (l == 0.f ? 0.f : vs / l);
            const long long orow = static_cast<long long>(td.b) * p.R + row.i;
            // The rows leave through 4 KB of shared memory a warp, 128 bytes of each of
            // the 32 rows at a time (fp32 partial: 32 columns, bf16: 64), so that eight
            // lanes write one row's line.
            const long long dst_row =
                td.slot >= 0 ? (static_cast<long long>(td.slot) * ROWS * (D + 2) + static_cast<long long>(r) * D) * 4
                             : (orow * p.ldo + static_cast<long long>(row.hq) * D) * 2;
            uint8_t* dst_base = td.slot >= 0 ? reinterpret_cast<uint8_t*>(p.partial)
                                             : reinterpret_cast<uint8_t*>(p.out);
            const int my_row = live ? 1 : 0;
            uint8_t* stage = smem + S::kOffStage + warp * 4096;
            const int width = td.slot >= 0 ? 32 : 64;  // columns a line
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
                if (td.slot >= 0) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<uint4*>(stage + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                            make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
                } else {
                    const int k0 = c & 32 ? 4 : 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack2<false>(__uint_as_float(y[8 * k + 2 * e]) * f,
                                                __uint_as_float(y[8 * k + 2 * e + 1]) * f);
                        *reinterpret_cast<uint4*>(stage + lane * 128 + (((k0 + k) ^ (lane & 7)) << 4)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (k0 == 0) continue;  // the other half of the lines is to come
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int rr = k * 4 + (lane >> 3);
                    const long long to = __shfl_sync(0xffffffffu, dst_row, rr);
                    const int on = __shfl_sync(0xffffffffu, my_row, rr);
                    if (on)
                        *reinterpret_cast<uint4*>(dst_base + to + (c / width) * 128 + (lane & 7) * 16) =
                            *reinterpret_cast<const uint4*>(stage + rr * 128 +
                                                            (((lane & 7) ^ (rr & 7)) << 4));
                }
            }
            __syncwarp();
            tc_fence_before();
            if (live) {
                if (td.slot >= 0) {
                    float* po = p.partial + static_cast<long long>(td.slot) * ROWS * (D + 2);
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
