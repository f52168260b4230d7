// attn4_tc.cuh -- attention of many query rows of a key head over the 4-bit cache on the
// 5th-generation tensor cores: the same units, partials and results as attn4_kernel.
//
// One CTA an SM, warps with roles.  Two warps load raw tiles of K and of V (codes and block
// scales, TMA and bulk copies); four turn K into f16, four V (exact, as in attn4.cuh), in the
// swizzled layout that the tensor cores read: neither needs to be transposed, for the
// instructions take V by its dimensions.  One thread issues S = Q K^T of a tile, then
// O += P V of the tile before.  The softmax warps own query rows, one a thread, or (blocks of
// up to 64 rows) half a row: they bring an item's queries into tensor memory, form P over
// their S, and write the rows of an item that is done.  Q, S and P, and O stay in tensor
// memory: at head size 256 tiles of 64 keys leave the room.
//
// What bounds it: the way of a tile from its scores to its weights in the softmax warps, a
// chain of latencies of about 1 us under the load of the other warps (16384 keys' and as many
// values' elements; their conversion takes 0.5 us beside it, the products 0.5, the bytes from
// HBM 0.4).  Without conversions and exponentials a tile still takes 1.1 us of its 1.4.  So
// the time hardly grows with the rows: 32 sequences of up to 32768 tokens, 8 key heads of
// size 128, are 220 us at 48 rows, 235 at 64 and 310 at 128, of 424 MB.  Tried and slower:
// weights formed at once against the lagging reference (252 at 64 rows), the rows' copies in
// the other lanes so that every sub-core has softmax warps (332), keys as the rows of the
// instructions and eight warps of weights through shared memory (541).
//
// The reference of the weights follows the running maximum lazily, as in attn4.cuh.
#pragma once
#include "attn4.cuh"

namespace vw4 {

constexpr int attn4_tc_tk(int D) { return D == 256 ? 64 : 128; }
constexpr int kAttn4TcGrid = kAttnMaxGrid256;

#ifdef __CUDACC__
template <int D, int ROWS>
struct Attn4TcShape {
    static constexpr int kTK = attn4_tc_tk(D);
    static constexpr int kThreads = 16 * 32;
    static constexpr int kHalves = ROWS == 64 ? 2 : 1;  // threads of a row
    static constexpr int kKB = D / 2, kNB = D / 16;
    static constexpr int kTile = kTK * kKB;
    static constexpr int kRaw = kTile + kTK * kNB;      // codes, scales
    static constexpr int kNR = 4;                       // places of a raw ring
    static constexpr int kBlk = D / 64;                 // blocks of 64 dimensions
    static constexpr int kF = kTK * D * 2;              // a tile in f16
    static constexpr int kNF = 2;                       // places of an f16 ring
    static constexpr int kNQ = D == 256 ? 1 : 2;        // query buffers
    static constexpr int kOffV = kNF * kF;
    static constexpr int kOffRawK = 2 * kNF * kF;
    static constexpr int kOffRawV = kOffRawK + kNR * kRaw;
    static constexpr int kUsed = kOffRawV + kNR * kRaw + 1024;
    static constexpr int kSmem = kUsed < 115 * 1024 ? 115 * 1024 : kUsed;  // one CTA an SM
    static_assert(kSmem <= 221 * 1024, "shared memory");
    static_assert(kRaw % (8 * kKB) == 0 && kF % 1024 == 0, "alignment");
    // tensor memory columns: O, two S (P over them), the queries
    static constexpr uint32_t kColS = D, kColQ = D + 2 * kTK;
    static_assert(D + 2 * kTK + kNQ * D / 2 <= 512, "tensor memory");
    // warps: softmax 0 .. 3, or 0, 1 and 4, 5 (which reach the same lanes)
    static constexpr int kLoadK = kHalves > 1 ? 2 : 4, kLoadV = kLoadK + 1;
    __device__ static __forceinline__ uint32_t raw_at(int key, int chunk) {  // 32 codes of a key
        const int x = kKB == 128 ? key & 7 : (kKB == 64 ? (key >> 1) & 3 : (key >> 2) & 1);
        return static_cast<uint32_t>(key * kKB + ((chunk ^ x) << 4));
    }
    __device__ static __forceinline__ uint32_t f_at(int key, int chunk) {  // 8 values of a key
        return static_cast<uint32_t>((key >> 3) * (kBlk * 1024) + (chunk >> 3) * 1024 + (key & 7) * 128 +
                                     (((chunk & 7) ^ (key & 7)) << 4));
    }
};
constexpr int kTc4Mma = 6, kTc4K = 8, kTc4V = 12;  // first warps of the roles

template <int D, int ROWS>
__global__ void __launch_bounds__(Attn4TcShape<D, ROWS>::kThreads, 1)
    attn4_tc_kernel(const AttnParams p, const Kv4Blocks kb, const __grid_constant__ AttnMaps maps) {
    using S = Attn4TcShape<D, ROWS>;
    constexpr int TK = S::kTK, NR = S::kNR, NF = S::kNF, NQ = S::kNQ, H = S::kHalves, NB = S::kNB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    __shared__ volatile int s_odd[8];            // seg + 1: the part's values lost NaN
    __shared__ AttnUnit s_unit[kUnitRing], s_vunit[kUnitRing], s_part[16];
    __shared__ float s_mx[2][2][H > 1 ? ROWS : 1];  // of a tile's columns, for the other half
    __shared__ float s_sum[H > 1 ? ROWS : 1];       // of a part's weights
    __shared__ __align__(8) uint64_t b_rk[NR], b_rke[NR], b_rv[NR], b_rve[NR];
    __shared__ __align__(8) uint64_t b_k[NF], b_ke[NF], b_v[NF], b_ve[NF];
    __shared__ __align__(8) uint64_t b_s[2], b_p[2], b_pv[2], b_q[2], b_qe[2], b_part[16], b_o, b_end;
    __shared__ __align__(8) uint64_t b_x[2][4];     // s_mx of a half's warp is there
    __shared__ __align__(8) uint64_t b_l[4];        // s_sum of the other half's warp is there
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row_warps = (p.tb * p.gb + 31) / 32;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == S::kLoadK * 32) {
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
    }
    if (warp == kTc4Mma) {
        tmem_alloc<512>(&s_tmem);
        if (lane == 0) {
            for (int k = 0; k < NR; ++k) {
                mbar_init(&b_rk[k], 1);
                mbar_init(&b_rv[k], 1);
                mbar_init(&b_rke[k], 4);
                mbar_init(&b_rve[k], 4);
            }
            for (int k = 0; k < NF; ++k) {
                mbar_init(&b_k[k], 4);
                mbar_init(&b_v[k], 4);
                mbar_init(&b_ke[k], 1);
                mbar_init(&b_ve[k], 1);
            }
            for (int k = 0; k < 2; ++k) {
                mbar_init(&b_s[k], 1);
                mbar_init(&b_pv[k], 1);
                mbar_init(&b_p[k], H * row_warps);
                mbar_init(&b_q[k], H * row_warps);
                mbar_init(&b_qe[k], 1);
                for (int j = 0; j < 4; ++j) mbar_init(&b_x[k][j], 1);
            }
            for (int k = 0; k < 16; ++k) mbar_init(&b_part[k], 1);
            for (int k = 0; k < 4; ++k) mbar_init(&b_l[k], 1);
            mbar_init(&b_o, H * row_warps);
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

    if (n_units > 0 && (warp == S::kLoadK || warp == S::kLoadV)) {
        // -------------------------------------------------------- loading warps
        const bool keys = warp == S::kLoadK;
        const CUtensorMap* map = keys ? &maps.k : &maps.v;
        const uint8_t* blocks = keys ? kb.k : kb.v;
        uint64_t* full = keys ? b_rk : b_rv;
        uint64_t* empty = keys ? b_rke : b_rve;
        const uint64_t policy = policy_evict_normal();
        const uint32_t box = static_cast<uint32_t>(p.box_rows * NB);
        AttnWalk<TK> w;
        w.begin(p, span, cap, lane);
        int u = 0;
        for (; u < n_units; ++u) {
            const int st = u % NR;
            const AttnUnit d = w.unit(p);
            const AttnTile t = w.tile(p);
            if (u + 1 < n_units) w.next(p, lane);
            if (lane == 0 && keys && (d.flags & kUnitFirst)) {
                // (its place was read by the queries of sixteen parts before)
                s_part[d.seg & 15] = d;
                mbar_arrive(&b_part[d.seg & 15]);
            }
            const bool there = t.page >= 0 && t.page < p.num_pages;
            const uint32_t bytes = t.template bytes<TK, 1, S::kKB>(0, lane) +
                                   __popc(__ballot_sync(0xffffffffu, there)) * box;
            const uint8_t* from = blocks;
            if (there)
                from += t.page * kb.page_stride + t.h * kb.head_stride +
                        ((t.start + lane * p.box_rows) & (p.page_size - 1)) * NB;
            const int off = (keys ? S::kOffRawK : S::kOffRawV) + st * S::kRaw;
            uint8_t* sdst = smem + off + S::kTile + lane * box;
            if (u >= NR && !warp_wait(&empty[st], u / NR - 1)) break;
            if (t.page == p.num_pages) {  // no such page: zeros
                for (uint32_t c = 0; c < box; c += 16)
                    *reinterpret_cast<uint4*>(sdst + c) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
            }
            __syncwarp();
            if (lane == 0) {
                (keys ? s_unit : s_vunit)[u % kUnitRing] = d;
                mbar_arrive_expect_tx(&full[st], bytes);
            }
            __syncwarp();
            t.template load<TK, 1, 1, S::kKB, 1>(p, map, sm + off, &full[st], 0, 0, lane);
            if (there) bulk_load(sdst, from, box, &full[st], policy);
            __syncwarp();
        }
        if (u < n_units)  // copies in flight land before the block ends
            for (int k = u > NR ? u - NR : 0; k < u; ++k)
                mbar_wait_bounded(&full[k % NR], (k / NR) & 1, p.wait_ns, nullptr);
    } else if (n_units > 0 && warp >= kTc4K) {
        // -------------------------------------------------- K and V become f16
        const bool keys = warp < kTc4V;
        const int cw = warp & 3;
        uint64_t* raw = keys ? b_rk : b_rv;
        uint64_t* raw_e = keys ? b_rke : b_rve;
        uint64_t* full = keys ? b_k : b_v;
        uint64_t* empty = keys ? b_ke : b_ve;
        // Eight neighbouring lanes take the same 32 dimensions of eight keys: loads and stores
        // then fall into different banks.
        constexpr int CH = D / 32;                        // chunks of a key
        constexpr int STEP = 32 / CH > 8 ? 32 / CH : 8;   // keys that a warp takes at once
        constexpr int PASS = CH > 4 ? CH / 4 : 1;         // passes over their chunks
        const int lk = (lane & 7) + (CH == 2 ? (lane >> 4) * 8 : 0);
        const int lc = CH == 2 ? (lane >> 3) & 1 : lane >> 3;
        for (int u = 0; u < n_units; ++u) {
            const int st = u % NR, ft = u % NF;
            if (!warp_wait(&raw[st], u / NR)) break;
            if (u >= NF && !warp_wait(&empty[ft], u / NF - 1)) break;
            const uint8_t* src = smem + (keys ? S::kOffRawK : S::kOffRawV) + st * S::kRaw;
            uint8_t* dst = smem + (keys ? 0 : S::kOffV) + ft * S::kF;
            AttnUnit d;
            bool edge = false, odd = false;
            if (!keys) {
                d = s_vunit[u % kUnitRing];
                edge = d.flags & kUnitEdge;
            }
#pragma unroll
            for (int g = 0; g < TK / STEP / 4; ++g) {
                const int key = (g * 4 + cw) * STEP + lk;
#pragma unroll
                for (int q = 0; q < PASS; ++q) {
                    const int c = lc + 4 * q;
                    const uint4 v = *reinterpret_cast<const uint4*>(src + S::raw_at(key, c));
                    uint32_t s = *reinterpret_cast<const uint16_t*>(src + S::kTile + key * NB + c * 2);
                    if (edge) {
                        // values that no row sees become zeros, whatever the cache holds there; a
                        // NaN scale that only some rows see too: the end of the part gives it to
                        // those
                        const int j = d.start + key;
                        if (!key_some(j, d.len, d.p0, p.window, p.sinks)) {
                            s = 0u;
                        } else if (!key_all(j, d.len, d.p0, p.window, p.sinks)) {
                            if ((s & 0x7fu) == 0x7fu) s &= 0xff00u, odd = true;
                            if ((s & 0x7f00u) == 0x7f00u) s &= 0xffu, odd = true;
                        }
                    }
                    const uint32_t s2 = e4m3x2_f16x2(s);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t x[4];
                        e2m1x8_f16(w[k], x);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            x[i] = k < 2 ? mul_f16x2_half<false>(x[i], s2) : mul_f16x2_half<true>(x[i], s2);
                        *reinterpret_cast<uint4*>(dst + S::f_at(key, 4 * c + k)) =
                            make_uint4(x[0], x[1], x[2], x[3]);
                    }
                }
            }
            if (odd) s_odd[d.seg & 7] = d.seg + 1;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&full[ft]);
                mbar_arrive(&raw_e[st]);
            }
        }
    } else if (n_units > 0 && warp == kTc4Mma) {
        // ----------------------------------------------- the tensor cores
        if (elect_one()) {
            constexpr uint32_t iS = tc_idesc(false, 128, TK, false), iO = tc_idesc(false, 128, D, true);
            auto scores = [&](int u) {
                if (!wait(&b_k[u % NF], u / NF)) return false;
                const int flags = s_unit[u % kUnitRing].flags, seg = s_unit[u % kUnitRing].seg;
                if ((flags & kUnitFirst) && !wait(&b_q[seg % NQ], seg / NQ)) return false;
                tc_fence_after();
                const uint64_t kd = tc_desc<128>(sm + u % NF * S::kF, 16, S::kBlk * 1024);
                const uint32_t tq = tmem + S::kColQ + seg % NQ * (D / 2);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    tc_mma_ts<false>(tmem + S::kColS + (u & 1) * TK, tq + ks * 8,
                                     kd + (((ks / 4) * 1024 + (ks % 4) * 32) >> 4), iS, ks > 0);
                tc_commit(&b_ke[u % NF]);
                tc_commit(&b_s[u & 1]);
                if (flags & kUnitLast) tc_commit(&b_qe[seg % NQ]);
                return true;
            };
            auto values = [&](int u) {
                const bool first = s_unit[u % kUnitRing].flags & kUnitFirst;
                const int seg = s_unit[u % kUnitRing].seg;
                if (!wait(&b_p[u & 1], u >> 1) || !wait(&b_v[u % NF], u / NF)) return false;
                if (first && seg > 0 && !wait(&b_o, seg - 1)) return false;
                tc_fence_after();
                const uint64_t vd = tc_desc<128>(sm + S::kOffV + u % NF * S::kF, 1024, S::kBlk * 1024);
#pragma unroll
                for (int ks = 0; ks < TK / 16; ++ks)
                    tc_mma_ts<false>(tmem, tmem + S::kColS + (u & 1) * TK + ks * 8,
                                     vd + ((ks * 2 * S::kBlk * 1024) >> 4), iO, !(first && ks == 0));
                tc_commit(&b_ve[u % NF]);
                tc_commit(&b_pv[u & 1]);
                return true;
            };
            // S of a unit under the softmax of the unit before, then the product of that; at
            // the end of a part the product first, for the next part's queries come later
            for (int u = 0; u <= n_units; ++u) {
                const bool last = u > 0 && (s_unit[(u - 1) % kUnitRing].flags & kUnitLast);
                if (last && !values(u - 1)) break;
                if (u < n_units && !scores(u)) break;
                if (u > 0 && !last && !values(u - 1)) break;
            }
            // everything issued is complete before the tensor memory is given back
            tc_commit(&b_end);
            mbar_wait_bounded(&b_end, 0, p.wait_ns, nullptr);
        }
        __syncwarp();
    } else if (n_units > 0 && warp < 4 * H && (warp & 3) < row_warps) {
        // ------------------------------------------- queries in, softmax, rows out
        const int half = warp >> 2, rw = warp & 3;
        const int r = rw * 32 + lane;  // row of the block = lane of tensor memory
        const uint32_t lanes = static_cast<uint32_t>(rw * 32) << 16;
        const uint32_t tO = tmem + lanes;
        float m = -INFINITY, l = 0.f, c2 = 1.f, c2_next = 1.f;
        AttnRow row{}, row_next{};
        int pr = -1, seg_start = 0;

        // An item's queries into tensor memory: f16 under a power of two per row that puts its
        // largest magnitude into [2^14, 2^15), with the sign of the head's scale.  A half of
        // a row's threads reads all of it and brings its half.
        auto queries = [&](int seg) {
            if (!warp_wait(&b_part[seg & 15], seg >> 4)) return false;
            const AttnUnit d = s_part[seg & 15];
            const int h = d.g / p.row_blocks;
            const float ks = p.k_scale ? __ldg(p.k_scale + h) : 1.f;
            row_next = attn_row(p, d.g, r);
            const uint4* src = reinterpret_cast<const uint4*>(
                p.q + (static_cast<long long>(d.b) * p.R + row_next.i) * p.ldq +
                static_cast<long long>(row_next.hq) * D);
            uint32_t mx = 0;
#pragma unroll 1
            for (int c = 0; c < D / 8; c += 8) {
                uint4 v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = row_next.live ? __ldg(src + c + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx = max(mx, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
                }
            }
            const int ex = static_cast<int>(mx >> 7);
            int sh = ex == 0 || ex == 255 ? 0 : 127 + 14 - ex;
            sh = max(-126, min(126, sh));
            const float up = copysignf(__uint_as_float(static_cast<uint32_t>(127 + sh) << 23), ks);
            c2_next = p.scale * kLog2e * fabsf(ks) * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
            if (c2_next < kMinFactor) c2_next = kMinFactor;  // (NaN stays)
            if (seg >= NQ && !warp_wait(&b_qe[seg % NQ], seg / NQ - 1)) return false;
            tc_fence_after();
            __syncwarp();
            const uint32_t tq = tmem + lanes + S::kColQ + seg % NQ * (D / 2);
#pragma unroll 1
            for (int c = half * (D / 8 / H); c < (half + 1) * (D / 8 / H); c += 4) {  // 32 dimensions
                uint32_t y[16];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 v = row_next.live ? __ldg(src + c + k) : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[4 * k + e] = pack2<true>(__uint_as_float(w[e] << 16) * up,
                                                   __uint_as_float(w[e] & 0xffff0000u) * up);
                }
                __syncwarp();
                tmem_st16(tq + c * 4, y);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b_q[seg % NQ]);
            return true;
        };

        // A part's rows from tensor memory to the output, or to its partial.
        auto finish = [&](const AttnUnit& td, int u) {
            if constexpr (H > 1) {
                // the sums of both halves
                if (half == 1) {
                    s_sum[r] = l;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&b_l[2 + rw]);
                }
                if (!warp_wait(&b_l[half ? rw : 2 + rw], td.seg)) return false;
                if (half == 0) {
                    l += s_sum[r];
                    s_sum[r] = l;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&b_l[rw]);
                } else {
                    l = s_sum[r];
                }
            }
            if (!warp_wait(&b_pv[u & 1], u >> 1)) return false;
            tc_fence_after();
            const int h = td.g / p.row_blocks;
            const float M = m == -INFINITY ? -INFINITY : m * c2 - kTail4;
            const float vs = p.v_scale ? __ldg(p.v_scale + h) : 1.f;
            const float f = l == 0.f ? 0.f : vs / l;
            uint32_t nan = 0;  // blocks of 16 dimensions that a NaN reached
            if (s_odd[td.seg & 7] == td.seg + 1 && row.live) {
                auto look = [&](int j0, int j1) {
                    for (int j = max(j0, seg_start); j <= min(j1, td.start + TK - 1); ++j) {
                        const int pg = p.table[static_cast<long long>(td.b) * p.table_stride + (j >> p.page_shift)];
                        if (pg < 0 || pg >= p.num_pages || !key_seen(j, pr, p.window, p.sinks)) continue;
                        const uint8_t* s = kb.v + pg * kb.page_stride + h * kb.head_stride +
                                           static_cast<long long>(j & (p.page_size - 1)) * NB;
                        for (int k = 0; k < NB; ++k)
                            if ((s[k] & 0x7fu) == 0x7fu) nan |= 1u << k;
                    }
                };
                // the ends of the rows' windows, then the verify rows themselves
                if (p.window > 0) look(max(0, td.p0 - p.window + 1), min(td.p0, td.len - 1 - p.window));
                look(max(0, td.p0 + 1), td.len - 1);
            }
            const long long orow = static_cast<long long>(td.b) * p.R + row.i;
            __nv_bfloat16* out = p.out + orow * p.ldo + static_cast<long long>(row.hq) * D;
            float* po = p.partial + static_cast<long long>(td.slot < 0 ? 0 : td.slot) * ROWS * (D + 2);
            __syncwarp();
#pragma unroll 1
            for (int c = half * (D / H); c < (half + 1) * (D / H); c += 32) {
                uint32_t y[32];
                tmem_ld32(y, tO + c);
                if (nan & (3u << (c / 16))) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if ((nan >> (c / 16 + k / 16)) & 1u) y[k] = 0x7fffffffu;
                }
                if (row.live) {
                    if (td.slot >= 0) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            *reinterpret_cast<uint4*>(po + r * D + c + 4 * k) =
                                make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = pack2<false>(__uint_as_float(y[8 * k + 2 * e]) * f,
                                                    __uint_as_float(y[8 * k + 2 * e + 1]) * f);
                            *reinterpret_cast<uint4*>(out + c + 8 * k) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
                __syncwarp();
            }
            if (row.live && half == 0) {
                if (td.slot >= 0) {
                    po[ROWS * D + r] = M;
                    po[ROWS * (D + 1) + r] = l;
                } else if (p.lse) {
                    p.lse[orow * p.Hq + row.hq] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b_o);
            return true;
        };

        bool ok = queries(0);
        for (int u = 0; u < n_units && ok; ++u) {
            ok = warp_wait(&b_s[u & 1], u >> 1);
            if (!ok) break;
            tc_fence_after();
            const AttnUnit td = s_unit[u % kUnitRing];
            const bool first = td.flags & kUnitFirst, edge = td.flags & kUnitEdge;
            if (first) {
                seg_start = td.start;
                row = row_next;
                pr = row.live ? td.p0 + row.i : -1;
                c2 = c2_next;
                l = 0.f;
            }
            const uint32_t tS = tmem + lanes + S::kColS + (u & 1) * TK;
            // seen: k <= hi and (k > lo or k < sk), as bits of the 32 columns from column c
            auto mask = [&](uint32_t* x, int c) {
                const int hi = pr - td.start - c;
                auto below = [](int n) {  // bits 0 .. n - 1
                    return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u);
                };
                uint32_t seen = below(hi + 1);
                if (p.window > 0) seen &= ~below(hi - p.window + 1) | below(p.sinks - td.start - c);
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    if (!((seen >> k) & 1u)) x[k] = 0xff800000u;
            };
            // half a row is read once, a whole one twice, 32 columns at a time
            constexpr int CW = H > 1 ? TK / H : 32;
            uint32_t x[CW];
            auto columns = [&](int c) {
                if constexpr (CW == 64) tmem_ld64(x, tS + c);
                else tmem_ld32(x, tS + c);
                if (edge) {
#pragma unroll
                    for (int k = 0; k < CW; k += 32) mask(x + k, c + k);
                }
            };
            const int c0 = half * CW, c1 = H > 1 ? c0 + CW : TK;
            float mx = -INFINITY;
#pragma unroll 1
            for (int c = c0; c < c1; c += CW) {
                columns(c);
                float m1 = -INFINITY;
#pragma unroll
                for (int k = 0; k < CW; k += 2) {
                    mx = fmaxf(mx, __uint_as_float(x[k]));
                    m1 = fmaxf(m1, __uint_as_float(x[k + 1]));
                }
                mx = fmaxf(mx, m1);
            }
            if constexpr (H > 1) {
                s_mx[u & 1][half][r] = mx;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b_x[u & 1][half * 2 + rw]);
                ok = warp_wait(&b_x[u & 1][(half ^ 1) * 2 + rw], u >> 1);
                if (!ok) break;
                tc_fence_after();
                mx = fmaxf(mx, s_mx[u & 1][half ^ 1][r]);
            }
            bool grow = false;
            float corr = 1.f;
            if (first) {
                m = mx;
            } else if (row.live && (mx - m) * c2 > kLazy4) {  // (the other rows hold anything)
                // (m = -infinity: O and l are zeros still)
                if (m != -INFINITY) {
                    corr = ex2((m - mx) * c2);
                    grow = true;
                }
                l *= corr;
                m = mx;
            }
            if (__any_sync(0xffffffffu, grow)) {
                ok = warp_wait(&b_pv[(u - 1) & 1], (u - 1) >> 1);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = half * (D / H); c < (half + 1) * (D / H); c += 32) {
                    uint32_t y[32];
                    tmem_ld32(y, tO + c);
#pragma unroll
                    for (int k = 0; k < 32; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * corr);
                    tmem_st32(tO + c, y);
                }
            }
            const float mc = m == -INFINITY ? 0.f : m * c2 - kTail4;
            float s0 = 0.f, s1 = 0.f;
#pragma unroll 1
            for (int c = c0; c < c1; c += CW) {
                // (P's columns c / 2 .. hold scores that have been read)
                if (H == 1) columns(c);
                uint32_t y[CW / 2];
#pragma unroll
                for (int k = 0; k < CW; k += 2) {
                    const float a = ex2(fmaf(__uint_as_float(x[k]), c2, -mc));
                    const float b = ex2(fmaf(__uint_as_float(x[k + 1]), c2, -mc));
                    s0 += a;
                    s1 += b;
                    y[k / 2] = pack2<true>(a, b);
                }
                if constexpr (CW == 64) tmem_st32(tS + c / 2, y);
                else tmem_st16(tS + c / 2, y);
            }
            l += s0 + s1;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b_p[u & 1]);
            if (!(td.flags & kUnitLast)) continue;
            // the next part's queries first: its scores wait for them, not for these rows
            if (u + 1 < n_units) ok = queries(td.seg + 1);
            if (ok) ok = finish(td, u);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kTc4Mma) {
        tc_fence_after();
        tmem_dealloc<512>(tmem);
    }
}

template <int D, int ROWS>
cudaError_t attn4_tc_launch(const AttnParams& p, const Kv4Blocks& kb, const AttnMaps& maps, int* grid,
                            int sms, cudaStream_t s) {
    using S = Attn4TcShape<D, ROWS>;
    static std::atomic<unsigned long long> once;
    auto* kernel = attn4_tc_kernel<D, ROWS>;
    const cudaError_t e = set_attribute_per_device(once, [] {
        return cudaFuncSetAttribute(attn4_tc_kernel<D, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    S::kSmem);
    });
    if (e != cudaSuccess) return e;
    if (*grid > sms) *grid = sms;
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
#endif  // __CUDACC__

}  // namespace vw4
