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
// HBM 0.4).  The exponentials are 0.5 of it: tensor memory's lanes bind a block of up to 64 rows
// to two of the four sub-cores.  Without conversions and exponentials a tile still takes 1.1 us
// of its 1.4; a second issuing thread, for the other product, changes nothing.  So
// the time hardly grows with the rows: 32 sequences of up to 32768 tokens, 4 key heads of
// size 128 (219 MB), are 112 us at 36 rows, 117 at 64 and 150 at 128; head size 256 182 / 192 /
// 260.  Tried and slower: weights formed at once against the lagging reference (252 us
// against 235 at 64 rows of 8 heads), the rows' copies in the other lanes so that every
// sub-core has softmax warps (332), keys as the rows of the instructions and eight warps of
// weights through shared memory (541).
//
// What happens once a part of an item, its queries and its rows, is code that no instruction
// cache holds yet: divisions once a row, rows handed on by shuffles and maxima of pairs took
// 8 rows of 6 heads of 4 sequences from 33 to 28.5 us, windows of 1024 from 92 to 70.
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
    static constexpr int kOffX = kOffRawV + kNR * kRaw;  // 4 KB a softmax warp
    static constexpr int kUsed = kOffX + 4 * 4096 + 1024;
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

__device__ __forceinline__ void tmem_ld16(uint32_t* r, uint32_t a) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
          "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
          "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(a)
        : "memory");
}

struct Attn4TcRow {
    float c2, vs;
    int at;  // verify index << 16 | head (dead: -1)
};

// What the warps of a CTA share beside the tiles.
template <int D, int ROWS>
struct Attn4TcShared {
    using S = Attn4TcShape<D, ROWS>;
    static constexpr int NR = S::kNR, NF = S::kNF, H = S::kHalves;
    uint32_t s_tmem;
    volatile int s_abort;
    volatile int s_odd[8];            // seg + 1: the part's values lost NaN
    AttnUnit s_unit[kUnitRing], s_vunit[kUnitRing], s_part[16];
    float s_mx[2][2][H > 1 ? ROWS : 1];  // of a tile's columns, for the other half
    Attn4TcRow s_row[2][H][ROWS];        // of a part, by seg & 1: each thread its own
    float s_sum[H > 1 ? ROWS : 1];       // of a part's weights
    uint32_t s_top[2][H > 1 ? ROWS : 1]; // of the queries' halves: largest magnitudes
    uint64_t b_rk[NR], b_rke[NR], b_rv[NR], b_rve[NR];
    uint64_t b_k[NF], b_ke[NF], b_v[NF], b_ve[NF];
    uint64_t b_s[2], b_p[2], b_pv[2], b_q[2], b_qe[2], b_part[16], b_o, b_end;
    uint64_t b_x[2][4];     // s_mx of a half's warp is there
    uint64_t b_l[4], b_t[4];  // s_sum and s_top of a half's warp are there
};

struct Attn4TcWarp {
    int half, rw, r, lane;
    uint32_t tmem;
    uint8_t* stage;  // 16 bytes of 32 rows of 128: eight lanes take a row, or a lane its own
};

// (the same answer in every lane: what follows is executed by whole warps)
template <class Shared>
__device__ __forceinline__ bool attn4_tc_wait(const AttnParams& p, Shared& sh, uint64_t* bar, int phase) {
    bool ok = mbar_wait_bounded(bar, phase & 1, p.wait_ns, &sh.s_abort);
    if (!ok) {
        sh.s_abort = 1;
        atomicOr(p.status, kStatusWaitTimeout);
    }
    return __all_sync(0xffffffffu, ok) != 0;
}

// An item's queries into tensor memory: f16 under a power of two per row that puts its
// largest magnitude into [2^14, 2^15), with the sign of the head's scale.  Eight lanes
// read 64 dimensions of a row.  The halves take every other 64, all read at once, and
// exchange their magnitudes; a thread of a whole row reads it twice.
template <int D, int ROWS>
__device__ __forceinline__ bool attn4_tc_queries(const AttnParams& p, Attn4TcShared<D, ROWS>& sh, const Attn4TcWarp& w,
                                              int seg) {
    using S = Attn4TcShape<D, ROWS>;
    constexpr int NQ = S::kNQ, H = S::kHalves;
    const int half = w.half, rw = w.rw, r = w.r, lane = w.lane;
    const uint32_t lanes = static_cast<uint32_t>(rw * 32) << 16, tmem = w.tmem;
    auto& s_part = sh.s_part;
    auto& s_row = sh.s_row;
    auto& s_top = sh.s_top;
    auto& b_q = sh.b_q;
    auto& b_qe = sh.b_qe;
    auto& b_part = sh.b_part;
    auto& b_t = sh.b_t;
    uint4* stage = reinterpret_cast<uint4*>(w.stage);
    auto x_at = [](int row, int chunk) { return row * 8 + (chunk ^ (row & 7)); };
    auto warp_wait = [&](uint64_t* bar, int phase) { return attn4_tc_wait(p, sh, bar, phase); };
    if (!warp_wait(&b_part[seg & 15], seg >> 4)) return false;
    const AttnUnit d = s_part[seg & 15];
    const int h = d.g / p.row_blocks;
    const float ks = p.k_scale ? __ldg(p.k_scale + h) : 1.f;
    const float vs = p.v_scale ? __ldg(p.v_scale + h) : 1.f;
    const AttnRow own = attn_row(p, d.g, r);
    const int at = own.live ? own.i << 16 | own.hq : -1;
    const uint4* src[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int a = __shfl_sync(0xffffffffu, at, 4 * j + (lane >> 3));
        src[j] = a >= 0 ? reinterpret_cast<const uint4*>(
                              p.q + (static_cast<long long>(d.b) * p.R + (a >> 16)) * p.ldq +
                              static_cast<long long>(a & 0xffff) * D) + (lane & 7)
                        : nullptr;
    }
    auto read = [&](uint4* v, int c) {  // 64 dimensions
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = src[j] ? __ldg(src[j] + c * 8) : make_uint4(0, 0, 0, 0);
    };
    constexpr int NC = (D / 64 + H - 1) / H;  // of a half
    uint4 all[H > 1 ? NC : 1][8];
    uint32_t mx[8] = {};
    auto largest = [&](const uint4* v) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[j] = __vmaxu2(mx[j], w[e] & 0x7fff7fffu);
        }
    };
    if constexpr (H > 1) {
#pragma unroll
        for (int k = 0; k < NC; ++k)
            if (half + k * H < D / 64) read(all[k], half + k * H);
#pragma unroll
        for (int k = 0; k < NC; ++k)
            if (half + k * H < D / 64) largest(all[k]);
    } else {
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
            read(all[0], c);
            largest(all[0]);
        }
    }
    uint32_t top = 0;  // of the lane's own row
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int s = 4; s > 0; s >>= 1) mx[j] = __vmaxu2(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], s));
        const uint32_t t = __shfl_sync(0xffffffffu, mx[j], (lane & 3) * 8);
        if (lane >> 2 == j) top = t;
    }
    if constexpr (H > 1) {
        s_top[half][r] = top;
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_t[half * 2 + rw]);
        if (!warp_wait(&b_t[(half ^ 1) * 2 + rw], seg)) return false;
        top = __vmaxu2(top, s_top[half ^ 1][r]);
    }
    top = max(top & 0xffffu, top >> 16);
    const int ex = static_cast<int>(top >> 7);
    int shift = ex == 0 || ex == 255 ? 0 : 127 + 14 - ex;
    shift = max(-126, min(126, shift));
    const float up = copysignf(__uint_as_float(static_cast<uint32_t>(127 + shift) << 23), ks);
    float c = p.scale * kLog2e * fabsf(ks) * __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
    if (c < kMinFactor) c = kMinFactor;  // (NaN stays)
    s_row[seg & 1][half][r] = {c, vs, at};
    if (seg >= NQ && !warp_wait(&b_qe[seg % NQ], seg / NQ - 1)) return false;
    tc_fence_after();
    const uint32_t tq = tmem + lanes + S::kColQ + seg % NQ * (D / 2);
    auto bring = [&](const uint4* v, int c) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) stage[x_at(4 * j + (lane >> 3), lane & 7)] = v[j];
        __syncwarp();
        uint32_t y[32];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint4 x = stage[x_at(lane, k)];
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y[4 * k + e] = pack2<true>(__uint_as_float(w[e] << 16) * up,
                                           __uint_as_float(w[e] & 0xffff0000u) * up);
        }
        tmem_st32(tq + c * 32, y);
    };
    if constexpr (H > 1) {
#pragma unroll
        for (int k = 0; k < NC; ++k)
            if (half + k * H < D / 64) bring(all[k], half + k * H);
    } else {
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
            read(all[0], c);
            bring(all[0], c);
        }
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&b_q[seg % NQ]);
    return true;
}

// A part's rows from tensor memory to the output, or to its partial.
template <int D, int ROWS>
__device__ __forceinline__ bool attn4_tc_finish(const AttnParams& p, const Kv4Blocks& kb, Attn4TcShared<D, ROWS>& sh,
                                             const Attn4TcWarp& w, const AttnUnit& td, int u, int seg_start,
                                             int pr, bool live, float m, float l, float c2) {
    using S = Attn4TcShape<D, ROWS>;
    constexpr int H = S::kHalves, NB = S::kNB, TK = S::kTK;
    const int half = w.half, rw = w.rw, r = w.r, lane = w.lane;
    const uint32_t tO = w.tmem + (static_cast<uint32_t>(rw * 32) << 16);
    auto& s_odd = sh.s_odd;
    auto& s_row = sh.s_row;
    auto& s_sum = sh.s_sum;
    auto& b_pv = sh.b_pv;
    auto& b_o = sh.b_o;
    auto& b_l = sh.b_l;
    uint4* stage = reinterpret_cast<uint4*>(w.stage);
    auto x_at = [](int row, int chunk) { return row * 8 + (chunk ^ (row & 7)); };
    auto warp_wait = [&](uint64_t* bar, int phase) { return attn4_tc_wait(p, sh, bar, phase); };
    const float vs = s_row[td.seg & 1][half][r].vs;
    const int row_at = s_row[td.seg & 1][half][r].at;
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
    const float M = attn4_ref(m, c2);
    const float f = l == 0.f ? 0.f : vs / l;
    uint32_t nan = 0;  // blocks of 16 dimensions that a NaN reached
    if (s_odd[td.seg & 7] == td.seg + 1 && live) {
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
    int at[8];  // verify index << 16 | head of the rows that this lane writes (dead: -1)
#pragma unroll
    for (int j = 0; j < 8; ++j) at[j] = __shfl_sync(0xffffffffu, row_at, 4 * j + (lane >> 3));
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
        // through shared memory, so that eight lanes write a row's 32 columns
        const float to = td.slot >= 0 ? 1.f : f;
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k)
            stage[x_at(lane, k)] = make_uint4(__float_as_uint(__uint_as_float(y[4 * k]) * to),
                                              __float_as_uint(__uint_as_float(y[4 * k + 1]) * to),
                                              __float_as_uint(__uint_as_float(y[4 * k + 2]) * to),
                                              __float_as_uint(__uint_as_float(y[4 * k + 3]) * to));
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int q = 4 * j + (lane >> 3), col = c + (lane & 7) * 4;
            const uint4 x = stage[x_at(q, lane & 7)];
            if (at[j] < 0) {
            } else if (td.slot >= 0) {
                *reinterpret_cast<uint4*>(po + (rw * 32 + q) * D + col) = x;
            } else {
                *reinterpret_cast<uint2*>(
                    p.out + (static_cast<long long>(td.b) * p.R + (at[j] >> 16)) * p.ldo +
                    static_cast<long long>(at[j] & 0xffff) * D + col) =
                    make_uint2(pack2<false>(__uint_as_float(x.x), __uint_as_float(x.y)),
                               pack2<false>(__uint_as_float(x.z), __uint_as_float(x.w)));
            }
        }
    }
    if (live && half == 0) {
        if (td.slot >= 0) {
            po[ROWS * D + r] = M;
            po[ROWS * (D + 1) + r] = l;
        } else if (p.lse) {
            p.lse[(static_cast<long long>(td.b) * p.R + (row_at >> 16)) * p.Hq + (row_at & 0xffff)] =
                l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
        }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&b_o);
    return true;
}

template <int D, int ROWS>
__global__ void __launch_bounds__(Attn4TcShape<D, ROWS>::kThreads, 1)
    attn4_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ Kv4Blocks kb,
                    const __grid_constant__ AttnMaps maps) {
    using S = Attn4TcShape<D, ROWS>;
    constexpr int TK = S::kTK, NR = S::kNR, NF = S::kNF, NQ = S::kNQ, H = S::kHalves, NB = S::kNB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ Attn4TcShared<D, ROWS> sh;
    auto& s_tmem = sh.s_tmem;
    auto& s_abort = sh.s_abort;
    auto& s_odd = sh.s_odd;
    auto& s_unit = sh.s_unit;
    auto& s_vunit = sh.s_vunit;
    auto& s_part = sh.s_part;
    auto& s_mx = sh.s_mx;
    auto& s_row = sh.s_row;
    auto& b_rk = sh.b_rk;
    auto& b_rke = sh.b_rke;
    auto& b_rv = sh.b_rv;
    auto& b_rve = sh.b_rve;
    auto& b_k = sh.b_k;
    auto& b_ke = sh.b_ke;
    auto& b_v = sh.b_v;
    auto& b_ve = sh.b_ve;
    auto& b_s = sh.b_s;
    auto& b_p = sh.b_p;
    auto& b_pv = sh.b_pv;
    auto& b_q = sh.b_q;
    auto& b_qe = sh.b_qe;
    auto& b_part = sh.b_part;
    auto& b_o = sh.b_o;
    auto& b_end = sh.b_end;
    auto& b_x = sh.b_x;
    auto& b_l = sh.b_l;
    auto& b_t = sh.b_t;
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
            for (int k = 0; k < 4; ++k) {
                mbar_init(&b_l[k], 1);
                mbar_init(&b_t[k], 1);
            }
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
    auto warp_wait = [&](uint64_t* bar, int phase) { return attn4_tc_wait(p, sh, bar, phase); };

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
        float m = -INFINITY, l = 0.f, c2 = 1.f;
        bool live = false;
        int pr = -1, seg_start = 0;

        const Attn4TcWarp w{half, rw, r, lane, tmem, smem + S::kOffX + (half * (4 / H) + rw) * 4096};
        bool ok = true;
        AttnUnit td{};
        for (int u = -1; ok;) {
            // ---- between parts: the next one's queries first, for its scores wait for them,
            // not for these rows
            if (u + 1 < n_units) ok = attn4_tc_queries<D, ROWS>(p, sh, w, u < 0 ? 0 : td.seg + 1);
            if (ok && u >= 0)
                ok = attn4_tc_finish<D, ROWS>(p, kb, sh, w, td, u, seg_start, pr, live, m, l, c2);
            if (!ok || u + 1 >= n_units) break;
            do {
                ++u;
                ok = warp_wait(&b_s[u & 1], u >> 1);
                if (!ok) break;
                tc_fence_after();
                td = s_unit[u % kUnitRing];
                const bool first = td.flags & kUnitFirst, edge = td.flags & kUnitEdge;
                if (first) {
                    seg_start = td.start;
                    const Attn4TcRow& a = s_row[td.seg & 1][half][r];
                    c2 = a.c2;
                    live = a.at >= 0;
                    pr = live ? td.p0 + (a.at >> 16) : -1;
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
                } else if (live && (mx - m) * c2 > kLazy4) {  // (the other rows hold anything)
                    // (m = -infinity: O and l are zeros still)
                    if (m != -INFINITY) {
                        corr = ex2(attn4_ref(m, c2) - attn4_ref(mx, c2));
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
                    for (int c = half * (D / H); c < (half + 1) * (D / H); c += 16) {  // (beside the scores)
                        uint32_t y[16];
                        tmem_ld16(y, tO + c);
#pragma unroll
                        for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * corr);
                        tmem_st16(tO + c, y);
                    }
                }
                const float mc = m == -INFINITY ? 0.f : attn4_ref(m, c2);
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
            } while (!(td.flags & kUnitLast));
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
