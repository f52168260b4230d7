// attn_tc.cuh -- the attention of more than 16 query rows of a key head on the
// 5th-generation tensor cores: the same units, partials and results as
// attn_kernel (attn.cuh).
//
// One CTA per SM, warps with roles.  Two producer warps load tiles of 128 keys
// (TMA) into two rings in the swizzled layout the tensor cores read, one of K
// pieces and one of V pieces (a piece is the whole tile, or at head size 256
// half of K's dimensions; of V 32, 64 or all 128 keys).  One thread
// issues S = Q K^T and O += P V piece by piece, whichever has its operands first.
// (An elected one: chosen by its lane number it took twice as long over each product,
// e4m3 of head size 128 136 us against 114.)
// The softmax warps own one query row a thread, so the softmax has no shuffles,
// and S and P never pass through shared memory.  S has two buffers: Q K^T of the
// next tile runs under the softmax of this one; P overwrites the front of its S.  (A
// third, for which head size 64 has the room, changed nothing.)
// Q lies in tensor memory where O (D columns), the S (128 each) and two Q fit its 512
// columns, else (head size 256) in shared memory: tiles of 64 keys would make
// room, but the products of 64 columns run at half the rate of those of 128.
//
// Four warps bring an item's queries to their place and write the rows of the item
// before, while the softmax warps are on with the next; four pass V on, cleaned
// where not every row sees every key: together for bf16 (most tiles need nothing),
// for e4m3 a piece each, turned into f16 (exact) in a third ring: a piece is more
// latency than work, so several go on at once.
//
// e4m3 keys are multiplied as they are (kind::f8f6f4); a query row, scaled by a
// power of two that puts its largest magnitude into [2^7, 2^8), is the sum of two
// e4m3 terms, its nearest value and that of the rest: 4 + 4 significant bits, so
// exact for a bf16 value down to 2^-10 of the largest and off by at most 2^-17 of
// the largest below.  For the weights two such terms would not do: a long tail of
// small weights under one large one lies below their range.  So P is f16, times 2^6,
// and V becomes f16; converting K as well was bound by that step.
//
// What bounds it.  bf16: the bytes (8 key heads of 128, 24 rows each, 32 sequences of
// 4000 .. 8000 tokens: 130 us, 87 % of the copy rate).  e4m3 halves the bytes but not
// the work: at head size 256 shared memory's bandwidth (K is read twice for the two
// terms, V once raw, written and read as f16: about 1.5 us of a tile of 128 keys
// against 1.4 for its bytes) and the chain of V's conversion; at 128 and 64 the chain
// scores - softmax - P V, about 1 us a tile.
//
// The running maximum that the exponents use follows the true one lazily: O is
// rescaled only when a row's maximum grew by more than 2^8 (its weights are then
// at most 2^8, e4m3 caches 2^14, harmless in bf16, f16 and the fp32 sum).
#pragma once
#include "attn.cuh"

namespace vw4 {
#ifdef __CUDACC__

template <int D, bool F8, int ROWS>
struct AttnTcShape {
    static constexpr int kTK = 128;                  // keys of a tile
    static constexpr int kES = F8 ? 1 : 2;           // bytes of an element in memory
    static constexpr int kBoxB = D * kES < 128 ? D * kES : 128;  // bytes of a key in a box
    // K: pieces of kKBlks blocks of kBoxB bytes of a key
    static constexpr int kKP = D == 256 ? 2 : 1;
    static constexpr int kKBlks = D * kES / kKP / kBoxB;
    static constexpr int kAtom = 8 * kBoxB;          // 8 keys of a block
    static constexpr int kKPiece = kTK / 8 * kKBlks * kAtom;
    static constexpr int kSteps = kBoxB / 32;        // k steps (32 bytes) of a block
    static constexpr int kTerms = F8 ? 2 : 1;        // of Q
    // V: pieces of kVKeys keys, as loaded and as multiplied (16-bit, blocks of 64 dimensions)
    static constexpr int kVP = D < 256 ? (F8 && D == 128 ? 2 : 1) : (F8 ? 4 : 2);
    static constexpr int kVKeys = kTK / kVP;
    static constexpr int kVBlks = D * kES / kBoxB;
    static constexpr int kVLoad = kVKeys * D * kES;
    static constexpr int kVPiece = kVKeys * D * 2;
    static constexpr int kVBlk = kVKeys * 128;
    static constexpr bool kQSmem = D == 256;
    static constexpr int kQRow = D * kES;            // bytes of a term of a query row
    static constexpr int kQBlk = ROWS * kBoxB;
    static constexpr int kQ = kQSmem ? ROWS * D * 2 : 0;
    static constexpr int kNQ = kQSmem ? 1 : 2;       // query buffers
    static_assert(!(F8 && D == 256 && ROWS > 64), "blocks of 64 rows");
    static constexpr int kNK = F8 ? (D == 64 ? 6 : (D == 128 ? 4 : 3)) : (D == 64 ? 4 : (D == 128 ? 3 : 2));
    static constexpr int kNV = F8 ? (D == 256 ? 4 : 8) : (D == 64 ? 4 : (D == 128 || ROWS == 64 ? 3 : 2));
    static constexpr int kNF = !F8 ? 0 : (D == 256 ? 6 : 4);  // f16 pieces
    static constexpr int kPass = 4;                  // warps that pass V on
    // e4m3: each takes every kPass-th piece, and loads may land out of order.  A place of
    // the ring has to be one warp's, or a warp could wait for its next piece while the
    // place still waits for the one before, whose phase has the same parity as the one
    // two before that: over, it would seem.
    static_assert(!F8 || kNV % kPass == 0, "a place of the V ring belongs to one warp");
    // (a place of the f16 ring is waited for in the order of the products, which ends the
    // phase before: the warp's piece before was free of piece pc - kPass)
    static_assert(!F8 || kNF >= kPass, "f16 ring");
    static constexpr int kThreads = 16 * 32;
    static constexpr int kHalves = D == 64 && ROWS == 64 ? 2 : 1;  // threads of a softmax row
    static constexpr int kLoadV = kHalves > 1 ? 2 : 5, kLoadK = kHalves > 1 ? 3 : 6;  // warps
    static constexpr int kOffK = kQ;
    static constexpr int kOffV = kOffK + kNK * kKPiece;
    static constexpr int kOffF = kOffV + kNV * kVLoad;
    static constexpr int kOffStage = kOffF + kNF * kVPiece;    // 4 KB a softmax warp, for the output
    static constexpr int kUsed = kOffStage + ROWS / 32 * 4096 + 1024;  // and alignment
    static constexpr int kSmem = kUsed < 115 * 1024 ? 115 * 1024 : kUsed;  // one CTA per SM
    static_assert(kSmem + 5632 <= 227 * 1024, "shared memory");
    // the products read 128 rows of Q whatever ROWS is: what follows must be there
    static_assert(!kQSmem || kOffStage >= (kTerms * kQRow / kBoxB - 1) * kQBlk + 128 * kBoxB, "Q reads");
    // tensor memory columns: O, the S, the queries (two 16-bit values a column)
    static constexpr int kNS = 2;                    // score buffers
    static constexpr uint32_t kColO = 0, kColS = D, kColQ = D + kNS * kTK;
    static_assert(D + kNS * kTK + (kQSmem ? 0 : kNQ * D / 2) <= 512, "tensor memory");
    // 16 bytes of a key of a V piece as it is loaded
    __device__ static __forceinline__ uint32_t v_at(int row, int chunk) {
        return static_cast<uint32_t>((row >> 3) * kVBlks * kAtom) +
               at<kBoxB>(kAtom, row & 7, chunk);
    }
    // 16 bytes of a row: blocks of blk bytes, rows of BOXB bytes in them
    template <int BOXB>
    __device__ static __forceinline__ uint32_t at(int blk, int row, int chunk) {
        constexpr int CPB = BOXB / 16;
        const int x = BOXB == 64 ? (row >> 1) & 3 : row & 7;
        return static_cast<uint32_t>(chunk / CPB * blk + row * BOXB + (((chunk % CPB) ^ x) << 4));
    }
};

constexpr float kLazy = 8.f;  // (log2) see above

// Warps: 0 .. 3 softmax, 8 .. 11 queries, 12 .. 15 pass V on.  At head size 64 the softmax
// of one row a thread is the longest step; blocks of 64 rows leave warps 2 and 3 without
// rows, and warps 4 and 5, which reach the same lanes of tensor memory as 0 and 1, take
// half of the columns there (e4m3, 32 sequences of 4000 .. 8000 tokens, 8 key heads, 32
// rows each: 87 us instead of 98).  At 128 and 256 the products and V's conversion are as
// long: 115 instead of 114 us, and 62 instead of 57 with a window of 1024.
// The loading warps (one each for K and V: a box costs its warp some 60 ns, and a tile
// of 16-token pages has 32) and the one that issues the products (it polls) share
// schedulers with the softmax warps that only the largest blocks use.
constexpr int kTcMma = 7, kTcQ = 8, kTcPass = 12;

template <int D, bool F8, int ROWS>
__global__ void __launch_bounds__(AttnTcShape<D, F8, ROWS>::kThreads, 1)
    attn_tc_kernel(const AttnParams p, const __grid_constant__ AttnMaps maps) {
    using S = AttnTcShape<D, F8, ROWS>;
    constexpr int TK = S::kTK, NK = S::kNK, NV = S::kNV, NF = F8 ? S::kNF : 1;
    constexpr int KP = S::kKP, VP = S::kVP, H = S::kHalves, NS = S::kNS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    __shared__ volatile int s_odd[8];  // seg + 1: the part's values lost infinities or NaN
    __shared__ AttnUnit s_unit[kUnitRing], s_vunit[kUnitRing];  // by the K and the V warp
    __shared__ AttnUnit s_part[8];     // first units of the parts
    __shared__ AttnUnit s_end[2];      // a part's last unit (its start: the first unit's)
    __shared__ int s_end_u[2], s_end_start[2];  // its number, its first key
    __shared__ float2 s_ml[2][H][ROWS];  // maximum and sum of a part's rows
    __shared__ float s_mx[2][H][H > 1 ? ROWS : 1];  // of a tile's columns, for the other half
    __shared__ volatile int s_parts;   // how many parts, once it is known
    // A wait names a phase by its parity: when it begins, the phase before has to be over
    // and the one after not.  So products and scores have NS barriers each, taken in
    // turn: S of tile u is committed after the product of tile u - NS.
    // Loaded pieces and their release; V pieces passed on (bf16) or as f16 and released.
    __shared__ __align__(8) uint64_t b_k[NK], b_ke[NK], b_v[NV], b_ve[NV], b_clean[8], b_fe[NF];
    __shared__ __align__(8) uint64_t b_s[NS], b_p[NS], b_pv[NS], b_q[2], b_qe[2], b_part[8], b_ml[2];
    __shared__ __align__(8) uint64_t b_o, b_end;
    __shared__ __align__(8) uint64_t b_x[2][4];  // s_mx of a half's warp is there, S read
    // log2 of the row scales of e4m3 queries, by part: those of part n + 8 are written
    // after the last scores of part n + 6, which wait for the softmax of part n + 3
    __shared__ int8_t s_rs[F8 ? 8 : 1][F8 ? ROWS : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row_warps = (p.tb * p.gb + 31) / 32;     // softmax warps with rows

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == S::kLoadK * 32) {
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
        if (S::kQSmem && !F8) tma_prefetch_desc(&maps.q);
    }
    if (warp == kTcMma) {
        tmem_alloc<512>(&s_tmem);
        if (lane == 0) {
            for (int k = 0; k < NK; ++k) {
                mbar_init(&b_k[k], 1);
                mbar_init(&b_ke[k], 1);
            }
            for (int k = 0; k < NV; ++k) {
                mbar_init(&b_v[k], 1);
                mbar_init(&b_ve[k], 1);
            }
            for (int k = 0; k < NF; ++k) mbar_init(&b_fe[k], 1);
            for (int k = 0; k < NS; ++k) {
                mbar_init(&b_s[k], 1);
                mbar_init(&b_pv[k], 1);
                mbar_init(&b_p[k], H * row_warps);
            }
            for (int k = 0; k < 2; ++k) {
                mbar_init(&b_ml[k], H * row_warps);
                for (int j = 0; j < 4; ++j) mbar_init(&b_x[k][j], 1);
                mbar_init(&b_q[k], S::kQSmem ? 4 : row_warps);
                mbar_init(&b_qe[k], 1);
            }
            for (int k = 0; k < 8; ++k) {
                mbar_init(&b_part[k], 1);
                mbar_init(&b_clean[k], F8 ? 1 : S::kPass);
            }
            mbar_init(&b_o, row_warps);
            mbar_init(&b_end, 1);
            fence_barrier_init();
            s_abort = 0;
            s_parts = 1 << 30;
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

    // An item's queries to their place.  e4m3: as two terms (see above); a row with an
    // infinity or NaN is made NaN, for e4m3 has no infinity.
    auto q_scale = [&](uint32_t largest, const AttnUnit& d, int r, bool keep, uint32_t sign) {
        const int ex = static_cast<int>(largest >> 7);  // of the largest magnitude, bf16 bits
        int sh = ex == 0 || ex == 255 ? 0 : 127 + 7 - ex;  // to [2^7, 2^8)
        sh = max(-126, min(126, sh));
        if (keep) s_rs[F8 ? d.seg & 7 : 0][F8 ? r : 0] = static_cast<int8_t>(sh);
        return ex == 255 ? NAN : __uint_as_float((static_cast<uint32_t>(127 + sh) << 23) | sign);
    };
    auto largest_of = [](uint32_t mx, const uint4& v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = max(mx, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
        return mx;
    };
    // 8 bf16 values as 8 bytes of either term
    auto two_terms = [](const uint4& v, float up, uint32_t* hi, uint32_t* lo) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; e += 2)
            e4m3_terms(pack2<true>(__uint_as_float(w[e] << 16) * up,
                                   __uint_as_float(w[e] & 0xffff0000u) * up),
                       pack2<true>(__uint_as_float(w[e + 1] << 16) * up,
                                   __uint_as_float(w[e + 1] & 0xffff0000u) * up),
                       hi[e / 2], lo[e / 2]);
    };
    auto queries = [&](const AttnUnit& d, int vw) {
        const int qs = d.seg % S::kNQ;
        const uint32_t sign =
            F8 && p.k_scale && __ldg(p.k_scale + d.g / p.row_blocks) < 0.f ? 0x80000000u : 0u;
        auto source = [&](const AttnRow& row) {
            return reinterpret_cast<const uint4*>(p.q +
                                                  (static_cast<long long>(d.b) * p.R + row.i) * p.ldq +
                                                  static_cast<long long>(row.hq) * D);
        };
        const bool reused = d.seg >= S::kNQ;
        if constexpr (S::kQSmem && !F8) {
            // (every warp arrives, after it has written the part two before)
            if (reused && !warp_wait(&b_qe[qs], d.seg / S::kNQ - 1)) return false;
            if (lane == 0) {
                if (vw == 0) {
                    mbar_arrive_expect_tx(&b_q[qs], attn_q_bytes(p, D));
                    attn_load_q<D>(p, &maps.q, sm, S::kQBlk, d, &b_q[qs]);
                } else {
                    mbar_arrive(&b_q[qs]);
                }
            }
            __syncwarp();
        } else if constexpr (S::kQSmem) {
            // a warp a row, a lane 8 dimensions; the first rows are on their way while the
            // last products of the part before are waited for
            constexpr int W = 4, AHEAD = 8;
            const int rows = p.tb * p.gb;
            uint4 v[AHEAD];
            for (int r0 = vw; r0 < rows; r0 += W * AHEAD) {
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    const int r = r0 + k * W;
                    const AttnRow row = attn_row(p, d.g, r);
                    v[k] = r < rows && row.live ? __ldg(source(row) + lane) : make_uint4(0, 0, 0, 0);
                }
                if (r0 == vw && reused && !warp_wait(&b_qe[qs], d.seg / S::kNQ - 1)) return false;
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    const int r = r0 + k * W;
                    if (r >= rows) break;
                    const uint32_t mx = __reduce_max_sync(0xffffffffu, largest_of(0u, v[k]));
                    uint32_t hi[2], lo[2];
                    two_terms(v[k], q_scale(mx, d, r, lane == 0, sign), hi, lo);
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        *reinterpret_cast<uint2*>(
                            smem + S::template at<S::kBoxB>(S::kQBlk, r, t * (D / 16) + lane / 2) +
                            (lane & 1) * 8) = t ? make_uint2(lo[0], lo[1]) : make_uint2(hi[0], hi[1]);
                }
            }
            if (vw >= rows && reused && !warp_wait(&b_qe[qs], d.seg / S::kNQ - 1)) return false;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b_q[qs]);
        } else if (vw < row_warps) {
            // a row a thread (a warp reaches lanes 32 (warp % 4) .. of tensor memory)
            const int r = vw * 32 + lane;
            const AttnRow row = attn_row(p, d.g, r);
            const uint4* src = source(row);
            uint4 v[D / 8];
#pragma unroll
            for (int k = 0; k < D / 8; ++k) v[k] = row.live ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
            float up = 1.f;
            if (F8) {
                uint32_t mx = 0;
#pragma unroll
                for (int k = 0; k < D / 8; ++k) mx = largest_of(mx, v[k]);
                up = q_scale(mx, d, r, r < ROWS, sign);
            }
            if (reused && !warp_wait(&b_qe[qs], d.seg / S::kNQ - 1)) return false;
            tc_fence_after();
            const uint32_t tq = tmem + (static_cast<uint32_t>(vw * 32) << 16) + S::kColQ + qs * (D / 2);
            __syncwarp();  // (rows that are not live took another way)
#pragma unroll
            for (int c = 0; c < D / 8; c += 8) {  // 64 dimensions
                uint32_t y[32];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (F8) {  // hi: y[0 .. 15], lo: y[16 .. 31]
                        two_terms(v[c + k], up, y + 2 * k, y + 16 + 2 * k);
                    } else {
                        y[4 * k] = v[c + k].x;
                        y[4 * k + 1] = v[c + k].y;
                        y[4 * k + 2] = v[c + k].z;
                        y[4 * k + 3] = v[c + k].w;
                    }
                }
                if (F8) {
                    tmem_st16(tq + c * 2, y);
                    tmem_st16(tq + D / 4 + c * 2, y + 16);
                } else {
                    tmem_st32(tq + c * 4, y);
                }
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b_q[qs]);
        }
        return true;
    };

    // A part's rows from tensor memory to the output, or to its partial.
    auto finish = [&](int part, int vw) {
        const int r = vw * 32 + lane;  // row of the block = lane of tensor memory
        const uint32_t tO = tmem + (static_cast<uint32_t>(vw * 32) << 16) + S::kColO;
        if (!warp_wait(&b_ml[part & 1], part >> 1)) return false;
        const AttnUnit td = s_end[part & 1];
        const int u = s_end_u[part & 1], h = td.g / p.row_blocks;
        const AttnRow row = attn_row(p, td.g, r);
        const int pr = row.live ? td.p0 + row.i : -1;
        float2 ml = s_ml[part & 1][0][min(r, ROWS - 1)];
        if (H > 1) ml.y += s_ml[part & 1][H - 1][min(r, ROWS - 1)].y;
        const float mm = ml.x, l = ml.y;
        // S of tile u was committed after the product of tile u - NS (see the barriers)
        if (!warp_wait(&b_pv[u % NS], u / NS)) return false;
        tc_fence_after();
        const int last_key = s_end_start[part & 1] + TK - 1;
        const bool live = row.live, odd = s_odd[part & 7] == part + 1;
        const float vs = F8 && p.v_scale ? __ldg(p.v_scale + h) : 1.f;
        const float f = td.slot >= 0 ? 1.f : (l == 0.f ? 0.f : vs / l);
        const long long orow = static_cast<long long>(td.b) * p.R + row.i;
        // The rows leave through 4 KB of shared memory a warp, 128 bytes of each of
        // the 32 rows at a time (fp32 partial: 32 columns, bf16: 64), so that eight
        // lanes write one row's line.
        // Rows are passed round as offsets in 16 bytes (they start on 16) from the sequence's
        // first row, or the partial's: 15 strides of at most 2^32 bytes fit 32 bits.
        uint8_t* dst_base =
            td.slot >= 0
                ? reinterpret_cast<uint8_t*>(p.partial + static_cast<long long>(td.slot) * ROWS * (D + 2))
                : reinterpret_cast<uint8_t*>(p.out + static_cast<long long>(td.b) * p.R * p.ldo);
        const long long dst_row =
            td.slot >= 0 ? static_cast<long long>(r) * (D * 4)
                         : (row.i * p.ldo + static_cast<long long>(row.hq) * D) * 2;
        const uint32_t mine = live ? static_cast<uint32_t>(dst_row >> 4) : 0xffffffffu;
        uint32_t to[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) to[k] = __shfl_sync(0xffffffffu, mine, k * 4 + (lane >> 3));
        uint8_t* stage = smem + S::kOffStage + vw * 4096;
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
                    for (int j = max(j0, td.start); j <= min(j1, last_key); ++j) {
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
                if (to[k] != 0xffffffffu)
                    *reinterpret_cast<uint4*>(dst_base + (static_cast<long long>(to[k]) << 4) +
                                              (c / width) * 128 + (lane & 7) * 16) =
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
        return true;
    };

    if (n_units > 0 && (warp == S::kLoadK || warp == S::kLoadV)) {
        // -------------------------------------------------------- producers
        const bool keys = warp == S::kLoadK;
        constexpr int ESZ = S::kES, BOXB = S::kBoxB, KB = S::kKBlks, VB = S::kVBlks;
        uint64_t* full = keys ? b_k : b_v;
        uint64_t* empty = keys ? b_ke : b_ve;
        const int ring = keys ? NK : NV;
        AttnWalk<TK> w;
        w.begin(p, span, cap, lane);
        int n = 0, st = 0, round = 0;  // pieces loaded; the next one's place
        bool ok = true;
        // waits for the place and announces the bytes that come
        auto place = [&](uint32_t bytes) {
            ok = round == 0 || warp_wait(&empty[st], round - 1);
            if (ok && lane == 0) mbar_arrive_expect_tx(&full[st], bytes);
            __syncwarp();
            return ok;
        };
        for (int u = 0; u < n_units; ++u) {
            if (lane == 0) {
                const AttnUnit d = w.unit(p);
                (keys ? s_unit : s_vunit)[u % kUnitRing] = d;
                if (keys && (d.flags & kUnitFirst)) {
                    s_part[d.seg & 7] = d;
                    mbar_arrive(&b_part[d.seg & 7]);  // its queries may be read
                }
                if (keys && u == n_units - 1) {
                    s_parts = d.seg + 1;
                    mbar_arrive(&b_part[(d.seg + 1) & 7]);
                }
            }
            const AttnTile t = w.tile(p);
            if (u + 1 < n_units) w.next(p, lane);
#pragma unroll 1
            for (int i = 0; i < (keys ? KP : VP) && ok; ++i) {
                const int from = keys ? 0 : i * S::kVKeys, blk = keys ? i * KB : 0;
                if (!place(keys ? t.template bytes<TK, KB, BOXB>(0, lane)
                                : t.template bytes<S::kVKeys, VB, BOXB>(from, lane)))
                    break;
                if (keys)
                    t.template load<TK, KB, VB, BOXB, ESZ>(p, &maps.k, sm + S::kOffK + st * S::kKPiece,
                                                           &full[st], from, blk, lane);
                else
                    t.template load<S::kVKeys, VB, VB, BOXB, ESZ>(
                        p, &maps.v, sm + S::kOffV + st * S::kVLoad, &full[st], from, blk, lane);
                ++n;
                if (++st == ring) st = 0, ++round;
            }
            if (!ok) break;
        }
        if (!ok)  // copies in flight land before the block ends
            for (int k = n > ring ? n - ring : 0; k < n; ++k)
                mbar_wait_bounded(&full[k % ring], (k / ring) & 1, p.wait_ns, nullptr);
    } else if (n_units > 0 && warp >= kTcQ && warp < kTcPass) {
        // ------------------------------------------- queries in, finished rows out
        // The walk over the parts is held back by the warps whose queries the products wait
        // for, all four at head size 256, else those with rows: one that is not waited
        // for could fall two phases of b_part behind, so it does not walk.
        const int vw = warp - kTcQ;
        int asked = -1;  // the last part whose queries were asked for
        for (int k = 0; S::kQSmem || vw < row_warps; ++k) {
            if (!warp_wait(&b_part[k & 7], k >> 3)) break;
            const bool more = k < s_parts;
            if (more) {
                const AttnUnit d = s_part[k & 7];
                if (!queries(d, vw)) break;
                asked = k;
            }
            if (k > 0 && vw < row_warps && !finish(k - 1, vw)) break;
            if (!more) break;
        }
        if (S::kQSmem && !F8 && vw == 0 && asked >= 0)  // a load in flight lands before the end
            mbar_wait_bounded(&b_q[0], asked & 1, p.wait_ns, nullptr);
    } else if (n_units > 0 && warp >= kTcPass) {
        // ---------------------------------------------------- V pieces passed on
        const int at = tid - kTcPass * 32;
        constexpr int CH = D * S::kES / 16;
        for (int pc = F8 ? warp - kTcPass : 0; pc < n_units * VP; pc += F8 ? S::kPass : 1) {
            const int u = pc / VP, st = pc % NV;
            if (!warp_wait(&b_v[st], pc / NV)) break;
            const AttnUnit d = s_vunit[u % kUnitRing];
            // Values that no row sees become zeros; infinities and NaN of values that only
            // some rows see too (0 times them must not reach the other rows): the end of
            // the part gives them to the rows that see them.
            const bool edge = d.flags & kUnitEdge;
            const int key0 = d.start + (pc % VP) * S::kVKeys;
            uint8_t* src = smem + S::kOffV + st * S::kVLoad;
            bool odd = false;
            if (!F8) {
                if (edge) {
#pragma unroll 1
                    for (int c = at; c < S::kVKeys * CH; c += S::kPass * 32) {
                        const int row = c / CH, j = key0 + row;
                        if (key_all(j, d.len, d.p0, p.window, p.sinks)) continue;
                        uint4* q = reinterpret_cast<uint4*>(src + S::v_at(row, c % CH));
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
                if (lane == 0) mbar_arrive(&b_clean[pc & 7]);
                continue;
            }
            if (pc >= NF && !warp_wait(&b_fe[pc % NF], pc / NF - 1)) break;
            uint8_t* dst = smem + S::kOffF + pc % NF * S::kVPiece;
            auto write = [&](const uint32_t* w, uint8_t* lo, uint8_t* hi) {  // 16 dimensions
                uint32_t f[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[2 * e] = e4m3x2_f16x2(w[e]);
                    f[2 * e + 1] = e4m3x2_f16x2(w[e] >> 16);
                }
                *reinterpret_cast<uint4*>(lo) = make_uint4(f[0], f[1], f[2], f[3]);
                *reinterpret_cast<uint4*>(hi) = make_uint4(f[4], f[5], f[6], f[7]);
            };
            if (edge) {
#pragma unroll 1
                for (int c = lane; c < S::kVKeys * CH; c += 32) {
                    const int row = c / CH, ch = c % CH, j = key0 + row;
                    const uint4 v = *reinterpret_cast<const uint4*>(src + S::v_at(row, ch));
                    uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    if (!key_some(j, d.len, d.p0, p.window, p.sinks)) {
                        w[0] = w[1] = w[2] = w[3] = 0u;
                    } else if (!key_all(j, d.len, d.p0, p.window, p.sinks)) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll 1
                            for (int q = 0; q < 32; q += 8)
                                if (((w[e] >> q) & 0x7Fu) == 0x7Fu) {
                                    w[e] &= ~(0xFFu << q);
                                    odd = true;
                                }
                    }
                    write(w, dst + S::template at<128>(S::kVBlk, row, 2 * ch),
                          dst + S::template at<128>(S::kVBlk, row, 2 * ch + 1));
                }
            } else {
                // Eight neighbouring lanes take four chunks of rows r and r + 5 of a group of
                // eight: loads and stores then fall into different banks.  The offsets within
                // a group are the lane's own, so the loop is loads, conversions and stores.
                constexpr int P = CH / 4;  // passes of a warp over a group of eight rows
                uint32_t from[P], lo[P], hi[P];
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    const int idx = (lane >> 3) + 4 * k;         // 4 chunks of a pair of rows
                    const int ch = idx % P * 4 + (lane & 3);
                    const int row = (idx / P * 2 + (lane & 4 ? 5 : 0)) & 7;
                    from[k] = S::v_at(row, ch);
                    lo[k] = S::template at<128>(S::kVBlk, row, 2 * ch);
                    hi[k] = S::template at<128>(S::kVBlk, row, 2 * ch + 1);
                }
#pragma unroll 1
                for (int g = 0; g < S::kVKeys / 8; ++g) {
                    const uint8_t* sg = src + g * (S::kVBlks * S::kAtom);
                    uint8_t* dg = dst + g * 1024;
                    uint4 v[P];
#pragma unroll
                    for (int k = 0; k < P; ++k) v[k] = *reinterpret_cast<const uint4*>(sg + from[k]);
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
                        write(w, dg + lo[k], dg + hi[k]);
                    }
                }
            }
            if (odd) s_odd[d.seg & 7] = d.seg + 1;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&b_clean[pc & 7]);
                mbar_arrive(&b_ve[st]);
            }
        }
    } else if (n_units > 0 && warp == kTcMma) {
        // ----------------------------------------------- the tensor cores
        if (elect_one()) {
            constexpr uint32_t iS = tc_idesc(!F8, 128, TK, false);  // bf16, or e4m3
            constexpr uint32_t iO = tc_idesc(!F8, 128, D, true);    // bf16, or f16
            const uint64_t qd0 = tc_desc<S::kBoxB>(sm, 16, 8 * S::kBoxB);
            int fl = 0, parts = 0;  // flags of the tiles qk - 1 (low byte), qk - 2, ..
            int qk = 0, kp = 0, pv = 0, vp = 0;  // next tile and piece of either product
            bool p_in = false;  // P of tile pv is there, and O free for it
            uint64_t t0 = 0;
            uint32_t idle = 0;
            while (pv < n_units) {
                // S of tile qk takes the buffer of tile qk - NS, whose P has been read
                if (qk < n_units && qk < pv + NS) {
                    const int pc = qk * KP + kp, st = pc % NK;
                    if (mbar_test(&b_k[st], (pc / NK) & 1)) {
                        const AttnUnit* d = &s_unit[qk % kUnitRing];
                        const int flags = d->flags, seg = d->seg, qs = seg % S::kNQ;
                        if (kp > 0 || !(flags & kUnitFirst) || mbar_test(&b_q[qs], (seg / S::kNQ) & 1)) {
                            tc_fence_after();
                            const uint64_t kd0 = tc_desc<S::kBoxB>(sm + S::kOffK + st * S::kKPiece, 16,
                                                                   S::kKBlks * S::kAtom);
                            const uint32_t dS = tmem + S::kColS + qk % NS * TK;
                            constexpr int KS = S::kKBlks * S::kSteps;  // k steps of the piece
#pragma unroll
                            for (int t = 0; t < S::kTerms; ++t)
#pragma unroll
                                for (int ks = 0; ks < KS; ++ks) {
                                    const uint64_t kd =
                                        kd0 + (((ks / S::kSteps) * S::kAtom + (ks % S::kSteps) * 32) >> 4);
                                    const int kq = t * (S::kQRow / 32) + kp * KS + ks;  // k step of Q
                                    const bool add = t > 0 || kp > 0 || ks > 0;
                                    if (S::kQSmem)
                                        tc_mma_ss<F8>(
                                            dS,
                                            qd0 + (((kq / S::kSteps) * S::kQBlk + (kq % S::kSteps) * 32) >> 4),
                                            kd, iS, add);
                                    else
                                        tc_mma_ts<F8>(dS, tmem + S::kColQ + qs * (D / 2) + kq * 8, kd, iS, add);
                                }
                            tc_commit(&b_ke[st]);
                            if (++kp == KP) {
                                tc_commit(&b_s[qk % NS]);
                                if (flags & kUnitLast) tc_commit(&b_qe[qs]);
                                fl = (fl << 8) | flags;
                                kp = 0;
                                ++qk;
                            }
                            t0 = 0;
                            continue;
                        }
                    }
                }
                if (pv < qk) {
                    const bool first = (fl >> (8 * (qk - 1 - pv))) & kUnitFirst;
                    p_in = p_in || (mbar_test(&b_p[pv % NS], (pv / NS) & 1) &&
                                    (!first || parts == 0 || mbar_test(&b_o, (parts - 1) & 1)));
                    bool went = false;
                    while (p_in && vp < VP) {
                        const int pc = pv * VP + vp;
                        if (!mbar_test(&b_clean[pc & 7], (pc >> 3) & 1)) break;
                        tc_fence_after();
                        const uint64_t vd =
                            F8 ? tc_desc<128>(sm + S::kOffF + pc % NF * S::kVPiece, S::kVBlk, 1024)
                               : tc_desc<128>(sm + S::kOffV + pc % NV * S::kVLoad, S::kAtom,
                                              S::kVBlks * S::kAtom);
#pragma unroll
                        for (int ks = 0; ks < S::kVKeys / 16; ++ks)
                            tc_mma_ts<false>(tmem + S::kColO,
                                             tmem + S::kColS + pv % NS * TK + (vp * (S::kVKeys / 16) + ks) * 8,
                                             vd + ((ks * (F8 ? 2048 : 2 * S::kVBlks * S::kAtom)) >> 4), iO, !(first && vp == 0 && ks == 0));
                        tc_commit(F8 ? &b_fe[pc % NF] : &b_ve[pc % NV]);
                        ++vp;
                        went = true;
                    }
                    if (vp == VP) {
                        tc_commit(&b_pv[pv % NS]);
                        parts += first;
                        vp = 0;
                        p_in = false;
                        ++pv;
                    }
                    if (went) {
                        t0 = 0;
                        continue;
                    }
                }
                if (++idle & 63) continue;
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
    } else if (n_units > 0 && warp < 4 * H && (warp & 3) < row_warps) {
        // ---------------------------------------------------------- softmax
        const int half = warp >> 2, rw = warp & 3;
        const int r = rw * 32 + lane;  // row of the block = lane of tensor memory
        const uint32_t lanes = static_cast<uint32_t>(rw * 32) << 16;
        const uint32_t tO = tmem + lanes + S::kColO;
        float m = -INFINITY, l = 0.f, c2 = 1.f;
        int pr = -1, seg_start = 0;
        AttnRow row{};
        for (int u = 0; u < n_units; ++u) {
            if (!warp_wait(&b_s[u % NS], u / NS)) break;
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
                    if (p.k_scale) c2 *= fabsf(__ldg(p.k_scale + h));
                    c2 *= __uint_as_float(
                        static_cast<uint32_t>(127 - s_rs[F8 ? td.seg & 7 : 0][F8 ? min(r, ROWS - 1) : 0]) << 23);
                    if (c2 < kMinFactor) c2 = kMinFactor;  // (NaN stays)
                }
                l = 0.f;
            }
            const uint32_t tS = tmem + lanes + S::kColS + u % NS * TK;
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
            // A whole row is walked 32 columns at a time, twice, by rolled loops: the roles
            // share the instruction caches, and unrolled over 128 columns this one alone
            // overflowed them (a fifth of all warp stalls waited for instructions).  Half a
            // row is read once: the other half writes P over its scores.
            constexpr int CW = H > 1 ? TK / H : 32;
            uint32_t x[CW];
            float mx = -INFINITY;
            auto columns = [&](int c) {
                if constexpr (H > 1) tmem_ld64(x, tS + c);
                else tmem_ld32(x, tS + c);
                if (edge) {
#pragma unroll
                    for (int k = 0; k < CW; k += 32) mask(x + k, c + k);
                }
            };
            const int c0 = H > 1 ? half * CW : 0, c1 = H > 1 ? c0 + CW : TK;
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
                if (!warp_wait(&b_x[u & 1][(half ^ 1) * 2 + rw], u >> 1)) break;
                tc_fence_after();
                mx = fmaxf(mx, s_mx[u & 1][half ^ 1][r]);
            }
            bool grow = false;
            float corr = 1.f;
            if (first) {
                m = mx;
            } else if (row.live && (mx - m) * c2 > kLazy) {  // (the other rows hold anything)
                // (m = -infinity: O and l are zeros still)
                if (m != -INFINITY) {
                    corr = ex2((m - mx) * c2);
                    grow = true;
                }
                l *= corr;
                m = mx;
            }
            if (__any_sync(0xffffffffu, grow)) {
                if (!warp_wait(&b_pv[(u - 1) % NS], (u - 1) / NS)) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = half * (D / H); c < (half + 1) * (D / H); c += 32) {
                    uint32_t y[32];
                    tmem_ld32(y, tO + c);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        y[k] = __float_as_uint(__uint_as_float(y[k]) * corr);
                    tmem_st32(tO + c, y);
                }
            }
            const float mc = m == -INFINITY ? 0.f : m * c2 - (F8 ? kTailBitsTc : 0.f);
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
                    y[k / 2] = pack2<F8>(a, b);
                }
                if constexpr (H > 1) tmem_st32(tS + c / 2, y);
                else tmem_st16(tS + c / 2, y);
            }
            l += s0 + s1;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b_p[u % NS]);
            if (!(td.flags & kUnitLast)) continue;

            // ---- end of the part: its rows are written by the query warps
            if (r < ROWS) s_ml[td.seg & 1][half][r] = make_float2(m == -INFINITY ? -INFINITY : mc, l);
            if (tid == 0) {
                AttnUnit d = td;
                d.start = seg_start;
                s_end[td.seg & 1] = d;
                s_end_u[td.seg & 1] = u;
                s_end_start[td.seg & 1] = td.start;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&b_ml[td.seg & 1]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kTcMma) {
        tc_fence_after();
        tmem_dealloc<512>(tmem);
    }
}

#endif  // __CUDACC__
}  // namespace vw4
