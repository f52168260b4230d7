// attn4.cuh -- attention of the verify rows over a paged cache in 4 bits (nvfp4), as a
// template over the head size and the number of query rows, instantiated per head size in
// attn4_d*.cu.  The work schedule, the page loads and the join of split items are those of
// the other cache types (attn.cuh).
//
// Mathematics.  S = Q K^T, P = exp(S - max), O = P V with a running maximum and sum over
// tiles of 64 to 256 keys, all transposed: keys, then dimensions are the rows of the matrix
// instructions and the query rows their columns, eight to an instruction, so that the
// converted cache values are the operand that is made once and the query rows cost little
// where they are few.  K^T and V become f16 in registers, exactly: e2m1 times its block's
// e4m3 scale has six significant bits.
//
// A tile.  Each warp takes 16 to 64 keys for S = K Q^T (32 dimensions of 8 keys are a register
// of codes a lane), forms P against the block's common reference, and leaves it in shared
// memory; beside it, the warps leave V's scales as f16, token by token.  After the barrier
// each warp takes a slice of V's dimensions for O = V^T P^T, so nothing is converted twice
// however many query rows there are, and S of the next tile runs in the same phase: one
// barrier a tile.
//
// What bounds it: the chain of a tile, which eight computing warps an SM hide in part: with few
// rows no unit is a limit (the ALU, whose work is mostly conversions, a cvt for two codes and a
// multiply by the scale, is 50 % busy, the issue slots 53 %, HBM 53 %); from 16 rows on the
// products are in the chain too.  32 sequences of up to 32768 tokens, 8 key heads of size 128,
// four rows each: 104 us of 424 MB, 62.5 at the copy rate; 24 rows of size 256 over 64 windows of
// 1024: 53 us.  Without conversions and products the loads alone take 78 and 39.
//
// The reference that the weights use is the running maximum, followed lazily: only where a
// score exceeds it by 2^6 do the warps meet for the true maximum, rescale and form P again
// (the first tile of an item; rarely later).  Weights are at most 2^15 in f16, and reach
// down to 2^-33 of the largest (f16 ends at 2^-24).  What a weight's exponent takes from its score
// is the reference less 9, rounded up once; rescaling and the join take the same number, so that
// its rounding is a common factor of a row and no weight leaves f16, however large the scores.
#pragma once
#include "attn.cuh"

namespace vw4 {

constexpr float kTail4 = 9.f;     // weights carry 2^9
constexpr float kLazy4 = 6.f;     // (log2) of the reference

// Keys of a tile: four warps and about 18 KB of K and V put two blocks on an SM (three with 9 KB,
// at head size 64).  One n-tile of query rows, and two at head size 64, leave the registers for
// twice as many: fewer meetings, rings and edges for the same bytes (32 sequences of up to 32768
// tokens, one row of four heads: head size 64 71.5 us instead of 118.6, 128 105 instead of 109
// with three blocks, 256 98 instead of 108; 16 rows at head size 64 85 instead of 105).  16 rows of
// larger heads are faster so over long sequences (128: 126 instead of 138) and slower over short
// ones and windows (30 us instead of 38 there), for want of room for the rings.  One n-tile keeps
// the small tiles too, for tables that do not hold a large one for every SM (one sequence of 517
// tokens, 4 key heads of size 256, one row of six heads: 9.5 us instead of 10.2).  The lengths are
// the device's: the rule, and the grid, go by the table, and a wide one costs a short sequence
// what the grid costs: 517 tokens under tables of 4608 (small tiles), 5000 (large) and 131072
// tokens 10.4, 10.5 and 11.6 us, with 8 heads of size 128 10.5, 11.4 and 12.0 (9.6 under their own).
__host__ __device__ constexpr int attn4_tk(int D, bool large) {
    return (D == 256 ? 64 : 128) * (large ? 2 : 1);
}
// Places of the ring of K tiles: what shared memory leaves.
__host__ __device__ constexpr int attn4_places(int D, int nt, bool large) {
    return large      ? (D > 64 ? 2 : (nt == 1 ? 3 : 4))
           : D == 64  ? 6
           : nt == 1  ? 3
           : D == 128 ? (nt == 4 ? 3 : 4)
                      : (nt >= 3 ? 3 : 4);
}

#ifdef __CUDACC__
// What the exponents take from scores whose largest is m under the factor c2 (-infinity: none).
__device__ __forceinline__ float attn4_ref(float m, float c2) {
    return m == -INFINITY ? -INFINITY : __fmaf_ru(m, c2, -kTail4);
}

template <int D, int NT, bool LARGE>
struct Attn4Shape {
    static constexpr int kWarps = 4;
    static constexpr int kThreads = (kWarps + 2) * 32;
    static constexpr int kTK = attn4_tk(D, LARGE);
    static constexpr int kKM = kTK / kWarps / 16;     // 16-key row tiles of a warp
    static constexpr int kRows = 8 * NT;
    static constexpr int kKB = D / 2;                 // bytes of a key's codes
    static constexpr int kNB = D / 16;                // and of its scales
    static constexpr int kTile = kTK * kKB;
    static constexpr int kSTile = kTK * kNB;
    static constexpr int kStage = kTile + kSTile;     // of K or V: codes, scales
    static constexpr int kSlices = D / 32;            // slices of 32 of V's dimensions
    static constexpr int kOwn = kSlices > kWarps ? kSlices / kWarps : 1;    // of a warp
    static constexpr int kParts = kWarps > kSlices ? kWarps / kSlices : 1;  // parts of V's keys
    static constexpr int kQ = kRows * D * 2;
    static constexpr int kQBlk = kRows * 128;
    static constexpr int kP = NT * kTK * 16;          // weights: f16 [n-tile][key][8]
    static constexpr int kVRow = (kTK + 16) * 2;      // V's scales: f16 [block][v_at(token)]
    static constexpr int kVS = kNB * kVRow;
    static constexpr int kX = (kParts - 1) * kSlices * 1024;  // an n-tile's outputs of the other parts
    static constexpr int kMinBlocks = NT == 1 && (D == 64 || !LARGE) ? 3 : 2;
    // V of a tile is read a phase after its K: one place more, if it fits
    static constexpr int kNK = attn4_places(D, NT, LARGE), kNV = kNK + (NT == 1 && (D > 64 || LARGE) ? 0 : 1);
    static constexpr int kOffVal = kNK * kStage;
    static constexpr int kOffQ = (kOffVal + kNV * kStage + 1023) / 1024 * 1024;
    static constexpr int kOffP = kOffQ + 2 * kQ;
    static constexpr int kOffV = kOffP + 2 * kP;
    static constexpr int kOffX = kOffV + 2 * kVS;
    static constexpr int kOffML = kOffX + kX;          // float [2][warps][rows]: maxima, sums
    static constexpr int kOffRow = kOffML + 2 * kWarps * kRows * 4;  // [6][rows], see below
    static constexpr int kSmem = kOffRow + 6 * kRows * 4 + 1024;
    static_assert(kStage % (8 * kKB) == 0 && kQ % 1024 == 0 && kVS % 16 == 0, "alignment");
    static_assert(kSmem <= 225 * 1024, "shared memory");
    static_assert(kTK % (kParts * 32) == 0, "V's keys in steps of 32");
    __device__ static __forceinline__ uint32_t at(int key, int chunk) {  // 16 bytes of a key's codes
        const int x = kKB == 128 ? key & 7 : (kKB == 64 ? (key >> 1) & 3 : (key >> 2) & 1);
        return static_cast<uint32_t>(key * kKB + ((chunk ^ x) << 4));
    }
    __device__ static __forceinline__ uint32_t q_at(int row, int chunk) {  // 16 bytes of a query
        return static_cast<uint32_t>((chunk >> 3) * kQBlk + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
    }
    // where a token's scale stands: the four pairs of tokens that a lane of O's product
    // multiplies in a step of 32 keys are 16 bytes
    __device__ static __forceinline__ int v_at(int token) {
        return (token & ~31) | ((token >> 1) & 3) << 3 | ((token >> 3) & 3) << 1 | (token & 1);
    }
};

// Matrix loads that keep their order to the barriers alone, and products that keep none, so
// that they are free to overlap.
__device__ __forceinline__ void ldsm4_free(uint32_t* r, uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void ldsm4t_free(uint32_t* r, uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// by the low or the high half of s (a broadcast that costs no instruction)
template <bool HIGH>
__device__ __forceinline__ uint32_t mul_f16x2_half(uint32_t a, uint32_t s) {
    const __half2 h = *reinterpret_cast<const __half2*>(&s);
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), HIGH ? __high2half2(h) : __low2half2(h));
    return *reinterpret_cast<const uint32_t*>(&r);
}

template <int D, int NT, bool LARGE>
__global__ void __launch_bounds__(Attn4Shape<D, NT, LARGE>::kThreads, Attn4Shape<D, NT, LARGE>::kMinBlocks)
    attn4_kernel(const AttnParams p, const Kv4Blocks kb, const __grid_constant__ AttnMaps maps) {
    using S = Attn4Shape<D, NT, LARGE>;
    constexpr int TK = S::kTK, NK = S::kNK, NV = S::kNV, NB = S::kNB, KM = S::kKM;
    constexpr bool kValuesFirst = NT <= 3;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ __align__(8) uint64_t b_k[NK], b_ke[NK], b_v[NV], b_ve[NV], b_qe[2];
    __shared__ AttnUnit s_unit[kUnitRing];  // a part's first unit, by its number
    __shared__ int4 s_tile[kUnitRing];      // a unit's first key, flags, partial slot
    __shared__ volatile int s_abort;
    __shared__ float2 s_scale[2];    // a part's scales of its head of K and V, by seg & 1
    const int tid = threadIdx.x, lane = tid & 31, wk = tid >> 5;
    const uint32_t sm = smem_u32(smem);
    float* s_m = reinterpret_cast<float*>(smem + S::kOffML);
    float* s_l = s_m + S::kWarps * S::kRows;
    float* s_c2 = reinterpret_cast<float*>(smem + S::kOffRow);      // log2 of a score of a query row
    int* s_pos = reinterpret_cast<int*>(s_c2 + S::kRows);           // its position (dead: -1)
    int* s_out = s_pos + S::kRows;                                  // verify index << 16 | head (dead: -1)
    uint32_t* s_nan = reinterpret_cast<uint32_t*>(s_out + S::kRows);  // its blocks that a NaN reached
    float* s_ref = reinterpret_cast<float*>(s_nan + S::kRows);      // [2] its attn4_ref, in turn

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == S::kWarps * 32) {
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
        tma_prefetch_desc(&maps.q);
    }
    if (tid == 0) {
        for (int k = 0; k < NK; ++k) {
            mbar_init(&b_k[k], 1);
            mbar_init(&b_ke[k], 1);
        }
        for (int k = 0; k < NV; ++k) {
            mbar_init(&b_v[k], 1);
            mbar_init(&b_ve[k], 1);
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
        // ------------------------------------------------------- a loading warp for K, one for V
        const bool keys = wk == S::kWarps;
        const CUtensorMap* map = keys ? &maps.k : &maps.v;
        const uint8_t* blocks = keys ? kb.k : kb.v;
        uint64_t* full = keys ? b_k : b_v;
        uint64_t* empty = keys ? b_ke : b_ve;
        const int places = keys ? NK : NV, base = keys ? 0 : S::kOffVal;
        const uint64_t policy = policy_evict_normal();
        const uint32_t box = static_cast<uint32_t>(p.box_rows * NB);  // bytes of a box's scales
        AttnWalk<TK> w;
        w.begin(p, span, cap, lane);
        int u = 0, st = 0, round = 0;
        for (; u < n_units; ++u) {
            const AttnUnit d = w.unit(p);
            const AttnTile t = w.tile(p);
            const bool q = keys && (d.flags & kUnitFirst);
            float ks = 1.f, vs = 1.f;
            if (q) {
                if (p.k_scale) ks = __ldg(p.k_scale + t.h);
                if (p.v_scale) vs = __ldg(p.v_scale + t.h);
            }
            if (u + 1 < n_units) w.next(p, lane);
            const bool there = t.page >= 0 && t.page < p.num_pages;
            const uint32_t bytes = t.template bytes<TK, 1, S::kKB>(0, lane) +
                                   __popc(__ballot_sync(0xffffffffu, there)) * box;
            const uint8_t* from = blocks;
            if (there)
                from += t.page * kb.page_stride + t.h * kb.head_stride +
                        ((t.start + lane * p.box_rows) & (p.page_size - 1)) * NB;
            const int off = base + st * S::kStage;
            uint8_t* sdst = smem + off + S::kTile + lane * box;
            if (round > 0 && !wait(&empty[st], round - 1)) break;
            if (q && d.seg >= 2 && !wait(&b_qe[d.seg & 1], (d.seg >> 1) - 1)) break;
            if (t.page == p.num_pages) {  // no such page: zeros
                for (uint32_t c = 0; c < box; c += 16)
                    *reinterpret_cast<uint4*>(sdst + c) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
            }
            __syncwarp();
            if (lane == 0) {
                if (keys) s_tile[u % kUnitRing] = make_int4(d.start, d.flags, d.slot, 0);
                if (q) {
                    s_unit[d.seg % kUnitRing] = d;
                    s_scale[d.seg & 1] = make_float2(ks, vs);
                }
                mbar_arrive_expect_tx(&full[st], bytes + (q ? attn_q_bytes(p, D) : 0u));
                if (q)
                    attn_load_q<D>(p, &maps.q, sm + S::kOffQ + (d.seg & 1) * S::kQ, S::kQBlk, d, &full[st]);
            }
            __syncwarp();
            t.template load<TK, 1, 1, S::kKB, 1>(p, map, sm + off, &full[st], 0, 0, lane);
            if (there) bulk_load(sdst, from, box, &full[st], policy);
            __syncwarp();
            if (++st == places) st = 0, ++round;
        }
        // copies in flight land before the block ends
        if (u < n_units) {
            for (int k = u > places ? u - places : 0; k < u; ++k)
                mbar_wait_bounded(&full[k % places], (k / places) & 1, p.wait_ns, nullptr);
        }
        return;
    }

    // ---- the computing warps.  Every path between two meetings has the same number of them in
    // all warps: a wait that ran out makes a warp skip its work, and the next meeting ends
    // the block's.
    bool dead = false;
    auto meet = [&](bool flag) {  // the threads of the computing warps; any of the flags
        uint32_t r;
        asm volatile(
            "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\t"
            "barrier.cta.red.or.pred b, 1, %2, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
            : "=r"(r) : "r"(static_cast<uint32_t>(flag)), "n"(S::kWarps * 32) : "memory");
        return r != 0;
    };
    // rows: dimensions 4 u + 2 i, + 1 of the slice; columns: query rows
    float o[S::kOwn][2][NT][4];
    float l[NT][2];
    int turn = 0;  // of s_ref
    const int t4 = lane & 3, u8 = lane >> 2, lm = lane >> 3, lr = lane & 7;
    const int key0 = wk * 16 * KM;                     // of the warp's keys
    const int slice0 = wk % S::kSlices * S::kOwn, part = wk / S::kSlices;
    const int inv_gb = 65536 / p.gb + 1;               // r / gb = r * inv_gb >> 16 for r < 32
    // Matrix loads: the lane's part of the address, in which a further 32-dimension chunk of K
    // (even), slice of V or half of 64 query dimensions is an exclusive or.
    const uint32_t k_lane = S::at(key0 + lr + (lm & 1) * 8, lm >> 1);
    const uint32_t v_lane = S::at(part * (TK / S::kParts) + lr + 8 * lm, slice0);
    const uint32_t q_lane = S::q_at(lr, lm);
    const uint32_t p_lane = (part * (TK / S::kParts) + lr + 8 * lm) * 16;
    const uint32_t sc_lane = S::kOffV + t4 * 16 + (slice0 * 2 + (lane >> 4)) * S::kVRow +
                             part * (TK / S::kParts) * 2;
    int kst = 0, vst = 0, vlast = 0;                   // places of the unit's K and V, of the last V
    int kround = 0, vround = 0;

    auto row2 = [&](const float* a, int n, float* v) {  // of the lane's two query rows
        const float2 f = *reinterpret_cast<const float2*>(a + n * 8 + t4 * 2);
        v[0] = f.x;
        v[1] = f.y;
    };

    // O += V^T P^T of unit u, whose V is in place st
    auto values = [&](int u, int st) {
        const uint32_t vS = sm + S::kOffVal + st * S::kStage + v_lane;
        const uint32_t pS = sm + S::kOffP + (u & 1) * S::kP + p_lane;
        const uint8_t* sc = smem + (u & 1) * S::kVS + sc_lane;
#pragma unroll
        for (int k = 0; k < TK / S::kParts; k += 32) {
            uint32_t x[S::kOwn][4], b[NT][4];
            uint4 sv[S::kOwn];
#pragma unroll
            for (int q = 0; q < S::kOwn; ++q) {
                ldsm4t_free(x[q], (vS ^ (q << 4)) + k * S::kKB);
                sv[q] = *reinterpret_cast<const uint4*>(sc + q * 2 * S::kVRow + k * 2);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) ldsm4t_free(b[n], pS + n * (TK * 16) + k * 16);
#pragma unroll
            for (int q = 0; q < S::kOwn; ++q) {
                const uint32_t s[4] = {sv[q].x, sv[q].y, sv[q].z, sv[q].w};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // a register: two tokens x four dimensions; to pairs of tokens, scaled
                    uint32_t e[2][4];
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        uint32_t w[4];
                        e2m1x8_f16(x[q][2 * h + m], w);
                        e[m][0] = mul_f16x2(__byte_perm(w[0], w[2], 0x5410), s[2 * h + m]);
                        e[m][1] = mul_f16x2(__byte_perm(w[0], w[2], 0x7632), s[2 * h + m]);
                        e[m][2] = mul_f16x2(__byte_perm(w[1], w[3], 0x5410), s[2 * h + m]);
                        e[m][3] = mul_f16x2(__byte_perm(w[1], w[3], 0x7632), s[2 * h + m]);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma_f16(o[q][i][n], e[0][2 * i], e[0][2 * i + 1], e[1][2 * i], e[1][2 * i + 1],
                                    b[n][2 * h], b[n][2 * h + 1]);
                }
            }
        }
    };

    for (int u = 0, seg = 0; u < n_units; ++u) {
        // ---- a part of an item: its queries
        dead |= !wait(&b_k[kst], kround);
        const AttnUnit td = s_unit[seg % kUnitRing];
        const int qslot = seg++ & 1;
        const uint32_t qs = sm + S::kOffQ + qslot * S::kQ;
        const int h = td.g / p.row_blocks;
        float ks = 1.f, vs = 1.f;
        if (!dead) {
            ks = s_scale[qslot].x;
            vs = s_scale[qslot].y;
            // bf16 -> f16 under a power of two per row that puts its largest magnitude into
            // [2^14, 2^15), with the sign of the head's scale: exact for every value down to
            // 2^-31 of it.  Within 32 dimensions the order is that of the codes' registers.
            // Up to eight rows at once: a row is a chain of latencies.
            const int rb = td.g - h * p.row_blocks;
            const int bt = rb / p.blocks_g, bg = rb - bt * p.blocks_g;
            uint32_t* rows = reinterpret_cast<uint32_t*>(smem + S::kOffQ + qslot * S::kQ);
            constexpr int kAtOnce = S::kRows / S::kWarps;
            uint32_t v[kAtOnce][D / 64], mx[kAtOnce];
            int pos[kAtOnce], out[kAtOnce];
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
                const int r = wk + q * S::kWarps;
                const int t = (r * inv_gb) >> 16, gq = bg * p.gb + r - t * p.gb, i = bt * p.tb + t;
                const bool live = t < p.tb && i < p.R && gq < p.G;
                pos[q] = live ? td.p0 + i : -1;
                out[q] = live ? i << 16 | (h * p.G + gq) : -1;
                mx[q] = 0u;
#pragma unroll
                for (int k = 0; k < D / 64; ++k) {
                    const int e = lane + 32 * k;  // pair of dimensions 2e, 2e + 1
                    v[q][k] = live ? rows[(S::q_at(r, e >> 2) >> 2) + (e & 3)] : 0u;
                    mx[q] = __vmaxu2(mx[q], v[q][k] & 0x7fff7fffu);
                }
            }
#pragma unroll
            for (int s = 16; s > 0; s >>= 1)
#pragma unroll
                for (int q = 0; q < kAtOnce; ++q)
                    mx[q] = __vmaxu2(mx[q], __shfl_xor_sync(0xffffffffu, mx[q], s));
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
                const int r = wk + q * S::kWarps;
                const int ex = static_cast<int>(max(mx[q] & 0xffffu, mx[q] >> 16) >> 7);
                int sh = ex == 0 || ex == 255 ? 0 : 127 + 14 - ex;
                sh = max(-126, min(126, sh));
                const float up = copysignf(__uint_as_float(static_cast<uint32_t>(127 + sh) << 23), ks);
                if (lane == 0) {
                    float c2 = p.scale * kLog2e * fabsf(ks) *
                               __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
                    if (c2 < kMinFactor) c2 = kMinFactor;  // (NaN stays)
                    s_c2[r] = c2;
                    s_ref[r] = -INFINITY;
                    s_pos[r] = pos[q];
                    s_out[r] = out[q];
                    s_nan[r] = 0u;
                }
#pragma unroll
                for (int k = 0; k < D / 64; ++k) {
                    const int e = lane + 32 * k, s = (e & ~15) | ((e & 3) << 2) | ((e >> 2) & 3);
                    rows[(S::q_at(r, s >> 2) >> 2) + (s & 3)] =
                        pack2<true>(__uint_as_float(v[q][k] << 16) * up,
                                    __uint_as_float(v[q][k] & 0xffff0000u) * up);
                }
            }
            fence_async_smem();  // (a later load will write there)
        }
        if (meet(dead)) return;
        turn = 0;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int q = 0; q < S::kOwn; ++q)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    o[q][i][n][0] = o[q][i][n][1] = o[q][i][n][2] = o[q][i][n][3] = 0.f;
        }
        int4 tile;
        for (const int first = u;; ++u) {
            if (u > first) dead |= !wait(&b_k[kst], kround);
            tile = s_tile[u % kUnitRing];
            const int start = tile.x;
            const bool edge = tile.y & kUnitEdge;
            const uint8_t* keys = smem + kst * S::kStage;
            float s[KM][NT][4];
            float sum[NT][2];
            // weights of an n-tile against a reference, to shared memory
            auto weights = [&](int n, const float* c2, const float* ref) {
                uint8_t* dst = smem + S::kOffP + (u & 1) * S::kP + (key0 + u8) * 16 + t4 * 4 + n * (TK * 16);
                sum[n][0] = sum[n][1] = 0.f;
                const float r[2] = {ref[0] == -INFINITY ? 0.f : -ref[0], ref[1] == -INFINITY ? 0.f : -ref[1]};
#pragma unroll
                for (int m = 0; m < KM; ++m) {
                    float w[4];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        w[k] = ex2(fmaf(s[m][n][k], c2[k], r[k]));
                        w[k + 2] = ex2(fmaf(s[m][n][k + 2], c2[k], r[k]));
                        sum[n][k] += w[k] + w[k + 2];
                    }
                    *reinterpret_cast<uint32_t*>(dst + m * 256) = pack2<true>(w[0], w[1]);
                    *reinterpret_cast<uint32_t*>(dst + m * 256 + 128) = pack2<true>(w[2], w[3]);
                }
            };
            auto largest = [&](int n, int k) {
                float mx = fmaxf(s[0][n][k], s[0][n][k + 2]);
#pragma unroll
                for (int m = 1; m < KM; ++m) mx = fmaxf(mx, fmaxf(s[m][n][k], s[m][n][k + 2]));
                return mx;
            };
            bool grew = false;
            if (!dead) {
                // ---- S = K Q^T of the warp's keys
                const uint32_t kS = sm + kst * S::kStage + k_lane, qS = qs + q_lane;
                uint32_t sk[2 * KM][D / 64];  // scales of two 32-dimension chunks, of keys u8 + 8 k
#pragma unroll
                for (int k = 0; k < 2 * KM; ++k) {
                    const uint8_t* src = keys + S::kTile + (key0 + u8 + 8 * k) * NB;
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
                for (int m = 0; m < KM; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n) s[m][n][0] = s[m][n][1] = s[m][n][2] = s[m][n][3] = 0.f;
#pragma unroll
                for (int c = 0; c < D / 32; c += 2) {
                    uint32_t w[KM][4];
#pragma unroll
                    for (int m = 0; m < KM; ++m)
                        ldsm4_free(w[m], (kS ^ (c << 4)) + m * 16 * S::kKB);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t b[NT][4];
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            ldsm4_free(b[n], (qS ^ (e << 6)) + c / 2 * S::kQBlk + n * 1024);
#pragma unroll
                        for (int m = 0; m < KM; ++m) {
                            uint32_t x[4], y[4];
                            e2m1x8_f16(w[m][2 * e], x);
                            e2m1x8_f16(w[m][2 * e + 1], y);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t sx = sk[2 * m][c / 2], sy = sk[2 * m + 1][c / 2];
                                x[k] = e ? mul_f16x2_half<true>(x[k], sx) : mul_f16x2_half<false>(x[k], sx);
                                y[k] = e ? mul_f16x2_half<true>(y[k], sy) : mul_f16x2_half<false>(y[k], sy);
                            }
#pragma unroll
                            for (int n = 0; n < NT; ++n) mma_f16(s[m][n], x[0], y[0], x[1], y[1], b[n][0], b[n][1]);
#pragma unroll
                            for (int n = 0; n < NT; ++n) mma_f16(s[m][n], x[2], y[2], x[3], y[3], b[n][2], b[n][3]);
                        }
                    }
                }
                // (the products of S are on their way meanwhile, where the registers last for both)
                if (kValuesFirst && u > first) values(u - 1, vlast);
                if (edge) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int pos = s_pos[n * 8 + t4 * 2 + k];
#pragma unroll
                            for (int m = 0; m < KM; ++m) {
                                const int j = start + key0 + 16 * m + u8;
                                if (!key_seen(j, pos, p.window, p.sinks)) s[m][n][k] = -INFINITY;
                                if (!key_seen(j + 8, pos, p.window, p.sinks)) s[m][n][k + 2] = -INFINITY;
                            }
                        }
                }
                // ---- V's scales to f16, token by token: a thread a part of a token's
                dead |= !wait(&b_v[vst], vround);
                if (!dead) {
                    constexpr int ALL = TK * NB / (S::kWarps * 32);  // bytes of a thread
                    constexpr int PER = ALL < NB ? ALL : (NB < 8 ? NB : 8);  // of them one token's
                    static_assert(PER == 2 || PER == 4 || PER == 8, "up to two words");
                    constexpr int W = (PER + 3) / 4;
                    constexpr int TPT = NB / PER;                    // threads of a token
#pragma unroll
                    for (int round = 0; round < ALL / PER; ++round) {
                        const int token = tid / TPT + round * (S::kWarps * 32 / TPT), b0 = tid % TPT * PER;
                        const uint8_t* src = smem + S::kOffVal + vst * S::kStage + S::kTile + token * NB + b0;
                        uint32_t w[W];
                        if (PER == 2) w[0] = *reinterpret_cast<const uint16_t*>(src);
#pragma unroll
                        for (int k = 0; k < PER / 4; ++k) w[k] = reinterpret_cast<const uint32_t*>(src)[k];
                        if (edge) {
                            const int j = start + token;
                            if (!key_some(j, td.len, td.p0, p.window, p.sinks)) {
                                // no row sees it: zeros, whatever the cache holds there
#pragma unroll
                                for (int k = 0; k < W; ++k) w[k] = 0u;
                            } else if (!key_all(j, td.len, td.p0, p.window, p.sinks)) {
                                // NaN scales must not reach rows that do not see the key through a
                                // weight of zero: noted for the others, and taken out
#pragma unroll
                                for (int k = 0; k < PER; ++k) {
                                    if (((w[k / 4] >> (8 * (k & 3))) & 0x7fu) != 0x7fu) continue;
                                    w[k / 4] &= ~(0xffu << (8 * (k & 3)));
#pragma unroll 1
                                    for (int r = 0; r < S::kRows; ++r)
                                        if (s_out[r] >= 0 && key_seen(j, s_pos[r], p.window, p.sinks))
                                            atomicOr(&s_nan[r], 1u << (b0 + k));
                                }
                            }
                        }
                        uint8_t* dst = smem + S::kOffV + (u & 1) * S::kVS + b0 * S::kVRow + S::v_at(token) * 2;
#pragma unroll
                        for (int k = 0; k < PER; k += 2) {
                            const uint32_t f = e4m3x2_f16x2(w[k / 4] >> (8 * (k & 3)));
                            *reinterpret_cast<uint16_t*>(dst + k * S::kVRow) = static_cast<uint16_t>(f);
                            *reinterpret_cast<uint16_t*>(dst + (k + 1) * S::kVRow) =
                                static_cast<uint16_t>(f >> 16);
                        }
                    }
                }
                if (u == first) {
                    grew = true;  // the first maximum
                } else {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float c2[2], ref[2];
                        row2(s_c2, n, c2);
                        row2(s_ref + turn * S::kRows, n, ref);
                        grew |= __fmul_ru(largest(n, 0), c2[0]) > __fadd_rd(ref[0], kTail4 + kLazy4) ||
                                __fmul_ru(largest(n, 1), c2[1]) > __fadd_rd(ref[1], kTail4 + kLazy4);
                        weights(n, c2, ref);
                    }
                    if (!kValuesFirst) values(u - 1, vlast);
                }
            }
            if (meet(grew || dead)) {
                if (meet(dead)) return;
                // ---- the true maximum of the rows, and the weights again
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float c2[2], mx[2];
                    row2(s_c2, n, c2);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        mx[k] = largest(n, k);
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1)
                            mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], x));
                        mx[k] = attn4_ref(mx[k], c2[k]);
                    }
                    if (lane < 4)
                        *reinterpret_cast<float2*>(s_m + wk * S::kRows + n * 8 + t4 * 2) =
                            make_float2(mx[0], mx[1]);
                }
                meet(false);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float c2[2], ref[2], mx[2];
                    row2(s_c2, n, c2);
                    row2(s_ref + turn * S::kRows, n, ref);
                    mx[0] = ref[0];
                    mx[1] = ref[1];
#pragma unroll
                    for (int w = 0; w < S::kWarps; ++w) {
                        float m2[2];
                        row2(s_m + w * S::kRows, n, m2);
                        mx[0] = fmaxf(mx[0], m2[0]);
                        mx[1] = fmaxf(mx[1], m2[1]);
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float f = mx[k] == ref[k] ? 1.f : ex2(ref[k] - mx[k]);
                        l[n][k] *= f;
#pragma unroll
                        for (int q = 0; q < S::kOwn; ++q)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                o[q][i][n][k] *= f;
                                o[q][i][n][k + 2] *= f;
                            }
                    }
                    if (wk == 0 && lane < 4)
                        *reinterpret_cast<float2*>(s_ref + (turn ^ 1) * S::kRows + n * 8 + t4 * 2) =
                            make_float2(mx[0], mx[1]);
                    weights(n, c2, mx);
                }
                turn ^= 1;
                meet(false);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                l[n][0] += sum[n][0];
                l[n][1] += sum[n][1];
            }
            if (tid == 0) {
                mbar_arrive(&b_ke[kst]);
                if (u > first) mbar_arrive(&b_ve[vlast]);
            }
            vlast = vst;
            if (++kst == NK) kst = 0, ++kround;
            if (++vst == NV) vst = 0, ++vround;
            if (tile.y & kUnitLast) break;
        }
        values(u, vlast);
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
        const int slot = tile.z;
        float* po = nullptr;  // partial rows [rows][D], then m [rows], l [rows]
        if (slot >= 0) po = p.partial + static_cast<long long>(slot) * S::kRows * (D + 2);
        float4* xb = reinterpret_cast<float4*>(smem + S::kOffX);
        meet(false);
        if (tid < S::kRows) {  // a row's sum, its factor and the row's own outputs
            const int r = tid, to = s_out[r];
            float L = 0.f;
#pragma unroll
            for (int w = 0; w < S::kWarps; ++w) L += s_l[w * S::kRows + r];
            const float M = s_ref[turn * S::kRows + r];
            s_m[r] = L == 0.f ? 0.f : vs / L;
            if (slot >= 0) {
                po[S::kRows * D + r] = M;
                po[S::kRows * (D + 1) + r] = L;
            } else if (p.lse && to >= 0) {
                p.lse[(static_cast<long long>(td.b) * p.R + (to >> 16)) * p.Hq + (to & 0xffff)] =
                    L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
            }
        }
        meet(false);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float4 v[S::kOwn][2];
#pragma unroll
            for (int q = 0; q < S::kOwn; ++q)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    v[q][k] = make_float4(o[q][0][n][k], o[q][0][n][k + 2], o[q][1][n][k], o[q][1][n][k + 2]);
            if (S::kParts > 1) {
                if (part > 0) {
                    xb[(wk - S::kSlices) * 64 + lane] = v[0][0];
                    xb[(wk - S::kSlices) * 64 + 32 + lane] = v[0][1];
                }
                meet(false);
            }
            if (part == 0) {
                const int r = n * 8 + t4 * 2;
                const int2 to2 = *reinterpret_cast<const int2*>(s_out + r);
                const uint2 nan2 = *reinterpret_cast<const uint2*>(s_nan + r);
                float f2[2];
                row2(s_m, n, f2);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
#pragma unroll
                    for (int q = 1; q < S::kParts; ++q) {
                        const float4 a = xb[(slice0 + (q - 1) * S::kSlices) * 64 + 32 * k + lane];
                        v[0][k].x += a.x;
                        v[0][k].y += a.y;
                        v[0][k].z += a.z;
                        v[0][k].w += a.w;
                    }
                    const int to = k ? to2.y : to2.x;
                    const uint32_t nan = k ? nan2.y : nan2.x;
                    const float f = f2[k];
                    __nv_bfloat16* out = p.out + (static_cast<long long>(td.b) * p.R + (to >> 16)) * p.ldo +
                                         static_cast<long long>(to & 0xffff) * D;
#pragma unroll
                    for (int q = 0; q < S::kOwn; ++q) {
                        const int col = (slice0 + q) * 32 + u8 * 4;
                        if ((nan >> (col / 16)) & 1u) v[q][k] = make_float4(NAN, NAN, NAN, NAN);
                        if (to < 0) {
                        } else if (slot >= 0) {
                            *reinterpret_cast<float4*>(po + (r + k) * D + col) = v[q][k];
                        } else {
                            *reinterpret_cast<uint2*>(out + col) =
                                make_uint2(pack2<false>(v[q][k].x * f, v[q][k].y * f),
                                           pack2<false>(v[q][k].z * f, v[q][k].w * f));
                        }
                    }
                }
            }
            if (S::kParts > 1 || n == NT - 1) meet(false);
        }
        if (tid == 0) {
            mbar_arrive(&b_ve[vlast]);
            mbar_arrive(&b_qe[qslot]);
        }
    }
}

template <int D, int NT, bool LARGE>
cudaError_t attn4_launch(const AttnParams& p, const Kv4Blocks& kb, const AttnMaps& maps, int* grid,
                         int sms, cudaStream_t s) {
    using S = Attn4Shape<D, NT, LARGE>;
    static std::atomic<unsigned long long> once;
    static std::atomic<int> occ;
    auto* kernel = attn4_kernel<D, NT, LARGE>;
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
                           bool large, int* grid, int sms, cudaStream_t s) {
    switch (nt) {
        case 1:
            return large ? attn4_launch<D, 1, true>(p, kb, maps, grid, sms, s)
                         : attn4_launch<D, 1, false>(p, kb, maps, grid, sms, s);
        case 2: return attn4_launch<D, 2, D == 64>(p, kb, maps, grid, sms, s);
        case 3: return attn4_launch<D, 3, false>(p, kb, maps, grid, sms, s);
        case 4: return attn4_launch<D, 4, false>(p, kb, maps, grid, sms, s);
    }
    return cudaErrorInvalidValue;
}
#endif  // __CUDACC__

}  // namespace vw4
