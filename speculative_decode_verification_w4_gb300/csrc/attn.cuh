// attn.cuh -- attention of the verify rows over a paged key-value cache: the
// work schedule, the page loads, and the kernel for up to 16 query rows of a
// key head (plain decoding and narrow verify batches) as a template over the
// head size and the cache type, instantiated per head size in attn_d*.cu.
// More rows: attn_tc.cuh.
//
// Mathematics.  Sequence b's R new tokens sit at positions p_i = len - R + i.
// The R * G query rows (G query heads to a key head) that read the same keys
// are one item's matrix: S = Q K^T, P = exp(S - max), O = P V, with a running
// maximum and sum over key tiles, so that every key and value is read once.
//
// Work split.  The units are (sequence, key head, block of query rows, tile of
// TK keys), in that order; CTA i of G takes units [i T / G, (i + 1) T / G): the
// bytes are even to within one tile however ragged the lengths are.  An item
// whose tiles lie in several CTAs leaves one unnormalized partial per CTA (a
// CTA has at most two: its first and its last item), which the join kernel
// joins in order; an item inside one CTA is written directly.
//
// What bounds it.  Long caches: the bytes of K and V (32 sequences of 2000 .. 32768
// tokens, 8 key heads of 128, e4m3, 4 query heads each: 147 us, 75 % of the copy
// rate).  Short calls: a chain of latencies -- schedule, page id, first tile, softmax,
// join -- of about 11 us (one token over 517 of head size 256).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ptx.cuh"
#include "vw4_internal.cuh"

namespace vw4 {

// ------------------------------------------------------------- schedule
struct AttnSeq {
    int len;   // cache length, clamped to the table
    int p0;    // position of the first verify row (negative: that row is not in the cache)
    int ns;    // leading tiles that hold the visible first tokens
    int skip;  // tiles between them and the window
    int nt;    // tiles to read
};

// The tiles of tk keys that some row of a sequence sees.
__host__ __device__ inline AttnSeq attn_seq(int len_raw, int cap, int R, int window, int sinks,
                                            int tk) {
    AttnSeq s;
    s.len = len_raw < 0 ? 0 : (len_raw > cap ? cap : len_raw);
    s.p0 = s.len - R;
    s.ns = 0;
    s.skip = 0;
    s.nt = (s.len + tk - 1) / tk;
    if (window > 0 && s.nt > 0) {
        const int lo = s.p0 - window + 1 > 0 ? s.p0 - window + 1 : 0;  // first key of the window
        const int first = sinks < lo ? sinks : lo;
        s.ns = (first + tk - 1) / tk;
        s.skip = lo / tk > s.ns ? lo / tk - s.ns : 0;
        s.nt -= s.skip;
    }
    return s;
}

// Of a grid, attn_ctas take part (one unit at least for each); units
// [attn_unit(i), attn_unit(i + 1)) are CTA i's; attn_owner inverts that.
__host__ __device__ inline int attn_ctas(long long T, int grid) {
    return T < grid ? static_cast<int>(T) : grid;
}
__host__ __device__ inline long long attn_unit(long long T, int G, int i) { return T * i / G; }
__host__ __device__ inline int attn_owner(long long T, int G, long long u) {
    if (T < (1ll << 32) / (kAttnMaxGrid64 + 1))  // (T (G + 1) in 32 bits: a short division)
        return static_cast<int>((static_cast<uint32_t>(u + 1) * static_cast<uint32_t>(G) +
                                 static_cast<uint32_t>(T) - 1u) / static_cast<uint32_t>(T)) - 1;
    return static_cast<int>(((u + 1) * G + T - 1) / T - 1);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The factor of an e4m3 cache's scores is |k_scale| (its sign goes to the queries, so that
// the running maximum is that of the true scores), and at least this: times minus infinity,
// what is masked, it must not be NaN.  Scores are below 2^32 there, so a smaller factor
// gives the same weights, all 1.
constexpr float kMinFactor = 1.17549435e-38f;

// The f16 weights of e4m3 caches carry a power of two, and their sum with them: f16 ends at
// 2^-25, and under one large weight thousands of small ones are a part of the output that
// shows (a token of weight 1 whose values are zeros over a thousand of 2^-26: all of it).
// Weights of at most 2^12, or 2^8 times 2^6 where the maximum lags behind (attn_tc.cuh),
// leave f16 room for what the exponents' rounding adds to very large scores.
constexpr float kTailBits = 12.f, kTailBitsTc = 6.f;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

#ifdef __CUDACC__
// ------------------------------------------------------------ primitives
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
template <bool HALF>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    if (HALF)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool HALF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if (HALF) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// two e4m3 bytes (the low 16 bits) -> f16x2, exact
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
        : "=r"(r) : "r"(b));
    return r;
}

// four f16 values (two pairs) as e4m3 bytes hi + lo: hi the nearest, lo the nearest to
// the rest, which f16 holds exactly
__device__ __forceinline__ void e4m3_terms(uint32_t ab, uint32_t cd, uint32_t& hi, uint32_t& lo) {
    uint16_t h0, h1, l0, l1;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h0) : "r"(ab));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h1) : "r"(cd));
    uint32_t r0, r1;
    asm("{\n\t.reg .b32 t;\n\tcvt.rn.f16x2.e4m3x2 t, %1;\n\tsub.rn.f16x2 %0, %2, t;\n\t}"
        : "=r"(r0) : "h"(h0), "r"(ab));
    asm("{\n\t.reg .b32 t;\n\tcvt.rn.f16x2.e4m3x2 t, %1;\n\tsub.rn.f16x2 %0, %2, t;\n\t}"
        : "=r"(r1) : "h"(h1), "r"(cd));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(l0) : "r"(r0));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(l1) : "r"(r1));
    hi = h0 | (static_cast<uint32_t>(h1) << 16);
    lo = l0 | (static_cast<uint32_t>(l1) << 16);
}

// ------------------------------------------------------- units and pages
constexpr int kUnitFirst = 1;  // first / last tile of this CTA's part of an item
constexpr int kUnitLast = 2;
constexpr int kUnitEdge = 4;   // some row does not see some key of the tile

struct AttnUnit {  // what a tile is, from the producer to the other warps
    int b, g, start, len;
    int p0, flags;
    int slot;  // partial slot of the item's part, or -1: written directly
    int seg;   // part number within the CTA
};
constexpr int kUnitRing = 16;

// the rows of block rb of key head h: row r is verify index i, query head hq
struct AttnRow {
    int i, hq;
    bool live;
};
__device__ __forceinline__ AttnRow attn_row(const AttnParams& p, int g, int r) {
    const int h = g / p.row_blocks, rb = g - h * p.row_blocks;
    const int bt = rb / p.blocks_g, bg = rb - bt * p.blocks_g;
    const int t = r / p.gb, q = r - t * p.gb;
    AttnRow a;
    a.i = bt * p.tb + t;
    const int gq = bg * p.gb + q;
    a.hq = h * p.G + gq;
    a.live = t < p.tb && a.i < p.R && gq < p.G;
    return a;
}

__device__ __forceinline__ bool key_seen(int j, int p, int window, int sinks) {
    return j <= p && (window == 0 || j > p - window || j < sinks);
}
// seen by some row of the sequence / by every row (j < len)
__device__ __forceinline__ bool key_some(int j, int len, int p0, int window, int sinks) {
    return j < len && (window == 0 || j > p0 - window || j < sinks);
}
__device__ __forceinline__ bool key_all(int j, int len, int p0, int window, int sinks) {
    return j <= p0 && (window == 0 || j > len - 1 - window || j < sinks);
}

// Where this CTA's units begin, by a scan over the sequences' unit counts; CTA
// 0 leaves the scan for the join kernel.  All threads of the block call it.
struct AttnSpan {
    long long u0, u1, base;  // units; those before sequence b
    int b;
};
template <int NT>
__device__ __forceinline__ AttnSpan attn_span(const AttnParams& p, int cap, int tk) {
    __shared__ long long s_scan[NT / 32];
    __shared__ long long s_base;
    __shared__ int s_b;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + NT - 1) / NT;
    long long mine = 0;
    for (int k = 0; k < per; ++k) {
        const int b = tid * per + k;
        if (b < p.B)
            mine += static_cast<long long>(
                        attn_seq(p.seq_lens[b], cap, p.R, p.window, p.sinks, tk).nt) * p.groups;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    long long T = 0, at = incl - mine;  // units before this thread's sequences
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) at += s_scan[w];
        T += s_scan[w];
    }
    const int G = attn_ctas(T, static_cast<int>(gridDim.x)), cta = static_cast<int>(blockIdx.x);
    AttnSpan r;
    r.u0 = cta < G ? attn_unit(T, G, cta) : T;
    r.u1 = cta < G ? attn_unit(T, G, cta + 1) : T;
    if (cta == 0 || (r.u0 >= at && r.u0 < at + mine)) {
        for (int k = 0; k < per; ++k) {
            const int b = tid * per + k;
            if (b >= p.B) break;
            const long long n = static_cast<long long>(
                attn_seq(p.seq_lens[b], cap, p.R, p.window, p.sinks, tk).nt) * p.groups;
            if (cta == 0) p.base[b] = at;
            if (r.u0 >= at && r.u0 < at + n) {
                s_b = b;
                s_base = at;
            }
            at += n;
        }
    }
    if (cta == 0 && tid == 0) p.base[p.B] = T;
    __syncthreads();
    r.b = s_b;
    r.base = s_base;
    return r;
}

// A tile to load: every lane holds it, and the page of the lane's box.
struct AttnTile {
    int start, h, box_rows;
    int page;  // -1: no box to load
    // A part of the tile of K or V: keys from .. from + KEYS, BLKS blocks of BOXB
    // bytes of a key from block blk of ALL on.  In shared memory it is atoms of 8 keys x
    // BOXB bytes, the blocks of 8 keys next to each other.  Its bytes (the boxes that
    // some row sees), and its load, one box a page where the layout of the cache lets
    // the head be a coordinate of the blocks (heads next to each other) or of the
    // groups of 8 tokens (heads above tokens); a box an atom else.
    template <int KEYS, int BLKS, int BOXB>
    __device__ __forceinline__ uint32_t bytes(int from, int lane) const {
        const int key = lane * box_rows;
        return __popc(__ballot_sync(0xffffffffu, page >= 0 && key >= from && key < from + KEYS)) *
               static_cast<uint32_t>(box_rows * BLKS * BOXB);
    }
    template <int KEYS, int BLKS, int ALL, int BOXB, int ESZ>
    __device__ __forceinline__ void load(const AttnParams& p, const CUtensorMap* map, uint32_t dst,
                                         uint64_t* bar, int from, int blk, int lane) const {
        const int key = lane * box_rows;
        if (page >= 0 && key >= from && key < from + KEYS) {
            const int token = (start + key) & (p.page_size - 1);
            dst += (key - from) * (BLKS * BOXB);
            if (p.fold != kFoldNone) {
                tma_load_5d(dst, map, 0, 0, p.fold == kFoldBlocks ? h * ALL + blk : blk,
                            (p.fold == kFoldGroups ? h * p.fold_step : 0) + (token >> 3), page, bar);
            } else {
#pragma unroll 1
                for (int t = 0; t < box_rows; t += 8)
#pragma unroll 1
                    for (int k = 0; k < BLKS; ++k)
                        tma_load_4d(dst + (t * BLKS + k * 8) * BOXB, map, (blk + k) * (BOXB / ESZ), h,
                                    token + t, page, bar);
            }
        }
        __syncwarp();
    }
};

// The producer warps' walk over the CTA's units.  Every lane holds the walk;
// lane l also holds the page of the l-th box of the current tile.
template <int TK>
struct AttnWalk {
    int b, g, t, u, n, seg, cap;
    AttnSeq s;
    int box_rows, boxes;  // tokens of a page box, boxes of a tile
    int page;             // of this lane's box, as read (on its way until it is used)
    bool want;            // some row sees a key of that box
    __device__ __forceinline__ int start() const { return (t < s.ns ? t : t + s.skip) * TK; }
    __device__ __forceinline__ void fetch(const AttnParams& p, int lane) {
        const int lo = start() + lane * box_rows;
        want = false;
        if (lane < boxes && lo < s.len) {
            const int hi = min(lo + box_rows, s.len) - 1;
            want = p.window == 0 || hi > s.p0 - p.window || lo < p.sinks;
        }
        if (want)
            page = __ldg(p.table + static_cast<long long>(b) * p.table_stride + (lo >> p.page_shift));
    }
    __device__ __forceinline__ void enter(const AttnParams& p, int lane) {
        const int raw = p.seq_lens[b];
        s = attn_seq(raw, cap, p.R, p.window, p.sinks, TK);
        if (raw > cap && lane == 0) atomicOr(p.status, kStatusBadPage);
    }
    __device__ __forceinline__ void begin(const AttnParams& p, const AttnSpan& w, int cap_, int lane) {
        cap = cap_;
        b = w.b;
        u = 0;
        n = static_cast<int>(w.u1 - w.u0);
        seg = 0;
        box_rows = p.box_rows;
        boxes = TK / box_rows;
        enter(p, lane);
        const long long r = w.u0 - w.base;
        g = static_cast<int>(r / s.nt);
        t = static_cast<int>(r - static_cast<long long>(g) * s.nt);
        fetch(p, lane);
    }
    __device__ __forceinline__ AttnUnit unit(const AttnParams& p) const {
        AttnUnit d;
        d.b = b;
        d.g = g;
        d.start = start();
        d.len = s.len;
        d.p0 = s.p0;
        const bool edge = d.start + TK > s.p0 + 1 ||
                          (p.window > 0 && d.start <= s.len - 1 - p.window && d.start + TK > p.sinks);
        d.flags = (u == 0 || t == 0 ? kUnitFirst : 0) |
                  (u == n - 1 || t == s.nt - 1 ? kUnitLast : 0) | (edge ? kUnitEdge : 0);
        // a part that does not begin with the item's first tile is the CTA's first; one
        // that does not end with its last tile (read for a part's last unit) is the last
        const int cta = static_cast<int>(blockIdx.x);
        d.slot = u - t < 0 ? 2 * cta : (t != s.nt - 1 ? 2 * cta + 1 : -1);
        d.seg = seg;
        return d;
    }
    // to the next unit (not past the last)
    __device__ __forceinline__ void next(const AttnParams& p, int lane) {
        ++u;
        if (++t == s.nt) {
            t = 0;
            ++seg;
            if (++g == p.groups) {
                g = 0;
                do {
                    ++b;
                    enter(p, lane);
                } while (s.nt == 0);
            }
        }
        fetch(p, lane);
    }
    // The current tile, for its loads after the walk has moved on (so that the next
    // tile's pages are on their way meanwhile).  A page outside the cache becomes
    // num_pages, which reads as zeros.
    __device__ __forceinline__ AttnTile tile(const AttnParams& p) const {
        AttnTile t;
        t.start = start();
        t.h = g / p.row_blocks;
        t.box_rows = box_rows;
        t.page = want ? page : -1;
        if (want && (page < 0 || page >= p.num_pages)) {
            t.page = p.num_pages;
            atomicOr(p.status, kStatusBadPage);
        }
        return t;
    }
};

// The queries of an item's row block: a box of tb tokens x gb heads x 64
// dimensions a block, so that row r is token r / gb, head r % gb.
__device__ __forceinline__ uint32_t attn_q_bytes(const AttnParams& p, int D) {
    return static_cast<uint32_t>(p.tb * p.gb * D * 2);
}
template <int D>
__device__ __forceinline__ void attn_load_q(const AttnParams& p, const CUtensorMap* map, uint32_t dst,
                                            int block, const AttnUnit& d, uint64_t* bar) {
    const int h = d.g / p.row_blocks, rb = d.g - h * p.row_blocks;
    const int bt = rb / p.blocks_g, bg = rb - bt * p.blocks_g;
#pragma unroll
    for (int k = 0; k < D / 64; ++k)
        tma_load_3d(dst + k * block, map, k * 64, h * p.G + bg * p.gb, d.b * p.R + bt * p.tb, bar);
}

// ------------------------------------------------------- up to 16 query rows
// Four warps share the 16 rows and take a quarter of a tile's keys each, so
// every key and value byte is read from shared memory once; a fifth warp loads
// K and a sixth V (TMA, a box per page and 128 bytes of a key) into a ring.  The
// warps' running maxima, sums and outputs are joined at the end of an item's part.
// (16 rows fill a quarter of what a tcgen05 tile multiplies; the legacy matrix
// instructions keep ahead of the bytes here.)
template <int D, bool F8>
struct AttnShape {
    static constexpr int kWarps = 4;
    static constexpr int kThreads = (kWarps + 2) * 32;
    static constexpr int kTK = F8 ? 128 : 64;
    static constexpr int kRows = 16;
    static constexpr int kRB = D * (F8 ? 1 : 2);         // bytes of a key
    static constexpr int kBoxB = kRB < 128 ? kRB : 128;  // of them in a box
    static constexpr int kNBlk = kRB / kBoxB;
    static constexpr int kCPB = kBoxB / 16;
    static constexpr int kTile = kTK * kRB;              // 128 D bytes
    static constexpr int kStage = 2 * kTile;             // K then V
    static constexpr int kQ = kRows * D * 2;
    static constexpr int kQBlk = kRows * 128;
    static constexpr int kKW = kTK / kWarps;             // keys of a tile per warp
    static constexpr int kStages = D == 64 ? 6 : 3;
    static constexpr int kOffQ = kStages * kStage;
    static constexpr int kOffML = kOffQ + 2 * kQ;                  // float m, l [4][16]
    static constexpr int kOffRS = kOffML + 2 * kWarps * kRows * 4;  // float row scale [2][16]
    static constexpr int kSmem = kOffRS + 2 * kRows * 4 + 1024;
    static_assert(kWarps * kRows * D * 4 <= kStage, "the join of the warps uses a consumed stage");
    static_assert(kSmem <= 225 * 1024, "shared memory");
    __device__ static __forceinline__ uint32_t at(int row, int chunk) {  // chunk of 16 bytes of a key
        const int x = kBoxB == 64 ? (row >> 1) & 3 : row & 7;
        return static_cast<uint32_t>(((row >> 3) * kNBlk + chunk / kCPB) * (8 * kBoxB) +
                                     (row & 7) * kBoxB + (((chunk % kCPB) ^ x) << 4));
    }
    __device__ static __forceinline__ uint32_t q_at(int row, int chunk) {  // 16 bytes of a query
        return static_cast<uint32_t>((chunk >> 3) * kQBlk + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
    }
};

template <int D, bool F8, int MINB>
__global__ void __launch_bounds__(AttnShape<D, F8>::kThreads, MINB)
    attn_kernel(const AttnParams p, const __grid_constant__ AttnMaps maps) {
    using S = AttnShape<D, F8>;
    constexpr int TK = S::kTK, NST = S::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ __align__(8) uint64_t b_full[NST], b_empty[NST], b_qe[2], b_sync;
    __shared__ AttnUnit s_unit[kUnitRing];
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, lane = tid & 31, wk = tid >> 5;
    const uint32_t sm = smem_u32(smem);
    float* s_m = reinterpret_cast<float*>(smem + S::kOffML);
    float* s_l = s_m + S::kWarps * S::kRows;
    float* s_rs = reinterpret_cast<float*>(smem + S::kOffRS);

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 128) {
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
        tma_prefetch_desc(&maps.q);
    }
    if (tid == 0) {
        for (int k = 0; k < NST; ++k) {
            mbar_init(&b_full[k], 2);
            mbar_init(&b_empty[k], S::kWarps);
        }
        mbar_init(&b_qe[0], S::kWarps);
        mbar_init(&b_qe[1], S::kWarps);
        mbar_init(&b_sync, S::kWarps);
        fence_barrier_init();
        s_abort = 0;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int cap = p.max_blocks * p.page_size;
    const AttnSpan span = attn_span<S::kThreads>(p, cap, TK);
    const int n_units = static_cast<int>(span.u1 - span.u0);
    if (n_units == 0) return;
    // the same answer in every lane: what follows is executed by whole warps
    auto wait = [&](uint64_t* bar, int phase) {
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
            const uint32_t bytes = t.template bytes<TK, S::kNBlk, S::kBoxB>(0, lane);
            if (lane == 0) {
                if (keys) s_unit[u % kUnitRing] = d;
                mbar_arrive_expect_tx(&b_full[st], bytes + (q ? attn_q_bytes(p, D) : 0u));
                if (q)
                    attn_load_q<D>(p, &maps.q, sm + S::kOffQ + (d.seg & 1) * S::kQ, S::kQBlk, d,
                                   &b_full[st]);
            }
            __syncwarp();
            t.template load<TK, S::kNBlk, S::kNBlk, S::kBoxB, F8 ? 1 : 2>(
                p, keys ? &maps.k : &maps.v, sm + st * S::kStage + (keys ? 0 : S::kTile), &b_full[st],
                0, 0, lane);
        }
        // copies in flight land before the block ends
        if (u < n_units) {
            for (int k = u > NST ? u - NST : 0; k < u; ++k)
                mbar_wait_bounded(&b_full[k % NST], (k / NST) & 1, p.wait_ns, nullptr);
        }
        return;
    }

    // ---- compute state
    float o[D / 8][4];
    float m[2], l[2], c2[2];
    int pr[2];   // positions of this thread's two rows (below 0: sees nothing)
    AttnRow ar[2];
    const int r0 = lane >> 2, t4 = lane & 3;
    // ldmatrix lane addresses: (row, chunk) of the 8x8 matrices, see each use
    const int lm = lane >> 3, lr = lane & 7;
    int syncs = 0;
    auto warps_sync = [&] {  // the four warps (a wait with a limit, like every other)
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_sync);
        return wait(&b_sync, syncs++);
    };

    for (int done = 0; done < n_units; ++done) {
        const int st = done % NST;
        if (!wait(&b_full[st], done / NST)) break;
        const AttnUnit td = s_unit[done % kUnitRing];
        const int h = td.g / p.row_blocks;
        const int qslot = td.seg & 1;
        const uint32_t qs = sm + S::kOffQ + qslot * S::kQ;
        if (td.flags & kUnitFirst) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
            const float ks = F8 && p.k_scale ? __ldg(p.k_scale + h) : 1.f;
            if (F8) {
                // The queries become f16 under a power of two per row that puts the row's
                // largest magnitude into [2^14, 2^15), and the sign of the head's scale: exact
                // for every value down to 2^-31 of it (bf16 has 8 significant bits, f16 11
                // and subnormals).
                // Within 16 dimensions the order is that of the byte loads of K below.
                for (int r = wk; r < S::kRows; r += S::kWarps) {
                    uint32_t* row = reinterpret_cast<uint32_t*>(smem + S::kOffQ + qslot * S::kQ);
                    float v[D / 32];
                    uint32_t x[D / 64];
                    float mx = 0.f;
#pragma unroll
                    for (int k = 0; k < D / 64; ++k) {
                        const int e = lane + 32 * k;  // pair of dimensions 2e, 2e + 1
                        x[k] = row[(S::q_at(r, e >> 2) >> 2) + (e & 3)];
                        v[2 * k] = __uint_as_float(x[k] << 16);
                        v[2 * k + 1] = __uint_as_float(x[k] & 0xffff0000u);
                        mx = fmaxf(mx, fmaxf(fabsf(v[2 * k]), fabsf(v[2 * k + 1])));
                    }
#pragma unroll
                    for (int s = 16; s > 0; s >>= 1)
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
                    const int ex = static_cast<int>(__float_as_uint(mx) >> 23);
                    int sh = ex == 0 || ex == 255 ? 0 : 127 + 14 - ex;  // amax * 2^sh in [2^14, 2^15)
                    sh = max(-126, min(126, sh));
                    const float up = copysignf(
                        __uint_as_float(static_cast<uint32_t>(127 + sh) << 23), ks);
                    if (lane == 0)
                        s_rs[qslot * S::kRows + r] =
                            __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < D / 64; ++k) {
                        const int e = lane + 32 * k;
                        // pair (4t, 4t+1) -> stored pair t, (4t+2, 4t+3) -> stored pair t + 4
                        const int w = e & 7, s = (e & ~7) + (w >> 1) + (w & 1) * 4;
                        row[(S::q_at(r, s >> 2) >> 2) + (s & 3)] =
                            pack2<true>(v[2 * k] * up, v[2 * k + 1] * up);
                    }
                }
                fence_async_smem();  // (a later load will write there)
                if (!warps_sync()) break;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                m[k] = -INFINITY;
                l[k] = 0.f;
                ar[k] = attn_row(p, td.g, r0 + 8 * k);
                pr[k] = ar[k].live ? td.p0 + ar[k].i : -1;
                c2[k] = p.scale * kLog2e * fabsf(ks);
                if (F8) {
                    c2[k] *= s_rs[qslot * S::kRows + r0 + 8 * k];
                    if (c2[k] < kMinFactor) c2[k] = kMinFactor;  // (NaN stays)
                }
            }
        }
        const bool edge = td.flags & kUnitEdge;
        const uint32_t kS = sm + st * S::kStage, vS = kS + S::kTile;
        if (edge) {
            // values that no row sees are made zeros, whatever the cache holds there (0
            // times an infinity would not be 0); each warp cleans its own keys
#pragma unroll 1
            for (int c = lane; c < S::kKW * (S::kRB / 16); c += 32) {
                const int row = wk * S::kKW + c / (S::kRB / 16);
                if (!key_some(td.start + row, td.len, td.p0, p.window, p.sinks))
                    *reinterpret_cast<uint4*>(smem + st * S::kStage + S::kTile +
                                              S::at(row, c % (S::kRB / 16))) = make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
            __syncwarp();
        }

        const int k0 = wk * S::kKW;            // this warp's first key of the tile
        const int j0 = td.start + k0, j1 = min(j0 + S::kKW, td.len) - 1;
        // (the same for the warp) some row sees some of them
        if (j1 >= j0 && (p.window == 0 || j1 > td.p0 - p.window || j0 < p.sinks)) {
            float s[S::kKW / 8][4];
#pragma unroll
            for (int n = 0; n < S::kKW / 8; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
            if (!F8) {
#pragma unroll 4
                for (int ks = 0; ks < D / 16; ++ks) {
                    uint32_t a[4];
                    ldsm4(a, qs + S::q_at(lr + (lm & 1) * 8, ks * 2 + (lm >> 1)));
#pragma unroll
                    for (int n = 0; n < S::kKW / 16; ++n) {
                        uint32_t bk[4];
                        ldsm4(bk, kS + S::at(k0 + n * 16 + lr + (lm >> 1) * 8, ks * 2 + (lm & 1)));
                        mma16816<false>(s[2 * n], a, bk[0], bk[1]);
                        mma16816<false>(s[2 * n + 1], a, bk[2], bk[3]);
                    }
                }
            } else {
                // one byte matrix holds 16 dimensions of 8 keys: bytes 4t, 4t+1 and
                // 4t+2, 4t+3 of a lane are the two operand registers of a k step
#pragma unroll 2
                for (int ks = 0; ks < D / 32; ++ks) {
                    uint32_t a[2][4];
                    ldsm4(a[0], qs + S::q_at(lr + (lm & 1) * 8, ks * 4 + (lm >> 1)));
                    ldsm4(a[1],
                          qs + S::q_at(lr + (lm & 1) * 8, ks * 4 + 2 + (lm >> 1)));
#pragma unroll
                    for (int n = 0; n < S::kKW / 16; ++n) {
                        uint32_t bk[4];
                        ldsm4(bk, kS + S::at(k0 + n * 16 + lr + (lm >> 1) * 8, ks * 2 + (lm & 1)));
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            mma16816<true>(s[2 * n], a[e], e4m3x2_f16x2(bk[e]),
                                           e4m3x2_f16x2(bk[e] >> 16));
                            mma16816<true>(s[2 * n + 1], a[e], e4m3x2_f16x2(bk[2 + e]),
                                           e4m3x2_f16x2(bk[2 + e] >> 16));
                        }
                    }
                }
            }
            if (edge) {
#pragma unroll
                for (int n = 0; n < S::kKW / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = td.start + k0 + n * 8 + t4 * 2 + (e & 1);
                        if (!key_seen(j, pr[e >> 1], p.window, p.sinks)) s[n][e] = -INFINITY;
                    }
            }
            // running maximum and sum, in units of log2 (c2 > 0)
            float corr[2];
            bool grew = false;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float mx = -INFINITY;
#pragma unroll
                for (int n = 0; n < S::kKW / 8; ++n)
                    mx = fmaxf(mx, fmaxf(s[n][2 * k], s[n][2 * k + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = fmaxf(m[k], mx);
                corr[k] = mn == m[k] ? 1.f : ex2((m[k] - mn) * c2[k]);
                grew |= mn != m[k];
                m[k] = mn;
                const float mc = mn == -INFINITY ? 0.f : mn * c2[k] - (F8 ? kTailBits : 0.f);
                float sum = 0.f;
#pragma unroll
                for (int n = 0; n < S::kKW / 8; ++n) {
                    s[n][2 * k] = ex2(fmaf(s[n][2 * k], c2[k], -mc));
                    s[n][2 * k + 1] = ex2(fmaf(s[n][2 * k + 1], c2[k], -mc));
                    sum += s[n][2 * k] + s[n][2 * k + 1];
                }
                l[k] = l[k] * corr[k] + sum;
            }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    o[n][0] *= corr[0];
                    o[n][1] *= corr[0];
                    o[n][2] *= corr[1];
                    o[n][3] *= corr[1];
                }
            }
            // P V.  The weights go to the tensor cores in the cache's operand type (bf16,
            // or f16 for an e4m3 cache): each is off by at most half a step, or 2^-37 of the
            // largest where f16 ends, and the sum l is of the unrounded ones.
            auto load_v = [&](int n, int db, uint32_t* bv) {
                // bv: operand registers of two 8-column blocks, keys (2t, 2t+1) and + 8 each
                const int row = k0 + n * 16 + lr + (lm & 1) * 8;
                if (!F8) {
                    ldsm4t(bv, vS + S::at(row, db * 2 + (lm >> 1)));
                    return;
                }
                uint32_t x[4];
                ldsm4t(x, vS + S::at(row, db * 2 + (lm >> 1)));
                // x: 2 keys x 2 dimensions a register; even and odd dimensions apart
#pragma unroll
                for (int q = 0; q < 2; ++q) {  // dimensions 32 db + 16 q ..
                    bv[4 * q] = e4m3x2_f16x2(__byte_perm(x[2 * q], 0, 0x0020));
                    bv[4 * q + 1] = e4m3x2_f16x2(__byte_perm(x[2 * q + 1], 0, 0x0020));
                    bv[4 * q + 2] = e4m3x2_f16x2(__byte_perm(x[2 * q], 0, 0x0031));
                    bv[4 * q + 3] = e4m3x2_f16x2(__byte_perm(x[2 * q + 1], 0, 0x0031));
                }
            };
            constexpr int DB = F8 ? D / 32 : D / 16;   // value loads along a key
            constexpr int VR = F8 ? 8 : 4;             // registers of one
            constexpr uint32_t kExp = F8 ? 0x7C00u : 0x7F80u;
            bool odd = false;  // an infinity or NaN among keys that some rows do not see
            if (edge) {
#pragma unroll 1
                for (int n = 0; n < S::kKW / 16; ++n)
#pragma unroll 1
                    for (int db = 0; db < DB; ++db) {
                        uint32_t bv[VR];
                        load_v(n, db, bv);
#pragma unroll
                        for (int q = 0; q < VR; ++q)
                            odd |= (bv[q] & kExp) == kExp || ((bv[q] >> 16) & kExp) == kExp;
                    }
                odd = __any_sync(0xffffffffu, odd);
            }
            if (!odd) {
#pragma unroll
                for (int n = 0; n < S::kKW / 16; ++n) {
                    const uint32_t a[4] = {pack2<F8>(s[2 * n][0], s[2 * n][1]),
                                           pack2<F8>(s[2 * n][2], s[2 * n][3]),
                                           pack2<F8>(s[2 * n + 1][0], s[2 * n + 1][1]),
                                           pack2<F8>(s[2 * n + 1][2], s[2 * n + 1][3])};
#pragma unroll
                    for (int db = 0; db < DB; ++db) {
                        uint32_t bv[VR];
                        load_v(n, db, bv);
#pragma unroll
                        for (int q = 0; q < VR / 2; ++q)
                            mma16816<F8>(o[db * (VR / 2) + q], a, bv[2 * q], bv[2 * q + 1]);
                    }
                }
            } else {
                // 0 times infinity must not reach a row that does not see the key: one
                // product per verify index, its unseen values set to zero
                const int i_lo = attn_row(p, td.g, 0).i;
                const int i_hi = min(p.R, i_lo + p.tb) - 1;
#pragma unroll 1
                for (int i = i_lo; i <= i_hi; ++i)
#pragma unroll
                    for (int n = 0; n < S::kKW / 16; ++n) {
                        const bool a0 = ar[0].live && ar[0].i == i, a1 = ar[1].live && ar[1].i == i;
                        const uint32_t a[4] = {
                            a0 ? pack2<F8>(s[2 * n][0], s[2 * n][1]) : 0u,
                            a1 ? pack2<F8>(s[2 * n][2], s[2 * n][3]) : 0u,
                            a0 ? pack2<F8>(s[2 * n + 1][0], s[2 * n + 1][1]) : 0u,
                            a1 ? pack2<F8>(s[2 * n + 1][2], s[2 * n + 1][3]) : 0u};
                        uint32_t keep[2];
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int j = td.start + k0 + n * 16 + q * 8 + t4 * 2;
                            keep[q] = (key_seen(j, td.p0 + i, p.window, p.sinks) ? 0xffffu : 0u) |
                                      (key_seen(j + 1, td.p0 + i, p.window, p.sinks) ? 0xffff0000u
                                                                                     : 0u);
                        }
#pragma unroll
                        for (int db = 0; db < DB; ++db) {
                            uint32_t bv[VR];
                            load_v(n, db, bv);
                            // rows of other indexes multiply what is kept: zero by a
                            // value that index i sees, which may itself be an infinity,
                            // so their accumulators are put back
#pragma unroll
                            for (int q = 0; q < VR / 2; ++q) {
                                float* oq = o[db * (VR / 2) + q];
                                const float sv[4] = {oq[0], oq[1], oq[2], oq[3]};
                                mma16816<F8>(oq, a, bv[2 * q] & keep[0], bv[2 * q + 1] & keep[1]);
                                if (!a0) oq[0] = sv[0], oq[1] = sv[1];
                                if (!a1) oq[2] = sv[2], oq[3] = sv[3];
                            }
                        }
                    }
            }
        }

        if (!(td.flags & kUnitLast)) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&b_empty[st]);
            continue;
        }
        // ---- end of the item's part: join the warps' keys, write out
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
            l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
        }
        if (lane == 0) mbar_arrive(&b_qe[td.seg & 1]);
        const float vs = F8 && p.v_scale ? __ldg(p.v_scale + h) : 1.f;
        float* po = nullptr;   // partial rows [rows][D], then m [rows], l [rows]
        if (td.slot >= 0) po = p.partial + static_cast<long long>(td.slot) * S::kRows * (D + 2);
        if (t4 == 0) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                s_m[wk * S::kRows + r0 + 8 * k] =
                    m[k] == -INFINITY ? -INFINITY : m[k] * c2[k] - (F8 ? kTailBits : 0.f);
                s_l[wk * S::kRows + r0 + 8 * k] = l[k];
            }
        }
        if (!warps_sync()) break;  // also: every warp is done with this stage
        float* buf = reinterpret_cast<float*>(smem + st * S::kStage);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = r0 + 8 * k;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < S::kWarps; ++w) M = fmaxf(M, s_m[w * S::kRows + r]);
            const float f = M == -INFINITY ? 1.f : ex2(s_m[wk * S::kRows + r] - M);
            float* row = buf + (wk * S::kRows + r) * D;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
                if (F8) {
                    if (n & 1) continue;
                    const int col = ((n >> 1) * 16 + t4 * 4) ^ ((r & 1) << 4);
                    *reinterpret_cast<float4*>(row + col) =
                        make_float4(o[n][2 * k] * f, o[n + 1][2 * k] * f, o[n][2 * k + 1] * f,
                                    o[n + 1][2 * k + 1] * f);
                } else {
                    const int col = (n * 8 + t4 * 2) ^ ((r & 3) << 3);
                    *reinterpret_cast<float2*>(row + col) =
                        make_float2(o[n][2 * k] * f, o[n][2 * k + 1] * f);
                }
            }
        }
        if (!warps_sync()) break;
        for (int c = tid; c < S::kRows * (D / 8); c += S::kWarps * 32) {
            const int r = c / (D / 8), blk = c % (D / 8);
            const AttnRow row = attn_row(p, td.g, r);
            if (!row.live) continue;
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < S::kWarps; ++w) M = fmaxf(M, s_m[w * S::kRows + r]);
#pragma unroll
            for (int w = 0; w < S::kWarps; ++w)
                L += s_l[w * S::kRows + r] * (M == -INFINITY ? 1.f : ex2(s_m[w * S::kRows + r] - M));
            float x[8] = {};
            const int col = F8 ? (blk * 8) ^ ((r & 1) << 4) : (blk * 8) ^ ((r & 3) << 3);
#pragma unroll
            for (int w = 0; w < S::kWarps; ++w) {
                const float4* src = reinterpret_cast<const float4*>(buf + (w * S::kRows + r) * D + col);
                const float4 u = src[0], v = src[1];
                x[0] += u.x; x[1] += u.y; x[2] += u.z; x[3] += u.w;
                x[4] += v.x; x[5] += v.y; x[6] += v.z; x[7] += v.w;
            }
            const long long orow = static_cast<long long>(td.b) * p.R + row.i;
            if (td.slot >= 0) {
                float4* dst = reinterpret_cast<float4*>(po + r * D + blk * 8);
                dst[0] = make_float4(x[0], x[1], x[2], x[3]);
                dst[1] = make_float4(x[4], x[5], x[6], x[7]);
                if (blk == 0) {
                    po[S::kRows * D + r] = M;
                    po[S::kRows * (D + 1) + r] = L;
                }
            } else {
                const float f = L == 0.f ? 0.f : vs / L;
                __nv_bfloat16* out = p.out + orow * p.ldo + static_cast<long long>(row.hq) * D;
                *reinterpret_cast<uint4*>(out + blk * 8) =
                    make_uint4(pack2<false>(x[0] * f, x[1] * f), pack2<false>(x[2] * f, x[3] * f),
                               pack2<false>(x[4] * f, x[5] * f), pack2<false>(x[6] * f, x[7] * f));
                if (blk == 0 && p.lse)
                    p.lse[orow * p.Hq + row.hq] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
            }
        }
        fence_async_smem();  // the stage was written here; the next load writes it again
        if (!warps_sync()) break;  // (also before s_m and s_l are written again)
        if (lane == 0) mbar_arrive(&b_empty[st]);
    }
}

// The kernel's attributes and occupancy, once per device, and its launch on
// min(*grid, resident CTAs) CTAs (written back to *grid).
template <class K>
cudaError_t attn_launch(K kernel, int threads, int smem, std::atomic<unsigned long long>& once,
                        std::atomic<int>& occ, const AttnParams& p, const AttnMaps& maps, int* grid,
                        int sms, cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (!bit || !(once.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        int n = 0;
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
        if (e != cudaSuccess) return e;
        occ.store(n < 1 ? 1 : n);
        once.fetch_or(bit, std::memory_order_acq_rel);
    }
    const int resident = sms * occ.load();
    if (*grid > resident) *grid = resident;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(*grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, maps);
}
}  // namespace vw4

#include "attn_tc.cuh"

namespace vw4 {

template <int D, bool F8>
cudaError_t attn_dispatch_rows(const AttnParams& p, const AttnMaps& maps, int rows, int* grid, int sms,
                               cudaStream_t s) {
    static std::atomic<unsigned long long> once[3];
    static std::atomic<int> occ[3];
    constexpr int kMinBlocks = D == 256 ? 1 : 2;
    if (rows == 16)
        return attn_launch(attn_kernel<D, F8, kMinBlocks>, AttnShape<D, F8>::kThreads,
                           AttnShape<D, F8>::kSmem, once[0], occ[0], p, maps, grid, sms, s);
    if (rows == 64)
        return attn_launch(attn_tc_kernel<D, F8, 64>, AttnTcShape<D, F8, 64>::kThreads,
                           AttnTcShape<D, F8, 64>::kSmem, once[1], occ[1], p, maps, grid, sms, s);
    if constexpr (!(F8 && D == 256))
        return attn_launch(attn_tc_kernel<D, F8, 128>, AttnTcShape<D, F8, 128>::kThreads,
                           AttnTcShape<D, F8, 128>::kSmem, once[2], occ[2], p, maps, grid, sms, s);
    return cudaErrorInvalidValue;
}

template <int D>
cudaError_t attn_dispatch(const AttnParams& p, const AttnMaps& maps, bool f8, int rows, int* grid,
                          int sms, cudaStream_t s) {
    return f8 ? attn_dispatch_rows<D, true>(p, maps, rows, grid, sms, s)
              : attn_dispatch_rows<D, false>(p, maps, rows, grid, sms, s);
}
#endif  // __CUDACC__

}  // namespace vw4
