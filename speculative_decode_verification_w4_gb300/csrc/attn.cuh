// attn.cuh -- attention of the verify rows over a paged key-value cache: the
// work schedule, and the kernel as a template over the head size, the cache
// type and the warp layout (instantiated per head size in attn_d*.cu).
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
// CTA has at most two: its first and its last item), which the combine kernel
// joins in order; an item inside one CTA is written directly.
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
    return static_cast<int>(((u + 1) * G + T - 1) / T - 1);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

#ifdef __CUDACC__
// ------------------------------------------------------------ primitives
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;"); }
// all but the newest `newer` groups of this thread have landed
__device__ __forceinline__ void cp_async_wait(int newer) {
    if (newer >= 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (newer == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (newer == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}
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

// ---------------------------------------------------------------- layout
// TK keys of K and of V are one ring stage.  Rows of RB bytes are kept in
// 16-byte chunks whose index is exclusive-ored with the row, so that the 8
// rows of a matrix load fall into different banks.
template <int D, bool F8, int WR, int WK>
struct AttnShape {
    static constexpr int kWarps = WR * WK;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kTK = F8 ? 128 : 64;
    static constexpr int kRows = 16 * WR;            // query rows of an item
    static constexpr int kRB = D * (F8 ? 1 : 2);     // bytes of a key
    static constexpr int kCH = kRB / 16;             // 16-byte chunks of a key
    static constexpr int kTile = kTK * kRB;          // 128 D bytes
    static constexpr int kStage = 2 * kTile;         // K then V
    static constexpr int kQ = kRows * D * 2;         // bf16 queries (f16 for an e4m3 cache)
    static constexpr int kKW = kTK / WK;             // keys of a tile per warp
    static constexpr int kSB = kKW < 32 ? kKW : 32;  // keys per softmax step
    static constexpr int kStages =
        D == 256 ? (WR >= 4 ? 2 : 3) : (D == 128 && WR < 8 ? (WR == 4 ? 2 : 3) : 4);
    static constexpr int kOffQ = kStages * kStage;
    static constexpr int kOffML = kOffQ + 2 * kQ;              // float m, l [WK][rows]
    static constexpr int kOffRS = kOffML + 2 * WK * kRows * 4;  // float row scale [2][rows]
    static constexpr int kOffDesc = kOffRS + 2 * kRows * 4;
    static constexpr int kSmem = kOffDesc + kStages * 64 + 64;
    static_assert(WK == 1 || WK * kRows * D * 4 <= kStage, "the merge uses a consumed stage");
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ uint32_t swz(int row, int chunk, int rb) {
    // 64-byte rows: two rows share a 128-byte line
    const int x = rb == 64 ? ((row >> 1) & 3) : (row & 7);
    return static_cast<uint32_t>(row * rb + ((chunk ^ x) << 4));
}

struct AttnTile {  // what a ring stage holds
    int b, g, start;      // sequence, (key head, row block), first key
    int len, p0;
    int seg;              // segment of this CTA's units (query slot: seg & 1)
    int flags;
    int slot;             // partial slot, or -1: written directly
};
constexpr int kTileFirst = 1, kTileLast = 2;

__device__ __forceinline__ bool key_seen(int j, int p, int window, int sinks) {
    return j <= p && (window == 0 || j > p - window || j < sinks);
}

// ---------------------------------------------------------------- kernel
template <int D, bool F8, int WR, int WK, int MINB>
__global__ void __launch_bounds__(AttnShape<D, F8, WR, WK>::kThreads, MINB)
    attn_kernel(const AttnParams p) {
    using S = AttnShape<D, F8, WR, WK>;
    constexpr int NT = S::kThreads, TK = S::kTK;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ long long s_scan[S::kWarps];
    __shared__ long long s_base;
    __shared__ int s_b;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wr = warp % WR, wk = warp / WR;
    const uint32_t sm = smem_u32(smem);
    float* s_m = reinterpret_cast<float*>(smem + S::kOffML);
    float* s_l = s_m + WK * S::kRows;
    float* s_rs = reinterpret_cast<float*>(smem + S::kOffRS);
    AttnTile* s_desc = reinterpret_cast<AttnTile*>(smem + S::kOffDesc);

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // where this CTA's units begin: a scan over the sequences' unit counts
    const int cap = p.max_blocks * p.page_size;
    const int per = (p.B + NT - 1) / NT;
    long long mine = 0;
    for (int k = 0; k < per; ++k) {
        const int b = tid * per + k;
        if (b < p.B)
            mine += static_cast<long long>(
                        attn_seq(p.seq_lens[b], cap, p.R, p.window, p.sinks, TK).nt) * p.groups;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    long long T = 0, before = 0;
#pragma unroll
    for (int w = 0; w < S::kWarps; ++w) {
        if (w < warp) before += s_scan[w];
        T += s_scan[w];
    }
    const int G = attn_ctas(T, static_cast<int>(gridDim.x)), cta = static_cast<int>(blockIdx.x);
    const long long u0 = cta < G ? attn_unit(T, G, cta) : T;
    const long long u1 = cta < G ? attn_unit(T, G, cta + 1) : T;
    {
        long long at = before + incl - mine;  // units before this thread's sequences
        if (blockIdx.x == 0 || (u0 >= at && u0 < at + mine)) {
            for (int k = 0; k < per; ++k) {
                const int b = tid * per + k;
                if (b >= p.B) break;
                const long long n =
                    static_cast<long long>(
                        attn_seq(p.seq_lens[b], cap, p.R, p.window, p.sinks, TK).nt) * p.groups;
                if (blockIdx.x == 0) p.base[b] = at;  // for the combine kernel
                if (u0 >= at && u0 < at + n) {
                    s_b = b;
                    s_base = at;
                }
                at += n;
            }
        }
        if (blockIdx.x == 0 && tid == 0) p.base[p.B] = T;
    }
    __syncthreads();
    if (u0 >= u1) return;

    // ---- load cursor (the same in every thread)
    int lb = s_b, lg, lt;
    AttnSeq ls = attn_seq(p.seq_lens[lb], cap, p.R, p.window, p.sinks, TK);
    if (p.seq_lens[lb] > cap && tid == 0) atomicOr(p.status, kStatusBadPage);
    {
        const long long r = u0 - s_base;
        lg = static_cast<int>(r / ls.nt);
        lt = static_cast<int>(r - static_cast<long long>(lg) * ls.nt);
    }
    const int n_units = static_cast<int>(u1 - u0);
    int loaded = 0, l_seg = -1;
    const int ps_shift = p.page_shift;
    // lane l keeps the page of keys start + 8 l .. + 7 of the next tile to load
    auto fetch_pages = [&]() {
        const int t = lt < ls.ns ? lt : lt + ls.skip;
        const int j = t * TK + lane * 8;
        int pg = -1;
        if (lane < TK / 8 && j < ls.len) {
            pg = __ldg(p.table + static_cast<long long>(lb) * p.table_stride + (j >> ps_shift));
            // pages that no row sees may hold any id; key_seen decides below
            if (pg < 0 || pg >= p.num_pages) pg = -1;
        }
        return pg;
    };
    int pages = fetch_pages();

    auto issue = [&]() {
        const int st = loaded % S::kStages;
        const int t = lt < ls.ns ? lt : lt + ls.skip;
        const int start = t * TK;
        const int rb = lg % p.row_blocks, h = lg / p.row_blocks;
        const bool first = loaded == 0 || lt == 0;
        const bool last = loaded == n_units - 1 || lt == ls.nt - 1;
        if (first) ++l_seg;
        if (tid == 0) {
            AttnTile d;
            d.b = lb;
            d.g = lg;
            d.start = start;
            d.len = ls.len;
            d.p0 = ls.p0;
            d.seg = l_seg;
            d.flags = (first ? kTileFirst : 0) | (last ? kTileLast : 0);
            // a segment that does not begin with the item's first tile is the CTA's first;
            // one that does not end with its last tile is the CTA's last
            const bool cut_front = loaded - lt < 0;  // tile 0 lies before this CTA's units
            const bool cut_back = lt != ls.nt - 1;   // (read for the last tile of the segment)
            d.slot = cut_front ? 2 * cta : (cut_back ? 2 * cta + 1 : -1);
            s_desc[st] = d;
        }
        const uint8_t* kb = static_cast<const uint8_t*>(p.k);
        const uint8_t* vb = static_cast<const uint8_t*>(p.v);
        const uint32_t dst = sm + st * S::kStage;
        bool bad = false;
#pragma unroll 4
        for (int i = 0; i < TK * S::kCH / NT; ++i) {
            const int c = tid + i * NT;
            const int row = c / S::kCH, col = c % S::kCH;
            const int pg = __shfl_sync(0xffffffffu, pages, row >> 3);
            const int j = start + row;
            // keys that no row sees are zeros, whatever the cache holds there
            bool ok = j < ls.len && (p.window == 0 || j > ls.p0 - p.window || j < p.sinks);
            if (ok && pg < 0) {
                bad = true;
                ok = false;
            }
            const long long off =
                ok ? (static_cast<long long>(pg) * p.page_stride +
                      static_cast<long long>(j & (p.page_size - 1)) * p.token_stride +
                      static_cast<long long>(h) * p.head_stride) * (F8 ? 1 : 2) + col * 16
                   : 0;
            const uint32_t a = dst + swz(row, col, S::kRB);
            cp_async16(a, kb + off, ok ? 16 : 0);
            cp_async16(a + S::kTile, vb + off, ok ? 16 : 0);
        }
        if (bad) atomicOr(p.status, kStatusBadPage);
        if (first) {
            const uint32_t qd = sm + S::kOffQ + (l_seg & 1) * S::kQ;
            constexpr int QC = D / 8;
            for (int c = tid; c < S::kRows * QC; c += NT) {
                const int r = c / QC, col = c % QC;
                const int row = rb * S::kRows + r;  // i * G + query head of the group
                const bool ok = row < p.R * p.G;
                const int i = ok ? row / p.G : 0, gq = ok ? row - i * p.G : 0;
                const __nv_bfloat16* src = p.q + (static_cast<long long>(lb) * p.R + i) * p.ldq +
                                           (h * p.G + gq) * D + col * 8;
                cp_async16(qd + swz(r, col, D * 2), src, ok ? 16 : 0);
            }
        }
        cp_async_commit();
        ++loaded;
        if (loaded < n_units) {
            if (++lt == ls.nt) {
                lt = 0;
                if (++lg == p.groups) {
                    lg = 0;
                    do {
                        ++lb;
                        ls = attn_seq(p.seq_lens[lb], cap, p.R, p.window, p.sinks, TK);
                    } while (ls.nt == 0);
                    if (p.seq_lens[lb] > cap && tid == 0) atomicOr(p.status, kStatusBadPage);
                }
            }
            pages = fetch_pages();
        }
    };

    // ---- compute state
    float o[D / 8][4];
    float m[2], l[2], c2[2];
    int pr[2];   // positions of this thread's two rows (-1: no such row)
    int vi[2];   // their verify indexes
    const int r0 = wr * 16 + (lane >> 2);
    const int t4 = lane & 3;
    // ldmatrix lane addresses: (row, chunk) of the 8x8 matrices, see each use
    const int lm = lane >> 3, lr = lane & 7;

    for (int done = 0; done < n_units; ++done) {
        // every warp is past the tile whose stage the loads below overwrite
        __syncthreads();
        while (loaded < n_units && loaded < done + S::kStages) {
            // two query slots: a segment's queries replace those of the segment before
            // the last loaded one, which must be finished
            if (loaded > done && lt == 0 && l_seg >= 1 && s_desc[done % S::kStages].seg < l_seg)
                break;
            issue();
        }
        cp_async_wait(loaded - done - 1);
        __syncthreads();
        const int st = done % S::kStages;
        const AttnTile td = s_desc[st];
        const int rb = td.g % p.row_blocks, h = td.g / p.row_blocks;
        const int qslot = td.seg & 1;
        const uint32_t qs = sm + S::kOffQ + qslot * S::kQ;
        if (td.flags & kTileFirst) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
            const float ks = F8 && p.k_scale ? __ldg(p.k_scale + h) : 1.f;
            if (F8) {
                // The queries become f16 under a power of two per row that puts the
                // row's largest magnitude into [2^14, 2^15): exact for every value down
                // to 2^-31 of it (bf16 has 8 significant bits, f16 11 and subnormals).
                // Within 16 dimensions the order is that of the byte loads of K below.
                for (int r = warp; r < S::kRows; r += S::kWarps) {
                    uint32_t* row = reinterpret_cast<uint32_t*>(smem + S::kOffQ + qslot * S::kQ);
                    float v[D / 32];
                    uint32_t x[D / 64];
                    float mx = 0.f;
#pragma unroll
                    for (int k = 0; k < D / 64; ++k) {
                        const int e = lane + 32 * k;  // pair of dimensions 2e, 2e + 1
                        x[k] = row[(swz(r, e >> 2, D * 2) >> 2) + (e & 3)];
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
                    const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
                    if (lane == 0)
                        s_rs[qslot * S::kRows + r] =
                            __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < D / 64; ++k) {
                        const int e = lane + 32 * k;
                        // pair (4t, 4t+1) -> stored pair t, (4t+2, 4t+3) -> stored pair t + 4
                        const int w = e & 7, s = (e & ~7) + (w >> 1) + (w & 1) * 4;
                        row[(swz(r, s >> 2, D * 2) >> 2) + (s & 3)] =
                            pack2<true>(v[2 * k] * up, v[2 * k + 1] * up);
                    }
                }
                __syncthreads();
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                m[k] = -INFINITY;
                l[k] = 0.f;
                const int row = rb * S::kRows + r0 + 8 * k;
                vi[k] = row / p.G;
                pr[k] = row < p.R * p.G ? td.p0 + vi[k] : -1;
                c2[k] = p.scale * kLog2e * ks;
                if (F8) c2[k] *= s_rs[qslot * S::kRows + r0 + 8 * k];
            }
        }
        // keys that some row of the sequence does not see
        const bool edge = td.start + TK > td.p0 + 1 ||
                          (p.window > 0 && td.start <= td.len - 1 - p.window &&
                           td.start + TK > p.sinks);
        const uint32_t kS = sm + st * S::kStage, vS = kS + S::kTile;

#pragma unroll 1
        for (int sb = 0; sb < S::kKW; sb += S::kSB) {
            const int k0 = wk * S::kKW + sb;   // first key of the step within the tile
            if (td.start + k0 >= td.len) break;  // (uniform) nothing of the sequence left
            float s[S::kSB / 8][4];
#pragma unroll
            for (int n = 0; n < S::kSB / 8; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
            if (!F8) {
#pragma unroll 4
                for (int ks = 0; ks < D / 16; ++ks) {
                    uint32_t a[4];
                    ldsm4(a, qs + swz(wr * 16 + lr + (lm & 1) * 8, ks * 2 + (lm >> 1), D * 2));
#pragma unroll
                    for (int n = 0; n < S::kSB / 16; ++n) {
                        uint32_t bk[4];
                        ldsm4(bk, kS + swz(k0 + n * 16 + lr + (lm >> 1) * 8, ks * 2 + (lm & 1),
                                           S::kRB));
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
                    ldsm4(a[0], qs + swz(wr * 16 + lr + (lm & 1) * 8, ks * 4 + (lm >> 1), D * 2));
                    ldsm4(a[1],
                          qs + swz(wr * 16 + lr + (lm & 1) * 8, ks * 4 + 2 + (lm >> 1), D * 2));
#pragma unroll
                    for (int n = 0; n < S::kSB / 16; ++n) {
                        uint32_t bk[4];
                        ldsm4(bk, kS + swz(k0 + n * 16 + lr + (lm >> 1) * 8, ks * 2 + (lm & 1),
                                           S::kRB));
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
                for (int n = 0; n < S::kSB / 8; ++n)
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
                for (int n = 0; n < S::kSB / 8; ++n)
                    mx = fmaxf(mx, fmaxf(s[n][2 * k], s[n][2 * k + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = fmaxf(m[k], mx);
                corr[k] = mn == m[k] ? 1.f : ex2((m[k] - mn) * c2[k]);
                grew |= mn != m[k];
                m[k] = mn;
                const float mc = mn == -INFINITY ? 0.f : mn * c2[k];
                float sum = 0.f;
#pragma unroll
                for (int n = 0; n < S::kSB / 8; ++n) {
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
            // or f16 for an e4m3 cache): each is off by at most half a step, and the sum l
            // is of the unrounded ones.
            auto load_v = [&](int n, int db, uint32_t* bv) {
                // bv: operand registers of two 8-column blocks, keys (2t, 2t+1) and + 8 each
                const int row = k0 + n * 16 + lr + (lm & 1) * 8;
                if (!F8) {
                    ldsm4t(bv, vS + swz(row, db * 2 + (lm >> 1), S::kRB));
                    return;
                }
                uint32_t x[4];
                ldsm4t(x, vS + swz(row, db * 2 + (lm >> 1), S::kRB));
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
                for (int n = 0; n < S::kSB / 16; ++n)
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
                for (int n = 0; n < S::kSB / 16; ++n) {
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
                const int i_lo = (rb * S::kRows + wr * 16) / p.G;
                const int i_hi = min(p.R - 1, (rb * S::kRows + wr * 16 + 15) / p.G);
#pragma unroll 1
                for (int i = i_lo; i <= i_hi; ++i)
#pragma unroll
                    for (int n = 0; n < S::kSB / 16; ++n) {
                        const bool a0 = vi[0] == i, a1 = vi[1] == i;
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

        if (!(td.flags & kTileLast)) continue;
        // ---- end of the segment: join the warps' key slices, write out
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
            l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
        }
        const float vs = F8 && p.v_scale ? __ldg(p.v_scale + h) : 1.f;
        float* po = nullptr;   // partial rows [rows][D], then m [rows], l [rows]
        if (td.slot >= 0) po = p.partial + static_cast<long long>(td.slot) * S::kRows * (D + 2);
        if (WK == 1) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = r0 + 8 * k, row = rb * S::kRows + r;
                if (row >= p.R * p.G) continue;
                const float mc = m[k] == -INFINITY ? -INFINITY : m[k] * c2[k];
                const float f = td.slot >= 0 ? 1.f : (l[k] == 0.f ? 0.f : vs / l[k]);
                const long long orow = static_cast<long long>(td.b) * p.R + vi[k];
                const int hq = h * p.G + row - vi[k] * p.G;
                __nv_bfloat16* out = p.out + orow * p.ldo + static_cast<long long>(hq) * D;
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    // column of element e of block n
                    const int col = F8 ? (n >> 1) * 16 + t4 * 4 + (n & 1) : n * 8 + t4 * 2;
                    const float x = o[n][2 * k] * f, y = o[n][2 * k + 1] * f;
                    if (F8) {
                        if (n & 1) continue;
                        const float x1 = o[n + 1][2 * k] * f, y1 = o[n + 1][2 * k + 1] * f;
                        if (td.slot >= 0)
                            *reinterpret_cast<float4*>(po + r * D + col) = make_float4(x, x1, y, y1);
                        else
                            *reinterpret_cast<uint2*>(out + col) =
                                make_uint2(pack2<false>(x, x1), pack2<false>(y, y1));
                    } else if (td.slot >= 0) {
                        *reinterpret_cast<float2*>(po + r * D + col) = make_float2(x, y);
                    } else {
                        *reinterpret_cast<uint32_t*>(out + col) = pack2<false>(x, y);
                    }
                }
                if (t4 == 0) {
                    if (td.slot >= 0) {
                        po[S::kRows * D + r] = mc;
                        po[S::kRows * (D + 1) + r] = l[k];
                    } else if (p.lse) {
                        p.lse[orow * p.Hq + hq] =
                            l[k] == 0.f ? -INFINITY : (mc + log2f(l[k])) * kLn2;
                    }
                }
            }
        } else {
            if (t4 == 0) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    s_m[wk * S::kRows + r0 + 8 * k] = m[k] == -INFINITY ? -INFINITY : m[k] * c2[k];
                    s_l[wk * S::kRows + r0 + 8 * k] = l[k];
                }
            }
            __syncthreads();  // also: every warp is done with this stage
            float* buf = reinterpret_cast<float*>(smem + st * S::kStage);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = r0 + 8 * k;
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < WK; ++w) M = fmaxf(M, s_m[w * S::kRows + r]);
                const float f = M == -INFINITY ? 1.f : ex2(s_m[wk * S::kRows + r] - M);
                float* row = buf + (wk * S::kRows + r) * D;
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    if (F8) {
                        if (n & 1) continue;
                        const int col = ((n >> 1) * 16 + t4 * 4) ^ ((r & 1) << 4);
                        *reinterpret_cast<float4*>(row + col) =
                            make_float4(o[n][2 * k] * f, o[n + 1][2 * k] * f,
                                        o[n][2 * k + 1] * f, o[n + 1][2 * k + 1] * f);
                    } else {
                        const int col = (n * 8 + t4 * 2) ^ ((r & 3) << 3);
                        *reinterpret_cast<float2*>(row + col) =
                            make_float2(o[n][2 * k] * f, o[n][2 * k + 1] * f);
                    }
                }
            }
            __syncthreads();
            for (int c = tid; c < S::kRows * (D / 8); c += NT) {
                const int r = c / (D / 8), blk = c % (D / 8);
                const int row = rb * S::kRows + r;
                if (row >= p.R * p.G) break;  // later chunks are of later rows
                float M = -INFINITY, L = 0.f;
#pragma unroll
                for (int w = 0; w < WK; ++w) M = fmaxf(M, s_m[w * S::kRows + r]);
#pragma unroll
                for (int w = 0; w < WK; ++w)
                    L += s_l[w * S::kRows + r] *
                         (M == -INFINITY ? 1.f : ex2(s_m[w * S::kRows + r] - M));
                float x[8] = {};
                const int col = F8 ? (blk * 8) ^ ((r & 1) << 4) : (blk * 8) ^ ((r & 3) << 3);
#pragma unroll
                for (int w = 0; w < WK; ++w) {
                    const float4* src =
                        reinterpret_cast<const float4*>(buf + (w * S::kRows + r) * D + col);
                    const float4 u = src[0], v = src[1];
                    x[0] += u.x; x[1] += u.y; x[2] += u.z; x[3] += u.w;
                    x[4] += v.x; x[5] += v.y; x[6] += v.z; x[7] += v.w;
                }
                const int i = row / p.G, hq = h * p.G + row - i * p.G;
                const long long orow = static_cast<long long>(td.b) * p.R + i;
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
                    __nv_bfloat16* out = p.out + orow * p.ldo + static_cast<long long>(hq) * D;
                    *reinterpret_cast<uint4*>(out + blk * 8) =
                        make_uint4(pack2<false>(x[0] * f, x[1] * f), pack2<false>(x[2] * f, x[3] * f),
                                   pack2<false>(x[4] * f, x[5] * f), pack2<false>(x[6] * f, x[7] * f));
                    if (blk == 0 && p.lse)
                        p.lse[orow * p.Hq + hq] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
                }
            }
        }
    }
}

// The kernel's attributes and occupancy, once per device, and its launch on
// min(*grid, resident CTAs) CTAs (written back to *grid).
template <int D, bool F8, int WR, int WK, int MINB>
cudaError_t attn_launch(const AttnParams& p, int* grid, int sms, cudaStream_t s) {
    using S = AttnShape<D, F8, WR, WK>;
    static std::atomic<unsigned long long> once{0};
    static std::atomic<int> occ{0};
    cudaError_t e = set_attribute_per_device(once, [] {
        cudaError_t r = cudaFuncSetAttribute(attn_kernel<D, F8, WR, WK, MINB>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        int n = 0;
        if (r == cudaSuccess)
            r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                &n, attn_kernel<D, F8, WR, WK, MINB>, S::kThreads, S::kSmem);
        if (r == cudaSuccess) occ.store(n);
        return r;
    });
    if (e != cudaSuccess) return e;
    const int resident = sms * (occ.load() > 0 ? occ.load() : 1);
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
    return cudaLaunchKernelEx(&cfg, attn_kernel<D, F8, WR, WK, MINB>, p);
}

template <int D, bool F8>
cudaError_t attn_dispatch_rows(const AttnParams& p, int rows, int* grid, int sms, cudaStream_t s) {
    switch (rows) {
        case 16: return attn_launch<D, F8, 1, 4, D == 256 ? 1 : (D == 128 ? 2 : 3)>(p, grid, sms, s);
        case 32: return attn_launch<D, F8, 2, 2, D == 256 ? 1 : (D == 128 ? 2 : 3)>(p, grid, sms, s);
        case 64: return attn_launch<D, F8, 4, 1, D == 256 ? 1 : 2>(p, grid, sms, s);
    }
    if constexpr (D < 256) return attn_launch<D, F8, 8, 1, D == 64 ? 2 : 1>(p, grid, sms, s);
    return cudaErrorInvalidValue;
}

template <int D>
cudaError_t attn_dispatch(const AttnParams& p, bool f8, int rows, int* grid, int sms,
                          cudaStream_t s) {
    return f8 ? attn_dispatch_rows<D, true>(p, rows, grid, sms, s)
              : attn_dispatch_rows<D, false>(p, rows, grid, sms, s);
}
#endif  // __CUDACC__

}  // namespace vw4
