// logprobs.cu -- log probabilities of given tokens, ranks, entropy and the best
// alternatives of logits rows, in one pass over the rows.
//
// With c = scale log2(e) and a reference m that follows the running maximum of the logits,
//   Z = sum 2^(c (x - m)),   W = sum 2^(c (x - m)) c (x - m)
// and when m grows, by d = c (m' - m): W <- (W - d Z) 2^-d, Z <- Z 2^-d.  Then
//   lse = scale m + ln Z,   entropy = ln 2 (log2 Z - W / Z).
// The difference first: it is exact next to m, so that the error of an exponent goes with
// the entry's distance from m and not with the logits' size.  (A fused c x - c m is off by the
// rounding of c m, the same for all of a thread's entries and another for the next thread's:
// 4e-4 of ln Z at a logit of 10000, 12.7 where a row is masked with -1e9.)
// Each thread keeps its own m (moved where an entry exceeds it by 2^8), Z and W; they meet
// in a fixed order.  Z holds an entry of weight 1, and one of 2^-8 of any that exceeds m: no log
// probability comes out above 0.
//
// Alternatives: the block keeps the `top` largest entries as 64-bit keys (value, then lower
// index first) and lists those above the least of them; every few chunks of 4096 entries
// its threads meet and choose from the list: a candidate's place is the number of
// candidates above it, so nothing is sorted step by step.  The first chunk, where all are
// above, gets a threshold first: the ceil(top / 8)-th largest of each warp's maxima, of
// which the least has `top` entries that are not below it; and where that leaves too many
// (equal entries, warps without any), the exact one: of the `top` largest maxima of a thread
// the least has that many entries above it, which lie in that many threads.  Chunks that
// overfill the list (rows in ascending order) are read again that way.
//
// The bytes bound it (4 or 2 a logit) and, at 17 instructions a logit, the issue slots (71 % busy):
// 256 x 9 rows of 151936, of which 60 % are read, with five alternatives, take 157 us in fp32
// (124 at the copy rate; without alternatives 147) and 139 in bf16 (62; 113).  A row is split
// over blocks where the rows alone would leave SMs idle (one sequence's 8 rows of 262144: 9.2 us,
// 14.4 with 20 alternatives), and a second kernel joins the parts in order.
#include <cuda_bf16.h>
#include <algorithm>

#include "attn.cuh"

namespace vw4 {

constexpr int kLpThreads = 256;
constexpr int kLpEach = 16;                          // entries of a thread and chunk
constexpr int kLpChunk = kLpThreads * kLpEach;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kCand = kMaxTop * kLpEach;             // candidates of the list
constexpr int kCandFull = 8;                         // so many are worth choosing from
constexpr int kLpGroup = 16;                         // chunks between the block's meetings, at most
constexpr int kLpMaxSplit = 64;
constexpr long long kLpFill = 608;                   // blocks that fill the GPU (four on each of 152 SMs)
constexpr uint32_t kLpBadId = 0x10u;
constexpr float kLpLazy = 8.f;                       // log2 of an entry over its thread's reference
constexpr float kLpFar = 1024.f;                     // 2^-1024 is 0 in fp32

struct LpPart {
    float m, z, w;
    int before;   // entries before the token
};

// Parts of a row: a chunk at least where the blocks would not fill the GPU, else thirty-two
// chunks at least (each part begins with the search for a threshold), for eight times the
// blocks that fill it (no SM is left with a whole row alone at the end).
static int lp_split(long long rows, int V) {
    const long long chunks = (V + kLpChunk - 1) / kLpChunk;
    const long long fill = std::min(chunks, (kLpFill + rows - 1) / rows);
    const long long even = std::min(chunks / 32, (8 * kLpFill + rows - 1) / rows);
    const long long s = std::max(fill, even);
    return static_cast<int>(s < kLpMaxSplit ? s : kLpMaxSplit);
}
size_t logprob_workspace_bytes(long long rows, int V, int top) {
    const size_t parts = static_cast<size_t>(rows) * lp_split(rows, V);
    return (parts * (sizeof(LpPart) + static_cast<size_t>(top) * 8) + 511) & ~size_t(255);
}

// Larger keys come first: the value, then the lower index.  0: no entry.
__device__ __forceinline__ unsigned long long lp_key(float x, int v) {
    const uint32_t b = __float_as_uint(x + 0.f);  // (+0 for -0)
    const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
    return static_cast<unsigned long long>(o) << 32 | static_cast<uint32_t>(~v);
}
__device__ __forceinline__ float lp_key_value(unsigned long long k) {
    const uint32_t o = static_cast<uint32_t>(k >> 32);
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ int lp_key_index(unsigned long long k) {
    return static_cast<int>(~static_cast<uint32_t>(k));
}

struct LpSum {
    float m, z, w;
};
// The sum with its maximum moved up to m (of finite values, or -infinity).
__device__ __forceinline__ LpSum lp_move(LpSum s, float m, float c2) {
    if (s.m == m || s.z == 0.f) return LpSum{m, s.z, s.w};
    if (m == INFINITY) return LpSum{m, 0.f, 0.f};
    const float d = fminf((m - s.m) * c2, kLpFar), f = ex2(-d);
    return LpSum{m, s.z * f, fmaf(-d, s.z, s.w) * f};
}
__device__ __forceinline__ LpSum lp_add(LpSum a, LpSum b, float c2) {
    const float m = fmaxf(a.m, b.m);
    a = lp_move(a, m, c2);
    b = lp_move(b, m, c2);
    return LpSum{m, a.z + b.z, a.w + b.w};
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// log p_v, from x and the row's m and ln Z.
__device__ __forceinline__ float lp_log(const LogprobParams& p, float x, float m, float lnz) {
    if (m == INFINITY) return x == INFINITY ? -lnz : -INFINITY;
    return fmaf(x - m, p.scale, -lnz);
}
// The outputs of a row but the alternatives.
__device__ __forceinline__ void lp_write(const LogprobParams& p, long long row, LpSum s, int before,
                                         int t, float xt) {
    const float lnz = logf(s.z);
    const bool none = s.z == 0.f;  // nothing but -infinity
    const float lse = none ? -INFINITY : s.m == INFINITY ? INFINITY : fmaf(s.m, p.scale, lnz);
    if (p.lse) p.lse[row] = lse;
    if (p.entropy) p.entropy[row] = none ? 0.f : fmaxf(0.f, lnz - s.w / s.z * kLn2);
    const bool here = t >= 0 && t < p.V;
    if (p.logprob) p.logprob[row] = !here || none ? -INFINITY : lp_log(p, xt, s.m, lnz);
    if (p.rank) p.rank[row] = here ? before + 1 : 0;
}
__device__ __forceinline__ void lp_write_top(const LogprobParams& p, long long row, int k,
                                             unsigned long long key, float m, float lnz) {
    const float x = lp_key_value(key);
    const bool listed = key != 0 && x > -INFINITY;
    if (p.top_ids) p.top_ids[row * p.top + k] = listed ? lp_key_index(key) : -1;
    if (p.top_logprobs)
        p.top_logprobs[row * p.top + k] = listed ? lp_log(p, x, m, lnz) : -INFINITY;
}

// How many of n keys in shared memory are above k.
__device__ __forceinline__ int lp_above(const unsigned long long* keys, int n, unsigned long long k) {
    int r = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) r += keys[j] > k ? 1 : 0;
    return r;
}

template <bool BF16>
__global__ void __launch_bounds__(kLpThreads, 4)
    logprob_kernel(const LogprobParams p, LpPart* parts, unsigned long long* lists, int split) {
    constexpr int VEC = BF16 ? 8 : 4, N = kLpEach / VEC;  // entries of a load, loads of a chunk
    using X = std::conditional_t<BF16, uint16_t, float>;
    __shared__ unsigned long long s_best[kMaxTop], s_cand[kCand + kMaxTop], s_max[kLpThreads];
    __shared__ unsigned long long s_tau;
    __shared__ uint32_t s_first[kLpWarps];
    __shared__ int s_n;
    __shared__ LpSum s_sum[kLpWarps];
    __shared__ int s_before[kLpWarps];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x / split;
    const int part = static_cast<int>(blockIdx.x - row * split);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (p.len && static_cast<int>(row % p.R) >= __ldg(p.len + row / p.R)) return;
    const X* x = static_cast<const X*>(p.x) + row * p.ldx;
    // entries counted from the 16 bytes that hold the first one
    const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(X));
    const X* base = x - shift;
    const int chunks = (p.V + shift + kLpChunk - 1) / kLpChunk;
    const int c0 = chunks * part / split, c1 = chunks * (part + 1) / split;
    const int t = p.tokens ? __ldg(p.tokens + row) : -1;
    const bool here = t >= 0 && t < p.V;
    if (t < -1 || t >= p.V) {
        if (tid == 0 && part == 0) atomicOr(p.status, kLpBadId);
    }
    auto value = [](X raw) {
        const float f = BF16 ? __uint_as_float(static_cast<uint32_t>(raw) << 16)
                             : *reinterpret_cast<const float*>(&raw);
        return fmaxf(f, -INFINITY);  // (a NaN reads as -infinity)
    };
    const float xt = here ? value(x[t]) : INFINITY;
    const float c2 = p.scale * kLog2e;

    // The next chunk is on its way while this one is worked on.  (Without that, five blocks an SM
    // cover each other's loads, in fp32 for better and worse, by how many rows are read, which the
    // host does not know: 80 x 9 rows of 151936 80 us instead of 93 where all are, 76 instead of
    // 60 where 60 % are; 256 x 9, 60 %, 154 or, on some runs, 166 instead of 157, without
    // alternatives 136 instead of 147.  bf16 143 instead of 137.)
    uint4 next[N];
    const int end = shift + p.V;
    auto fetch = [&](int c) {
        if (c * kLpChunk >= shift && (c + 1) * kLpChunk <= end) {
            const uint4* from = reinterpret_cast<const uint4*>(base) +
                                static_cast<long long>(c) * (kLpChunk / VEC) + tid;
#pragma unroll
            for (int k = 0; k < N; ++k) next[k] = __ldcs(from + k * kLpThreads);
            return;
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int at = (c * (kLpChunk / VEC) + k * kLpThreads + tid) * VEC;  // from base
            if (at >= shift && at + VEC <= end) {
                next[k] = __ldcs(reinterpret_cast<const uint4*>(base + at));
            } else {
                uint32_t w[4] = {};
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    uint32_t raw = BF16 ? 0xFF80u : 0xFF800000u;  // -infinity
                    if (at + j >= shift && at + j < end) {
                        const X v = base[at + j];
                        raw = BF16 ? static_cast<uint32_t>(v) : *reinterpret_cast<const uint32_t*>(&v);
                    }
                    w[BF16 ? j / 2 : j & 3] |= BF16 && (j & 1) ? raw << 16 : raw;
                }
                next[k] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    };
    LpSum s{-INFINITY, 0.f, 0.f};
    int before = 0;
    if (tid < kMaxTop) s_best[tid] = 0ull;
    if (tid == 0) s_n = 0;
    if (c0 < c1) fetch(c0);
    if (p.top > 0) __syncthreads();
    float tau = -INFINITY;  // of the last of s_best: what is larger is a candidate
    int listed = 0;         // candidates at the last meeting
    // the `top` largest of n candidates and of those before (all threads)
    auto choose = [&](int n) {
        if (tid < p.top) s_cand[n + tid] = s_best[tid];
        __syncthreads();
        // four threads a candidate
        for (int j0 = 0; j0 < n + p.top; j0 += kLpThreads / 4) {
            if (j0 + warp * 8 >= n + p.top) break;
            const int j = j0 + (tid >> 2);
            const unsigned long long key = j < n + p.top ? s_cand[j] : 0ull;
            int r = 0;
#pragma unroll 4
            for (int i = tid & 3; i < n + p.top; i += 4) r += s_cand[i] > key ? 1 : 0;
            r += __shfl_xor_sync(0xffffffffu, r, 1);
            r += __shfl_xor_sync(0xffffffffu, r, 2);
            if (key && r < p.top && (tid & 3) == 0) s_best[r] = key;
        }
        if (tid == 0) s_n = 0;
        __syncthreads();
        listed = 0;
        const unsigned long long last = s_best[p.top - 1];
        tau = last ? lp_key_value(last) : -INFINITY;
    };
    int group = c0 + 1;     // first chunk since the last meeting
    int careful = c0 + 1;   // chunks before it get a threshold of their own
    bool again = false;     // of a second reading
    for (int c = c0; c < c1;) {
        float f[kLpEach];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint32_t w[4] = {next[k].x, next[k].y, next[k].z, next[k].w};
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const uint32_t raw = BF16 ? (j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16) : w[j & 3];
                f[k * VEC + j] = __uint_as_float(raw);  // (a NaN loses every comparison below)
            }
        }
        if (c + 1 < c1) fetch(c + 1);
        float mx = f[0];
#pragma unroll
        for (int k = 1; k + 1 < kLpEach; k += 2) mx = max3(mx, f[k], f[k + 1]);
        mx = fmaxf(mx, f[kLpEach - 1]);
        // (the reference follows lazily: exponents of up to kLpLazy cost their rounding alone)
        if (!again && (mx - s.m) * c2 > kLpLazy) s = lp_move(s, mx, c2);
        if (again) {
        } else if (s.m == INFINITY) {
#pragma unroll
            for (int k = 0; k < kLpEach; ++k) s.z += f[k] == INFINITY ? 1.f : 0.f;
        } else {
            const float m = s.m == -INFINITY ? 0.f : s.m;
            float z = 0.f, w = 0.f;
#pragma unroll
            for (int k = 0; k < kLpEach; ++k) {
                const float d = fmaxf((f[k] - m) * c2, -kLpFar), e = ex2(d);
                z += e;
                w = fmaf(e, d, w);
            }
            s.z += z;
            s.w += w;
        }
        auto index = [&](int k) {
            return (c * (kLpChunk / VEC) + (k / VEC) * kLpThreads + tid) * VEC + k % VEC - shift;
        };
        // (a chunk's entries are seldom before a likely token: one look at their maximum)
        if (here && !again && !(mx < xt)) {
            // equal entries count where they stand before the token
            const int at0 = c * kLpChunk - shift;
            float n = 0.f;
            if (c > 0 && at0 + kLpChunk <= t && xt > -INFINITY) {
#pragma unroll
                for (int k = 0; k < kLpEach; ++k) n += f[k] >= xt ? 1.f : 0.f;
                before += static_cast<int>(n);
            } else if (at0 > t && xt > -INFINITY) {
#pragma unroll
                for (int k = 0; k < kLpEach; ++k) n += f[k] > xt ? 1.f : 0.f;
                before += static_cast<int>(n);
            } else {
#pragma unroll
                for (int k = 0; k < kLpEach; ++k) {
                    const float v = fmaxf(f[k], -INFINITY);  // (a NaN reads as -infinity)
                    before += v > xt || (v == xt && index(k) >= 0 && index(k) < t) ? 1 : 0;
                }
            }
        }
        if (p.top == 0) {
            ++c;
            continue;
        }
        // ---- alternatives
        if (c < careful) {
            float least = tau;   // candidates: above tau, and not below this value
            {
                // the ceil(top / 8)-th largest of each warp's maxima
                uint32_t o = mx > -INFINITY ? static_cast<uint32_t>(lp_key(mx, 0) >> 32) : 0u, v = 0u;
                for (int k = 0; k < p.top; k += kLpWarps) {
                    v = __reduce_max_sync(0xffffffffu, o);
                    const unsigned who = __ballot_sync(0xffffffffu, o == v);
                    if (lane == __ffs(who) - 1) o = 0u;
                }
                if (lane == 0) s_first[warp] = v;
                __syncthreads();
#pragma unroll
                for (int k = 0; k < kLpWarps; ++k) v = min(v, s_first[k]);
                if (v) least = lp_key_value(static_cast<unsigned long long>(v) << 32);
            }
            unsigned long long thr = s_best[p.top - 1];
            int mine = 0, at = 0;
            if (mx > tau && mx >= least) {
#pragma unroll
                for (int k = 0; k < kLpEach; ++k) mine += f[k] > tau && f[k] >= least ? 1 : 0;
                at = atomicAdd(&s_n, mine);
            }
            __syncthreads();
            if (s_n > kCand) {
                unsigned long long best = 0;
#pragma unroll
                for (int k = 0; k < kLpEach; ++k)
                    if (f[k] > -INFINITY) best = max(best, lp_key(f[k], index(k)));
                // (threads without entries: keys of their own below every entry's)
                if (best == 0) best = static_cast<unsigned long long>(tid);
                s_max[tid] = best;
                __syncthreads();
                if (lp_above(s_max, kLpThreads, best) == p.top - 1) s_tau = best;
                if (tid == 0) s_n = 0;
                __syncthreads();
                thr = max(thr, s_tau - 1);  // (that entry itself is a candidate)
                least = -INFINITY;
                mine = 0;
#pragma unroll
                for (int k = 0; k < kLpEach; ++k)
                    mine += f[k] > -INFINITY && lp_key(f[k], index(k)) > thr ? 1 : 0;
                at = mine ? atomicAdd(&s_n, mine) : 0;
            }
            if (mine) {
#pragma unroll
                for (int k = 0; k < kLpEach; ++k)
                    if (f[k] > -INFINITY && f[k] >= least && lp_key(f[k], index(k)) > thr)
                        s_cand[at++] = lp_key(f[k], index(k));
            }
            __syncthreads();
            choose(s_n);
            if (++c == careful) {
                again = false;
                group = c;
            }
            continue;
        }
        if (mx > tau) {
            // (one of a thread's entries, as a rule)
#pragma unroll
            for (int k = 0; k < kLpEach; ++k) {
                if (f[k] > tau) {
                    const int at = atomicAdd(&s_n, 1);
                    if (at < kCand) s_cand[at] = lp_key(f[k], index(k));
                }
            }
        }
        if (++c < c1 && c - group < min(kLpGroup, 2 * (group - c0))) continue;
        // ---- the threads meet
        __syncthreads();
        const int now = s_n;
        if (now > kCand) {
            // more than the list holds: without this group's, which is read again
            choose(listed);
            careful = c;
            again = true;
            c = group;
            fetch(c);
        } else {
            if (now >= kCandFull || c == c1) {
                choose(now);
            } else {
                listed = now;
                __syncthreads();  // (all have read s_n)
            }
            group = c;
        }
    }

    // ---- the block's threads
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const LpSum q{__shfl_xor_sync(0xffffffffu, s.m, o), __shfl_xor_sync(0xffffffffu, s.z, o),
                      __shfl_xor_sync(0xffffffffu, s.w, o)};
        s = lp_add(s, q, c2);
        before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    if (lane == 0) {
        s_sum[warp] = s;
        s_before[warp] = before;
    }
    __syncthreads();
    s = s_sum[0];
    before = s_before[0];
#pragma unroll
    for (int k = 1; k < kLpThreads / 32; ++k) {
        s = lp_add(s, s_sum[k], c2);
        before += s_before[k];
    }
    const long long slot = row * split + part;
    if (tid == 0) {
        if (split > 1) parts[slot] = LpPart{s.m, s.z, s.w, before};
        else lp_write(p, row, s, before, t, xt);
    }
    if (tid < p.top) {
        if (split > 1) lists[slot * p.top + tid] = s_best[tid];
        else lp_write_top(p, row, tid, s_best[tid], s.m, logf(s.z));
    }
}

// Joins the parts of a row, a block a row.
template <bool BF16>
__global__ void __launch_bounds__(kLpThreads) logprob_join_kernel(const LogprobParams p,
                                                                  const LpPart* parts,
                                                                  const unsigned long long* lists,
                                                                  int split) {
    using X = std::conditional_t<BF16, uint16_t, float>;
    __shared__ unsigned long long s_head[kLpMaxSplit], s_cand[kMaxTop * kMaxTop], s_tau;
    __shared__ LpPart s_part[kLpMaxSplit];
    __shared__ int s_n;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x;
    const long long row = blockIdx.x;
    if (p.len && static_cast<int>(row % p.R) >= __ldg(p.len + row / p.R)) return;
    const int t = p.tokens ? __ldg(p.tokens + row) : -1;
    float xt = INFINITY;
    if (tid == 0 && t >= 0 && t < p.V) {
        const X raw = static_cast<const X*>(p.x)[row * p.ldx + t];
        xt = fmaxf(BF16 ? __uint_as_float(static_cast<uint32_t>(raw) << 16)
                        : *reinterpret_cast<const float*>(&raw), -INFINITY);
    }
    constexpr int kKeys = kLpMaxSplit * kMaxTop / kLpThreads;  // of a thread
    unsigned long long key[kKeys];  // on their way before the heads say which count
#pragma unroll
    for (int q = 0; q < kKeys; ++q) {
        const int j = tid + q * kLpThreads;
        key[q] = j < split * p.top ? __ldcg(lists + row * split * p.top + j) : 0ull;
    }
    if (tid < split) {
        s_part[tid] = parts[row * split + tid];
        s_head[tid] = p.top ? __ldcg(lists + (row * split + tid) * p.top) : 0ull;
    }
    if (tid == 0) s_n = 0, s_tau = 0ull;
    __syncthreads();
    // every warp sums the parts, two a lane
    const float c2 = p.scale * kLog2e;
    const int lane = tid & 31;
    auto part = [&](int k) {
        return k < split ? LpSum{s_part[k].m, s_part[k].z, s_part[k].w} : LpSum{-INFINITY, 0.f, 0.f};
    };
    static_assert(kLpMaxSplit == 64, "two parts a lane");
    LpSum s = lp_add(part(lane), part(lane + 32), c2);
    int before = (lane < split ? s_part[lane].before : 0) + (lane + 32 < split ? s_part[lane + 32].before : 0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s = lp_add(s, LpSum{__shfl_xor_sync(0xffffffffu, s.m, o), __shfl_xor_sync(0xffffffffu, s.z, o),
                            __shfl_xor_sync(0xffffffffu, s.w, o)}, c2);
        before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    if (tid == 0) lp_write(p, row, s, before, t, xt);
    if (p.top == 0) return;
    // of the `top` largest heads the least: the row's `top` largest are not below it, and lie
    // in those lists (with fewer parts: in any)
    if (tid < split && s_head[tid] && lp_above(s_head, split, s_head[tid]) == p.top - 1)
        s_tau = s_head[tid];
    __syncthreads();
    const unsigned long long tau = s_tau;
#pragma unroll
    for (int q = 0; q < kKeys; ++q)
        if (key[q] != 0ull && key[q] >= tau) s_cand[atomicAdd(&s_n, 1)] = key[q];
    __syncthreads();
    const int n = s_n;
    const float lnz = logf(s.z);
    for (int j0 = 0; j0 < n; j0 += kLpThreads / 4) {  // four threads a candidate
        const int j = j0 + (tid >> 2);
        const unsigned long long mine = j < n ? s_cand[j] : 0ull;
        int r = 0;
#pragma unroll 4
        for (int i = tid & 3; i < n; i += 4) r += s_cand[i] > mine ? 1 : 0;
        r += __shfl_xor_sync(0xffffffffu, r, 1);
        r += __shfl_xor_sync(0xffffffffu, r, 2);
        if (mine && r < p.top && (tid & 3) == 0) lp_write_top(p, row, r, mine, s.m, lnz);
    }
    if (tid >= n && tid < p.top) lp_write_top(p, row, tid, 0ull, s.m, lnz);
}

cudaError_t launch_logprobs(const LogprobParams& p, void* ws, int sms, cudaStream_t s) {
    (void)sms;
    const long long rows = static_cast<long long>(p.B) * p.R;
    const int split = lp_split(rows, p.V);
    LpPart* parts = static_cast<LpPart*>(ws);
    unsigned long long* lists = reinterpret_cast<unsigned long long*>(parts + rows * split);
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kLpThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(rows * split));
    cudaError_t e = cudaLaunchKernelEx(&cfg, p.x_bf16 ? logprob_kernel<true> : logprob_kernel<false>,
                                       p, parts, lists, split);
    if (e != cudaSuccess || split == 1) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(rows));
    return cudaLaunchKernelEx(&cfg, p.x_bf16 ? logprob_join_kernel<true> : logprob_join_kernel<false>,
                              p, static_cast<const LpPart*>(parts),
                              static_cast<const unsigned long long*>(lists), split);
}

}  // namespace vw4
