// advance.cu -- lengths, pages, block table and slots of the next step's rows, from the
// lengths that an accept left on the device.
//
// Three phases: scans over the sequences (what each gives back, needs and gets: prefix sums
// in the sequences' order make the outcome independent of the schedule); the returned pages
// onto the free list; the taken pages into the table and the rows' slots.  The second needs
// little of the first and runs beside it, in blocks that sum up the returned pages by
// themselves (as a launch of its own 28 us instead of 22 for 4096 sequences); the
// third looks its sequence up in the prefix sums, so that one long prompt is spread over the
// whole grid.
//
// Everything here is a chain of load latencies: the scan keeps its sequences in registers
// from one load, a warp finds its sequence with 32 probes at a time (three steps for 16384
// sequences instead of fourteen), and takes few entries.  Small calls (table and slots of
// at most kOneBlock* entries) are one block's work and one launch: 16 sequences of 8 rows 6.3 us
// instead of 7.1; one prompt of 2000 rows among them is 8.5 so, 7.0 in two, 256 sequences of 8
// with new ones 20.1 and 15.1.  A call without slots goes by its table alone: 2048 sequences of 32
// columns are 12.9 us in one block and 14.4 in two launches where no page moves, 21.4 and 13.7
// where an eighth of them ends and an eighth is new; which of them it is only the device knows.
#include "vw4_internal.cuh"

namespace vw4 {

constexpr int kAdvThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kWarpSlots = 64;           // consecutive entries that a warp takes at a time
constexpr long long kOneBlockTable = 65536, kOneBlockSlots = 512;

struct AdvancePlan {
    long long* back;   // [B + 1] pages given back before each sequence
    long long* take;   // [B + 1] pages taken before each sequence
    long long* count;  // [0] pages of the free list before, [1] with the returned ones
    // the outputs that may be inputs: themselves, or a copy until all have read the inputs
    int32_t* lens;
    int32_t* held;
    int32_t* free_count;
};

static AdvancePlan plan_of(const AdvanceParams& p, void* ws, bool direct) {
    const int B = p.B;
    AdvancePlan w;
    w.back = static_cast<long long*>(ws);
    w.take = w.back + (B + 2) / 2 * 2;  // (16-byte boundaries)
    w.count = w.take + (B + 2) / 2 * 2;
    int32_t* copies = reinterpret_cast<int32_t*>(w.count + 2);
    w.lens = direct ? p.lens_out : copies;
    w.held = direct ? p.held_out : copies + (B + 3) / 4 * 4;
    w.free_count = direct ? p.free_count_out : copies + 2 * ((B + 3) / 4 * 4);
    return w;
}
size_t advance_workspace_bytes(int B) {
    return ((2 * (static_cast<size_t>(B) + 2) + 2) * sizeof(long long) +
            (2 * (static_cast<size_t>(B) + 3) + 4) * sizeof(int32_t) + 255) & ~size_t(255);
}

// What a call finds of one sequence.  Lengths saturate at 2^31 - 1: beyond every table.
struct AdvSeq {
    int len, grow, need;   // need: -1 where the table is too short
    int held, back;        // pages kept, pages given back
};
__device__ __forceinline__ AdvSeq adv_seq(const AdvanceParams& p, bool ended, int held, int accepted,
                                          int lens, int grow) {
    AdvSeq s;
    held = max(0, min(p.max_blocks, held));
    const long long len = ended ? 0 : static_cast<long long>(max(0, lens)) + max(0, accepted);
    s.len = static_cast<int>(min(len, 2147483647LL));
    s.held = ended ? 0 : held;
    s.back = ended ? held : 0;
    s.grow = max(0, grow);
    const long long cols = (len + s.grow + p.page_size - 1) >> p.page_shift;
    s.need = cols > p.max_blocks ? -1 : max(0, static_cast<int>(cols) - s.held);
    return s;
}

// Exclusive prefix sums of two numbers over the block's threads, and their totals.
struct Pair {
    long long a, b;
};
__device__ __forceinline__ Pair block_scan(Pair v, Pair* total, Pair* s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Pair in = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, in.a, o), b = __shfl_up_sync(0xffffffffu, in.b, o);
        if (lane >= o) in.a += a, in.b += b;
    }
    __syncthreads();  // (s_warp was read)
    if (lane == 31) s_warp[warp] = in;
    __syncthreads();
    Pair w = s_warp[lane];  // kAdvThreads / 32 == 32 of them
    const Pair mine = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, w.a, o), b = __shfl_up_sync(0xffffffffu, w.b, o);
        if (lane >= o) w.a += a, w.b += b;
    }
    total->a = __shfl_sync(0xffffffffu, w.a, 31);
    total->b = __shfl_sync(0xffffffffu, w.b, 31);
    const long long ba = __shfl_sync(0xffffffffu, w.a - mine.a, warp);
    const long long bb = __shfl_sync(0xffffffffu, w.b - mine.b, warp);
    return Pair{in.a - v.a + ba, in.b - v.b + bb};
}

// N entries from b on of an array of n, four at a time where the arrays allow it (one at a
// time each of a warp's stores writes parts of 16 sectors: a call on 4096 sequences took 31.3 us
// instead of 27.8, then).
template <int N>
__device__ __forceinline__ void adv_load(int (&v)[N], const int32_t* a, int b, int n, bool vec, int none) {
    if (N % 4 == 0 && vec && b + N <= n) {
#pragma unroll
        for (int k = 0; k < N / 4; ++k) {
            const int4 x = a ? reinterpret_cast<const int4*>(a + b)[k] : make_int4(none, none, none, none);
            v[4 * k] = x.x, v[4 * k + 1] = x.y, v[4 * k + 2] = x.z, v[4 * k + 3] = x.w;
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = a && b + k < n ? a[b + k] : none;
}
template <int N>
__device__ __forceinline__ void adv_store(int32_t* a, const int (&v)[N], int b, int n, bool vec) {
    if (N % 4 == 0 && vec && b + N <= n) {
#pragma unroll
        for (int k = 0; k < N / 4; ++k)
            reinterpret_cast<int4*>(a + b)[k] = make_int4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        return;
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (b + k < n) a[b + k] = v[k];
}
template <int N>
__device__ __forceinline__ void adv_store(long long* a, const long long (&v)[N], int b, int n) {
    if (N % 2 == 0 && b + N <= n) {
#pragma unroll
        for (int k = 0; k < N / 2; ++k)
            reinterpret_cast<longlong2*>(a + b)[k] = make_longlong2(v[2 * k], v[2 * k + 1]);
        return;
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (b + k < n) a[b + k] = v[k];
}

// Phase 1, by one block of kAdvThreads, G groups of N sequences a thread.  More than one group
// is read again for each of the two scans and for the outputs.
template <int N, int G>
__device__ __forceinline__ void scan_phase(const AdvanceParams& p, const AdvancePlan& w) {
    static_assert(kAdvThreads == 1024, "32 warps");
    __shared__ Pair s_warp[32];
    const int b0 = threadIdx.x * (N * G);
    const long long stock = max(0, min(p.num_pages, p.free_count[0]));
    const bool vec = ((reinterpret_cast<uintptr_t>(p.ended) | reinterpret_cast<uintptr_t>(p.held) |
                       reinterpret_cast<uintptr_t>(p.accepted) | reinterpret_cast<uintptr_t>(p.lens) |
                       reinterpret_cast<uintptr_t>(p.grow) | reinterpret_cast<uintptr_t>(p.row_start) |
                       reinterpret_cast<uintptr_t>(w.lens) | reinterpret_cast<uintptr_t>(w.held) |
                       reinterpret_cast<uintptr_t>(p.seq_lens)) & 15u) == 0;
    AdvSeq s[N];
    auto group = [&](int g) {
        const int b = b0 + g * N;
        int ended[N], held[N], accepted[N], lens[N], grow[N];
        adv_load(ended, p.ended, b, p.B, vec, 0);
        adv_load(held, p.held, b, p.B, vec, 0);
        adv_load(accepted, p.accepted, b, p.B, vec, 0);
        adv_load(lens, p.lens, b, p.B, vec, 0);
        adv_load(grow, p.grow, b, p.B, vec, p.R);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            s[k] = AdvSeq{0, 0, 0, 0, 0};
            if (b + k < p.B) s[k] = adv_seq(p, ended[k] != 0, held[k], accepted[k], lens[k], grow[k]);
        }
    };
    bool short_of = false;
    Pair sum{0, 0}, total;
#pragma unroll 1
    for (int g = 0; g < G; ++g) {
        group(g);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            sum.a += s[k].back;
            sum.b += max(0, s[k].need);
        }
    }
    Pair at = block_scan(sum, &total, s_warp);
    const long long count = min(static_cast<long long>(p.num_pages), stock + total.a);
    if (stock + total.a > p.num_pages) short_of = true;
    // who gets what: ok[k], and what that adds up to
    uint32_t ok = 0;
    long long need = at.b;
    sum = Pair{0, 0};
#pragma unroll 1
    for (int g = 0; g < G; ++g) {
        if (G > 1) group(g);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (s[k].need == 0 || (s[k].need > 0 && need + s[k].need <= count)) {
                ok |= 1u << (g * N + k);
                sum.a += s[k].need;
                sum.b += s[k].grow;
            }
            need += max(0, s[k].need);
        }
    }
    const long long back_all = total.a;
    // (every input of a sequence has been read before its outputs, which may be the inputs: they
    // are the same thread's)
    Pair got = block_scan(sum, &total, s_warp);
#pragma unroll 1
    for (int g = 0; g < G; ++g) {
        if (G > 1) group(g);
        const int b = b0 + g * N;
        long long back[N], take[N];
        int start[N], lens[N], held[N], seq_lens[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const bool mine = (ok >> (g * N + k)) & 1u;
            back[k] = at.a;
            take[k] = got.a;
            start[k] = static_cast<int>(min(got.b, 2147483647LL));
            at.a += s[k].back;
            if (mine) {
                got.a += s[k].need;
                got.b += s[k].grow;
            } else if (b + k < p.B) {
                short_of = true;
            }
            lens[k] = s[k].len;
            held[k] = s[k].held + (mine ? s[k].need : 0);
            seq_lens[k] = mine && s[k].grow > 0 ? s[k].len + s[k].grow : 0;
        }
        adv_store(w.back, back, b, p.B);
        adv_store(w.take, take, b, p.B);
        adv_store(p.row_start, start, b, p.B, vec);
        adv_store(w.lens, lens, b, p.B, vec);
        adv_store(w.held, held, b, p.B, vec);
        adv_store(p.seq_lens, seq_lens, b, p.B, vec);
    }
    if (threadIdx.x == 0) {
        w.back[p.B] = back_all;
        w.take[p.B] = total.a;
        w.count[0] = stock;
        w.count[1] = count;
        p.row_start[p.B] = static_cast<int32_t>(min(total.b, 2147483647LL));
        w.free_count[0] = static_cast<int32_t>(count - total.a);
        if (p.slots && total.b > p.rows_max) short_of = true;
    }
    if (short_of) atomicOr(p.status, kStatusNoRoom);
}

// The returned pages onto the free list, by `blocks` blocks of kAdvThreads next to the one that
// scans: each sums up what comes before its sequences by itself, and takes every blocks-th
// eight of them, a warp a sequence.
template <int N, int G>
__device__ __forceinline__ void push_beside(const AdvanceParams& p, int block, int blocks) {
    __shared__ Pair s_warp[32];
    const int b0 = threadIdx.x * (N * G), lane = threadIdx.x & 31;
    const long long stock = max(0, min(p.num_pages, p.free_count[0]));
    const bool vec = ((reinterpret_cast<uintptr_t>(p.ended) | reinterpret_cast<uintptr_t>(p.held)) & 15u) == 0;
    int back[N];
    auto group = [&](int g) {
        int ended[N];
        adv_load(ended, p.ended, b0 + g * N, p.B, vec, 0);
        adv_load(back, p.held, b0 + g * N, p.B, vec, 0);
#pragma unroll
        for (int k = 0; k < N; ++k) back[k] = ended[k] != 0 ? max(0, min(p.max_blocks, back[k])) : 0;
    };
    Pair sum{0, 0}, total;
#pragma unroll 1
    for (int g = 0; g < G; ++g) {
        group(g);
#pragma unroll
        for (int k = 0; k < N; ++k) sum.a += back[k];
    }
    Pair at = block_scan(sum, &total, s_warp);
#pragma unroll 1
    for (int g = 0; g < G; ++g) {
        if (G > 1) group(g);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int b = b0 + g * N + k;
            unsigned who = __ballot_sync(0xffffffffu, back[k] > 0 && (b >> 3) % blocks == block);
            while (who) {
                const int l = __ffs(who) - 1;
                who &= who - 1;
                const int n = __shfl_sync(0xffffffffu, back[k], l), bl = __shfl_sync(0xffffffffu, b, l);
                const long long to = stock + __shfl_sync(0xffffffffu, at.a, l);
                const int32_t* row = p.table + bl * p.table_stride;
                for (int i = lane; i < n; i += 32)
                    if (to + i < p.num_pages) p.free_list[to + i] = row[i];
            }
            at.a += back[k];
        }
    }
}

// The sequence of entry i, the same in all lanes: the last with start[b] <= i.
template <class T>
__device__ __forceinline__ int seq_of(const T* start, int B, long long i) {
    const int lane = threadIdx.x & 31;
    int lo = 0, span = B;  // start[lo] <= i < start[lo + span]
    while (span > 1) {
        const int step = (span + 31) / 32, at = (lane + 1) * step;
        const bool low = at < span && static_cast<long long>(start[lo + at]) <= i;
        const int n = __popc(__ballot_sync(0xffffffffu, low)) * step;
        lo += n;
        span = min(step, span - n);
    }
    return lo;
}

// f(b, i) for every entry i < n of the sequences' consecutive entries, the warps of the grid
// taking kWarpSlots at a time.
template <class T, class F>
__device__ __forceinline__ void each_entry(const T* start, int B, long long n, long long warp,
                                           long long warps, F f) {
    const int lane = threadIdx.x & 31;
    for (long long c = warp * kWarpSlots; c < n; c += warps * kWarpSlots) {
        int b = seq_of(start, B, c);
        for (long long i = c + lane; i < min(n, c + kWarpSlots); i += 32) {
            while (static_cast<long long>(start[b + 1]) <= i) ++b;
            f(b, i);
        }
    }
}

__device__ __forceinline__ void push_phase(const AdvanceParams& p, const AdvancePlan& w,
                                           long long warp, long long warps) {
    const long long stock = w.count[0];
    each_entry(w.back, p.B, w.back[p.B], warp, warps, [&](int b, long long i) {
        if (stock + i < p.num_pages)
            p.free_list[stock + i] = p.table[b * p.table_stride + (i - w.back[b])];
    });
}

// columns of sequence b that held pages before
__device__ __forceinline__ int adv_kept(const AdvanceParams& p, const AdvancePlan& w, int b) {
    return w.held[b] - static_cast<int>(w.take[b + 1] - w.take[b]);
}
__device__ __forceinline__ void take_phase(const AdvanceParams& p, const AdvancePlan& w,
                                           long long warp, long long warps) {
    const long long top = w.count[1] - 1;
    each_entry(w.take, p.B, w.take[p.B], warp, warps, [&](int b, long long i) {
        p.table[b * p.table_stride + adv_kept(p, w, b) + (i - w.take[b])] = p.free_list[top - i];
    });
}
// (reads no table column that take_phase writes)
__device__ __forceinline__ void slot_phase(const AdvanceParams& p, const AdvancePlan& w,
                                           long long warp, long long warps) {
    if (!p.slots) return;
    const long long top = w.count[1] - 1;
    const long long rows = min(static_cast<long long>(p.row_start[p.B]), p.rows_max);
    bool bad = false;
    each_entry(p.row_start, p.B, rows, warp, warps, [&](int b, long long i) {
        const long long pos = w.lens[b] + (i - p.row_start[b]);
        const int col = static_cast<int>(pos >> p.page_shift), k = adv_kept(p, w, b);
        const int page = col < k ? p.table[b * p.table_stride + col]
                                 : p.free_list[top - (w.take[b] + col - k)];
        const bool ok = page >= 0 && page < p.num_pages;
        bad |= !ok;
        p.slots[i] = ok ? (static_cast<long long>(page) << p.page_shift) + (pos & (p.page_size - 1)) : -1;
    });
    if (bad) atomicOr(p.status, kStatusBadPage);
}

template <int N, int G>
__global__ void __launch_bounds__(kAdvThreads) advance_kernel(const AdvanceParams p,
                                                              const AdvancePlan w, int all) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x > 0) return push_beside<N, G>(p, blockIdx.x - 1, gridDim.x - 1);
    scan_phase<N, G>(p, w);
    if (!all) return;
    __syncthreads();
    const long long warp = threadIdx.x >> 5;
    push_phase(p, w, warp, kAdvThreads / 32);
    __syncthreads();
    take_phase(p, w, warp, kAdvThreads / 32);
    slot_phase(p, w, warp, kAdvThreads / 32);
}

// The first `takers` blocks fill the table and leave the outputs that may be inputs, the others
// fill the slots.
__global__ void __launch_bounds__(kFillThreads) advance_fill_kernel(const AdvanceParams p,
                                                                    const AdvancePlan w, int takers) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int blocks = static_cast<int>(gridDim.x), block = static_cast<int>(blockIdx.x);
    const int in = threadIdx.x >> 5;
    constexpr int W = kFillThreads / 32;
    if (block >= takers) return slot_phase(p, w, (block - takers) * W + in, (blocks - takers) * W);
    for (int i = block * kFillThreads + threadIdx.x; i < p.B; i += takers * kFillThreads) {
        p.lens_out[i] = w.lens[i];
        p.held_out[i] = w.held[i];
    }
    if (block == 0 && threadIdx.x == 0) p.free_count_out[0] = w.free_count[0];
    take_phase(p, w, block * W + in, takers * W);
}

cudaError_t launch_advance(const AdvanceParams& p, void* ws, int sms, cudaStream_t s) {
    const long long rows = p.slots ? p.rows_max : 0;
    const int all = static_cast<long long>(p.B) * p.max_blocks <= kOneBlockTable && rows <= kOneBlockSlots;
    const AdvancePlan w = plan_of(p, ws, all);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(all || !p.ended ? 1 : sms);
    cfg.blockDim = dim3(kAdvThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = p.B <= kAdvThreads       ? cudaLaunchKernelEx(&cfg, advance_kernel<1, 1>, p, w, all)
                    : p.B <= 4 * kAdvThreads ? cudaLaunchKernelEx(&cfg, advance_kernel<4, 1>, p, w, all)
                                             : cudaLaunchKernelEx(&cfg, advance_kernel<4, 4>, p, w, all);
    if (e != cudaSuccess || all) return e;
    cfg.blockDim = dim3(kFillThreads);
    // a block takes 512 slots at a time; how many pages move only the device knows
    const long long blocks = (rows + 511) / 512;
    cfg.gridDim = dim3(static_cast<unsigned>(sms + (blocks < 6LL * sms ? blocks : 6LL * sms)));
    return cudaLaunchKernelEx(&cfg, advance_fill_kernel, p, w, sms);
}

}  // namespace vw4
