// advance.cu -- lengths, pages, block table and slots of the next step's rows, from the
// lengths that an accept left on the device.
//
// Three phases, each over what the one before has written: scans over the sequences (what
// each gives back, needs and gets: prefix sums in the sequences' order make the outcome
// independent of the schedule); the returned pages onto the free list; the taken pages
// into the table and the rows' slots.  The second and the third look their sequence up in
// the prefix sums, so that one long prompt is spread over the whole grid.
//
// Small calls (table and slots of at most kOneBlock* entries) are one block's work and one
// launch: a chain of latencies, as the scans of the others are.  The slots bound large ones.
#include "vw4_internal.cuh"

namespace vw4 {

constexpr int kAdvThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kWarpSlots = 256;          // consecutive entries that a warp takes at a time
constexpr long long kOneBlockTable = 65536, kOneBlockSlots = 8192;

struct AdvancePlan {
    long long* back;   // [B + 1] pages given back before each sequence
    long long* take;   // [B + 1] pages taken before each sequence
    long long* count;  // [0] pages of the free list before, [1] with the returned ones
};

static AdvancePlan plan_of(void* ws, int B) {
    AdvancePlan w;
    w.back = static_cast<long long*>(ws);
    w.take = w.back + B + 1;
    w.count = w.take + B + 1;
    return w;
}
size_t advance_workspace_bytes(int B) {
    return ((2 * (static_cast<size_t>(B) + 1) + 2) * sizeof(long long) + 255) & ~size_t(255);
}

// What a call gives of one sequence.
struct AdvSeq {
    long long len, grow, need;  // need: -1 where the table is too short
    int held, back;             // pages kept, pages given back
};
__device__ __forceinline__ AdvSeq adv_seq(const AdvanceParams& p, int b) {
    AdvSeq s;
    const bool ended = p.ended && p.ended[b] != 0;
    const int held = max(0, min(p.max_blocks, p.held[b]));
    const long long acc = p.accepted ? max(0, p.accepted[b]) : 0;
    s.len = ended ? 0 : max(0, p.lens[b]) + acc;
    s.held = ended ? 0 : held;
    s.back = ended ? held : 0;
    s.grow = p.grow ? max(0, p.grow[b]) : p.R;
    const long long cols = (s.len + s.grow + p.page_size - 1) >> p.page_shift;
    s.need = cols > p.max_blocks ? -1 : max(0LL, cols - s.held);
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

// Phase 1, by one block of kAdvThreads.
__device__ void scan_phase(const AdvanceParams& p, const AdvancePlan& w) {
    static_assert(kAdvThreads == 1024, "32 warps");
    __shared__ Pair s_warp[32];
    const int per = (p.B + kAdvThreads - 1) / kAdvThreads, b0 = threadIdx.x * per;
    const int b1 = min(p.B, b0 + per);
    const long long stock = max(0, min(p.num_pages, p.free_count[0]));
    bool short_of = false;
    Pair sum{0, 0}, total;
    for (int b = b0; b < b1; ++b) {
        const AdvSeq s = adv_seq(p, b);
        sum.a += s.back;
        sum.b += max(0LL, s.need);
    }
    Pair at = block_scan(sum, &total, s_warp);
    const long long count = min(static_cast<long long>(p.num_pages), stock + total.a);
    if (stock + total.a > p.num_pages) short_of = true;
    // who gets what
    const Pair first = at;
    sum = Pair{0, 0};
    for (int b = b0; b < b1; ++b) {
        const AdvSeq s = adv_seq(p, b);
        const bool ok = s.need >= 0 && (s.need == 0 || at.b + s.need <= count);
        at.b += max(0LL, s.need);
        if (ok) {
            sum.a += s.need;
            sum.b += s.grow;
        }
    }
    Pair got = block_scan(sum, &total, s_warp);
    at = first;
    for (int b = b0; b < b1; ++b) {
        const AdvSeq s = adv_seq(p, b);  // (before any output, which may be an input)
        const bool ok = s.need >= 0 && (s.need == 0 || at.b + s.need <= count);
        w.back[b] = at.a;
        w.take[b] = got.a;
        p.row_start[b] = static_cast<int32_t>(min(got.b, 2147483647LL));
        at.a += s.back;
        at.b += max(0LL, s.need);
        if (ok) {
            got.a += s.need;
            got.b += s.grow;
        } else {
            short_of = true;
        }
        p.lens_out[b] = static_cast<int32_t>(min(s.len, 2147483647LL));
        p.held_out[b] = s.held + static_cast<int>(ok ? s.need : 0);
        p.seq_lens[b] = ok && s.grow > 0 ? static_cast<int32_t>(s.len + s.grow) : 0;
    }
    if (threadIdx.x == kAdvThreads - 1) {  // (its sums end with the last sequence)
        w.back[p.B] = at.a;
        w.take[p.B] = total.a;
        w.count[0] = stock;
        w.count[1] = count;
        p.row_start[p.B] = static_cast<int32_t>(min(total.b, 2147483647LL));
        p.free_count_out[0] = static_cast<int32_t>(count - total.a);
        if (p.slots && total.b > p.rows_max) short_of = true;
    }
    if (short_of) atomicOr(p.status, kStatusNoRoom);
}

// The sequence of entry i: the last with start[b] <= i.
template <class T>
__device__ __forceinline__ int seq_of(const T* start, int B, long long i) {
    int lo = 0, hi = B;  // start[lo] <= i < start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (static_cast<long long>(start[mid]) <= i) lo = mid;
        else hi = mid;
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

__device__ __forceinline__ void fill_phase(const AdvanceParams& p, const AdvancePlan& w,
                                           long long warp, long long warps) {
    const long long top = w.count[1] - 1;
    auto kept = [&](int b) {  // columns that held pages before
        return p.held_out[b] - static_cast<int>(w.take[b + 1] - w.take[b]);
    };
    each_entry(w.take, p.B, w.take[p.B], warp, warps, [&](int b, long long i) {
        p.table[b * p.table_stride + kept(b) + (i - w.take[b])] = p.free_list[top - i];
    });
    if (!p.slots) return;
    const long long rows = min(static_cast<long long>(p.row_start[p.B]), p.rows_max);
    bool bad = false;
    each_entry(p.row_start, p.B, rows, warp, warps, [&](int b, long long i) {
        const long long pos = p.lens_out[b] + (i - p.row_start[b]);
        const int col = static_cast<int>(pos >> p.page_shift), k = kept(b);
        const int page = col < k ? p.table[b * p.table_stride + col]
                                 : p.free_list[top - (w.take[b] + col - k)];
        const bool ok = page >= 0 && page < p.num_pages;
        bad |= !ok;
        p.slots[i] = ok ? (static_cast<long long>(page) << p.page_shift) + (pos & (p.page_size - 1)) : -1;
    });
    if (bad) atomicOr(p.status, kStatusBadPage);
}

__global__ void __launch_bounds__(kAdvThreads) advance_kernel(const AdvanceParams p,
                                                              const AdvancePlan w, int all) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    scan_phase(p, w);
    if (!all) return;
    __syncthreads();
    const long long warp = threadIdx.x >> 5;
    push_phase(p, w, warp, kAdvThreads / 32);
    __syncthreads();
    fill_phase(p, w, warp, kAdvThreads / 32);
}

template <bool FILL>
__global__ void __launch_bounds__(kFillThreads) advance_fill_kernel(const AdvanceParams p,
                                                                    const AdvancePlan w) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long warps = static_cast<long long>(gridDim.x) * (kFillThreads / 32);
    const long long warp = static_cast<long long>(blockIdx.x) * (kFillThreads / 32) + (threadIdx.x >> 5);
    if (FILL) fill_phase(p, w, warp, warps);
    else push_phase(p, w, warp, warps);
}

cudaError_t launch_advance(const AdvanceParams& p, void* ws, int sms, cudaStream_t s) {
    const AdvancePlan w = plan_of(ws, p.B);
    const long long rows = p.slots ? p.rows_max : 0;
    const int all = static_cast<long long>(p.B) * p.max_blocks <= kOneBlockTable && rows <= kOneBlockSlots;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kAdvThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, advance_kernel, p, w, all);
    if (e != cudaSuccess || all) return e;
    cfg.gridDim = dim3(4 * sms);
    cfg.blockDim = dim3(kFillThreads);
    if (p.ended) {
        e = cudaLaunchKernelEx(&cfg, advance_fill_kernel<false>, p, w);
        if (e != cudaSuccess) return e;
    }
    return cudaLaunchKernelEx(&cfg, advance_fill_kernel<true>, p, w);
}

}  // namespace vw4
