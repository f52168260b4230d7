// logits.cu -- the sampler's first stage on the verify logits: penalties for
// repeated tokens, sparse biases and grammar masks, with the block maxima that
// the sampled accept reads.
//
//   known(v) = v among prompt, output and the row's earlier drafts;
//   c(v)     = its count among output and the row's earlier drafts
//   y = known ? (x > 0 ? x / r : x r) : x;   y -= f c + q [c > 0];   y += bias
//   out = allowed ? y : -infinity
//
// One pass over the logits: a block owns a chunk of the vocabulary of one
// sequence and keeps its counts in shared memory, so the rows of a verify
// batch share one scan of the token history; the few drafts before a row are
// compared only at the entries that one of them names.  So the rows need no barrier
// between them.  The bytes bound it (8 a logit; masked logits are not read): 256 x 9
// rows of 151936 take 438 us, 97 % of the copy rate; 64 x 5 rows with 70 % of the ids
// masked away 69 us, 1.7 times its bytes (loads wait).  The scan re-reads the history
// once per chunk, from L2.  A small call is the scan's latency: 8 rows of 262144 with 2048
// ids of history 7.7 us.
#include "attn.cuh"

namespace vw4 {

constexpr int kLogitThreads = 256;
constexpr uint32_t kKnown = 0x80000000u;        // count word: in the prompt
constexpr uint32_t kDrafted = 0x40000000u;      // count word: a draft of the sequence
constexpr uint32_t kLogitBadDraft = 0x1u;

// VEC consecutive logits a thread and step, kLogitChunk vocabulary entries a block.  The
// first row's logits are on their way while the history is scanned; a later row's are
// asked for all at once when the row before has been written, by then with the mask words
// at hand that decide which of them are read.
template <int VEC, int kLogitChunk>
__global__ void __launch_bounds__(kLogitThreads, VEC == 4 ? 4 : 3)
    logits_kernel(const LogitsParams p, int row_step) {
    constexpr int N = kLogitChunk / (kLogitThreads * VEC);  // steps of a row
    __shared__ __align__(16) uint32_t s_cnt[kLogitChunk];
    __shared__ __align__(16) uint32_t s_bias[kLogitChunk];  // bias entry + 1 (0: none)
    __shared__ uint32_t s_hit[kLogitChunk / 32];            // entries with a count, a draft or a bias
    __shared__ int s_draft[kMaxVerifyRows];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, b = blockIdx.y;
    const int c0 = blockIdx.x * kLogitChunk;
    const int row0 = blockIdx.z * row_step, row1 = min(p.R, row0 + row_step);
    for (int k = tid; k < kLogitChunk / 4; k += kLogitThreads) {
        reinterpret_cast<uint4*>(s_cnt)[k] = make_uint4(0, 0, 0, 0);
        if (p.bias_ids) reinterpret_cast<uint4*>(s_bias)[k] = make_uint4(0, 0, 0, 0);
    }
    for (int k = tid; k < kLogitChunk / 32; k += kLogitThreads) s_hit[k] = 0u;
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // everything small that is needed later, asked for at once: a short call is a chain
    // of load latencies
    const int n_hist = p.history ? (p.hist_len ? max(0, min(p.hist_max, __ldg(p.hist_len + b))) : p.hist_max) : 0;
    const int n_prompt = p.prompt_len ? __ldg(p.prompt_len + b) : 0;
    const int n_bias = p.bias_ids ? (p.bias_len ? max(0, min(p.bias_max, __ldg(p.bias_len + b))) : p.bias_max) : 0;
    const int draft = tid < p.R - 1 ? __ldg(p.drafts + static_cast<long long>(b) * (p.R - 1) + tid) : -1;
    const float rep = p.repetition ? __ldg(p.repetition + b) : 1.f;
    const float pre = p.presence ? __ldg(p.presence + b) : 0.f;
    const float fre = p.frequency ? __ldg(p.frequency + b) : 0.f;
    const int32_t* bias_ids = p.bias_ids ? p.bias_ids + static_cast<long long>(b) * p.bias_stride : nullptr;
    const int bias_id = tid < p.bias_max ? __ldg(bias_ids + tid) : -1;
    // the first ids of the history, whether or not its length reaches them
    const int32_t* ids = p.history ? p.history + static_cast<long long>(b) * p.hist_stride : nullptr;
    const int head = static_cast<int>((16u - (reinterpret_cast<uintptr_t>(ids) & 15u)) & 15u) / 4;
    const int4 id4 = head + 4 * tid + 3 < p.hist_max
                         ? __ldg(reinterpret_cast<const int4*>(ids + head) + tid)
                         : make_int4(-1, -1, -1, -1);
    constexpr uint32_t kFull = VEC == 4 ? 0xfu : 1u;
    auto place = [&](int k) { return c0 + (k * kLogitThreads + tid) * VEC; };
    // mask words of a row (all ones without a mask)
    uint32_t words[N];
    auto masks = [&](int i) {
        const long long row = static_cast<long long>(b) * p.R + i;
        const uint32_t* mk = nullptr;
        if (p.mask) {
            const long long mr = p.mask_index ? p.mask_index[row] : row;
            if (mr >= 0 && mr < p.mask_rows) mk = p.mask + mr * p.mask_stride;
        }
#pragma unroll
        for (int k = 0; k < N; ++k)
            words[k] = mk && place(k) < p.V ? __ldg(mk + (place(k) >> 5)) : ~0u;
    };
    // a row's allowed logits (the masked ones are not read); step k's bits of `allow`
    float x[N][VEC];
    uint32_t allow = 0;
    auto fetch = [&](int i) {
        const float* src = p.x + (static_cast<long long>(b) * p.R + i) * p.ldx;
        allow = 0;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int v = place(k);
            const uint32_t a = v < p.V ? (words[k] >> (v & 31)) & kFull : 0u;
            allow |= a << (k * VEC);
            if (a) {
                if (VEC == 4) *reinterpret_cast<float4*>(x[k]) = *reinterpret_cast<const float4*>(src + v);
                else x[k][0] = src[v];
            }
        }
    };
    masks(row0);
    fetch(row0);
    __syncthreads();  // the tables are clear

    auto hit = [&](int at) { atomicOr(&s_hit[at >> 5], 1u << (at & 31)); };
    const bool flagger = blockIdx.x == 0 && blockIdx.z == 0;
    bool bad = false;
    auto count = [&](int t, int v) {
        const int at = v - c0;
        if (v >= c0 && at < kLogitChunk && v < p.V) {
            if (t < n_prompt) atomicOr(&s_cnt[at], kKnown);
            else atomicAdd(&s_cnt[at], 1u);
            hit(at);
        }
        bad |= v < 0 || v >= p.V;
    };
    // four ids a load from the first whole 16 bytes on
    if (tid < min(head, n_hist)) count(tid, __ldg(ids + tid));
    const int quads = max(0, n_hist - head) / 4;
    int4 v4 = id4;
#pragma unroll 1
    for (int q = tid; q < quads; q += kLogitThreads) {
        const int t = head + 4 * q;
        int4 next = v4;
        if (q + kLogitThreads < quads) next = __ldg(reinterpret_cast<const int4*>(ids + head) + q + kLogitThreads);
        count(t, v4.x);
        count(t + 1, v4.y);
        count(t + 2, v4.z);
        count(t + 3, v4.w);
        v4 = next;
    }
    if (head + 4 * quads + tid < n_hist) count(head + 4 * quads + tid, __ldg(ids + head + 4 * quads + tid));
    for (int t = tid; t < n_bias; t += kLogitThreads) {
        const int v = t == tid ? bias_id : __ldg(bias_ids + t), at = v - c0;
        if (v >= c0 && at < kLogitChunk && v < p.V) {
            atomicMax(&s_bias[at], static_cast<uint32_t>(t) + 1u);  // the last entry holds
            hit(at);
        }
        bad |= v < 0 || v >= p.V;
    }
    if (flagger && bad) atomicOr(p.status, kStatusBadListId);
    if (tid < p.R - 1) {
        s_draft[tid] = draft;
        if (draft >= c0 && draft < p.V && draft - c0 < kLogitChunk) {
            atomicOr(&s_cnt[draft - c0], kDrafted);
            hit(draft - c0);
        }
        if (flagger && (draft < 0 || draft >= p.V)) atomicOr(p.status, kLogitBadDraft);
    }
    const float* bias = p.bias_ids ? p.bias_vals + static_cast<long long>(b) * p.bias_stride : nullptr;

    __syncthreads();  // the tables are complete
    // row i's corrected logit at entry `at`
    auto correct = [&](int i, int at, float y) {
        uint32_t c = s_cnt[at];
        if (c & kDrafted) {
            c &= ~kDrafted;
#pragma unroll 1
            for (int j = 0; j < i; ++j) c += s_draft[j] == c0 + at ? 1u : 0u;
        }
        if (c) y = y > 0.f ? __fdiv_rn(y, rep) : y * rep;
        const float n = static_cast<float>(c & ~kKnown);
        if (n > 0.f) y = y - fre * n - pre;
        if (bias) {
            const uint32_t be = s_bias[at];
            if (be) y += __ldg(bias + be - 1);
        }
        return y;
    };
    for (int i = row0; i < row1; ++i) {
        if (i + 1 < row1) masks(i + 1);
        const long long row = static_cast<long long>(b) * p.R + i;
        float* dst = p.out + row * p.ldo;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int v = place(k), at = v - c0;
            const uint32_t a = (allow >> (k * VEC)) & kFull;
            const uint32_t hits = (s_hit[at >> 5] >> (at & 31)) & a;
            if (hits) {  // (one branch a step: four, one an element, took 8 % longer)
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if ((hits >> e) & 1u) x[k][e] = correct(i, at + e, x[k][e]);
            }
            float mx = -INFINITY;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                if (!((a >> e) & 1u)) x[k][e] = -INFINITY;
                mx = fmaxf(mx, x[k][e]);
            }
            if (v < p.V) {
                if (VEC == 4) *reinterpret_cast<float4*>(dst + v) = *reinterpret_cast<float4*>(x[k]);
                else dst[v] = x[k][0];
            }
            if (p.bmax) {
#pragma unroll
                for (int o = 1; o < 16 / VEC; o <<= 1)
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                if (v < p.V && (at & 15) == 0)
                    p.bmax[row * ((p.V + 15) / 16) + (v >> 4)] = mx;
            }
        }
        if (i + 1 < row1) fetch(i + 1);
    }
}

cudaError_t launch_logits(const LogitsParams& p, int sms, cudaStream_t s) {
    // Blocks own 4096 entries, 1024 when blocks of one row and 4096 entries would leave
    // half of the SMs' places free: a small call is one block's latency, which a shorter
    // chunk cuts.  15 rows of 32003 (120 such blocks): 5.8 us with 1024, 8.1 with 4096;
    // 8 rows of 262144 (512 blocks): 8.2 with 1024, 7.9 with 4096.
    const long long rows = static_cast<long long>(p.B) * p.R;
    const int per = (p.V + 4095) / 4096 * rows <= 2LL * sms ? 1024 : 4096;
    const int chunks = (p.V + per - 1) / per;
    // few sequences: the rows are split over blocks too (each scans the history again):
    // split to four blocks an SM 8 rows of 262144 take 7.9 us, to eight 8.1, to two 11.2,
    // all rows in a block 30.9
    const long long blocks = static_cast<long long>(chunks) * p.B;
    int split = static_cast<int>((4LL * sms + blocks - 1) / blocks);
    if (split > p.R) split = p.R;
    const int step = (p.R + split - 1) / split;
    const auto a16 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; };
    const bool vec = p.V % 4 == 0 && p.ldx % 4 == 0 && p.ldo % 4 == 0 && a16(p.x) && a16(p.out);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(chunks, p.B, (p.R + step - 1) / step);
    cfg.blockDim = dim3(kLogitThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (per == 1024)
        return vec ? cudaLaunchKernelEx(&cfg, logits_kernel<4, 1024>, p, step)
                   : cudaLaunchKernelEx(&cfg, logits_kernel<1, 1024>, p, step);
    return vec ? cudaLaunchKernelEx(&cfg, logits_kernel<4, 4096>, p, step)
               : cudaLaunchKernelEx(&cfg, logits_kernel<1, 4096>, p, step);
}

}  // namespace vw4
