// lb_logits.cu -- penalties for repeated tokens, biases and grammar masks on logits.
#include "lb_kv4.cuh"

namespace lb {

// A CTA owns a slice of one row's vocabulary.  For each of its tokens it keeps a word of shared
// memory: bit 31 = in the prompt, bits 0-29 = times in the output (and 16 bits more, 1 + the last
// entry of the bias list, if there are biases).  It reads the row's whole lists and counts the tokens
// of its slice (shared-memory atomics on integers, so the order does not matter); who finds a token's
// word empty queues the token.  Then it passes over the slice once with the mask alone, and at last
// goes through the queue.  So the work on listed tokens, many in the slices of common tokens and few
// elsewhere, is spread over the threads by their number, not over the lanes whose logits they are.
// The bytes would take 17.6 us for 96 rows of 151669 fp32 (bf16: 9.0).  With about 4000 listed tokens a
// row it takes 39 (27): a slice's words fill 64 KB, three CTAs fit an SM, and each is a chain of
// phases (words zeroed, ends of the lists, ids, counts, mask, queue) behind barriers, four times
// over; the lists' own bytes, read from L2 by every slice, are a few us.  With the lanes adjusting
// their own logits 48, with a row's lists shared by a cluster of 16 CTAs and counts in distributed
// shared memory 68 (clusters start one after another).
struct LogitParams {
    const void *x;
    void *out;
    int64_t stride, out_stride, mask_stride, mask_rows;
    const int32_t *prompt_ids, *prompt_start, *output_ids, *output_start, *bias_ids, *bias_start;
    const float *repetition, *presence, *frequency, *bias_values;
    const uint32_t *mask;
    const int32_t *mask_row;
    int V, slice;
};

constexpr int kLogitThreads = 512;
constexpr int kLogitSlice = 8192;    // tokens of a slice at most
constexpr int kLogitLeast = 1024;    // ... and at least
constexpr int kLogitPerSm = 3;       // CTAs per SM that fill the GPU
constexpr int kLogitIds = 4;         // ids of a list a thread asks for ahead
constexpr uint32_t kInPrompt = 0x80000000u, kBiased = 0x40000000u;

template <typename T>
__device__ __forceinline__ float logit_load(const T *p);
template <>
__device__ __forceinline__ float logit_load(const float *p) { return *p; }
template <>
__device__ __forceinline__ float logit_load(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void logit_store(float *p, float x) { *p = x; }
__device__ __forceinline__ void logit_store(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

struct RowRules {
    float repetition, presence, frequency;
    const uint32_t *mask;  // the row's words, or NULL
    const float *bias;     // values of the row's list
};

__device__ __forceinline__ float adjust(float x, uint32_t count, uint32_t bias, bool allowed,
                                        const RowRules &r) {
    if (count & ~kBiased) {
        x = x > 0.f ? __fdiv_rn(x, r.repetition) : __fmul_rn(x, r.repetition);
        const uint32_t n = count & ~(kInPrompt | kBiased);
        if (n) x = __fsub_rn(__fsub_rn(x, __fmul_rn((float)n, r.frequency)), r.presence);
    }
    if (bias) x = __fadd_rn(x, r.bias[bias - 1]);
    return allowed ? x : __int_as_float(0xff800000);
}

// *p = max(*p, entry) on 16 bits of shared memory, by the word they lie in.
__device__ __forceinline__ void later_entry(uint16_t *p, uint32_t entry) {
    uint32_t *word = reinterpret_cast<uint32_t *>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(3));
    const int up = reinterpret_cast<uintptr_t>(p) & 2 ? 16 : 0;
    uint32_t old = *reinterpret_cast<volatile uint32_t *>(word);
    while (((old >> up) & 0xFFFFu) < entry) {
        const uint32_t seen = atomicCAS(word, old, (old & ~(0xFFFFu << up)) | entry << up);
        if (seen == old) break;
        old = seen;
    }
}

// LISTS: the call has lists (otherwise the kernel has no shared memory); BIAS: one of them is a
// bias list.
template <typename T, bool LISTS, bool BIAS>
__global__ void __launch_bounds__(kLogitThreads) logits_kernel(const LogitParams p) {
    extern __shared__ uint4 smem[];
    constexpr int VEC = 16 / sizeof(T);
    constexpr int AHEAD = kLogitSlice / VEC / kLogitThreads;  // groups of a thread
    constexpr int LISTS_N = BIAS ? 3 : 2;
    const int tid = threadIdx.x, b = blockIdx.y;
    const int v0 = blockIdx.x * p.slice, n = min(p.slice, p.V - v0);
    // Elements before the row's first 16-byte boundary shift everything, so that a group of VEC
    // is one aligned load; slices are a multiple of 32, so the shift is the row's.
    const T *x = static_cast<const T *>(p.x) + (int64_t)b * p.stride + v0;
    T *out = static_cast<T *>(p.out) + (int64_t)b * p.out_stride + v0;
    const int shift = (int)(reinterpret_cast<uintptr_t>(x) / sizeof(T) % VEC);
    const bool same = (reinterpret_cast<uintptr_t>(out) & 15) == (reinterpret_cast<uintptr_t>(x) & 15);
    const int groups = (n + shift + VEC - 1) / VEC;
    // [slice] counts, [slice] queue, [slice] bias entries
    uint32_t *count = reinterpret_cast<uint32_t *>(smem);
    uint16_t *queue = reinterpret_cast<uint16_t *>(count + p.slice);
    uint16_t *bias = queue + p.slice;
    __shared__ int queued;
    if (LISTS) {
        for (int i = tid; i < p.slice / 4; i += kLogitThreads) smem[i] = make_uint4(0, 0, 0, 0);
        if (BIAS)
            for (int i = tid; i < p.slice / 8; i += kLogitThreads)
                reinterpret_cast<uint4 *>(bias)[i] = make_uint4(0, 0, 0, 0);
        if (tid == 0) queued = 0;
    }
    pdl_wait();
    pdl_launch_dependents();
    // What depends on nothing is asked for first: the logits, the row's numbers, its lists' ends.
    uint4 data[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; k++) {
        const int i0 = (tid + k * kLogitThreads) * VEC - shift;
        data[k] = make_uint4(0, 0, 0, 0);
        if (i0 >= 0 && i0 + VEC <= n) data[k] = *reinterpret_cast<const uint4 *>(x + i0);
    }
    RowRules r;
    const int64_t mask_row = p.mask ? (p.mask_row ? p.mask_row[b] : b) : -1;
    r.repetition = p.repetition ? p.repetition[b] : 1.f;
    r.presence = p.presence ? p.presence[b] : 0.f;
    r.frequency = p.frequency ? p.frequency[b] : 0.f;
    const int32_t *list[3] = {p.prompt_ids, p.output_ids, p.bias_ids};
    const int32_t *start[3] = {p.prompt_start, p.output_start, p.bias_start};
    int begin[3] = {}, end[3] = {};
    if (LISTS) {
#pragma unroll
        for (int k = 0; k < LISTS_N; k++)
            if (list[k]) begin[k] = start[k][b], end[k] = start[k][b + 1];
        if (BIAS) end[2] = (int)min((int64_t)end[2], (int64_t)begin[2] + LB_LOGITS_MAX_BIAS);
    }
    r.bias = BIAS ? p.bias_values + begin[2] : nullptr;
    r.mask = mask_row >= 0 && mask_row < p.mask_rows ? p.mask + mask_row * p.mask_stride : nullptr;
    // The first ids of each list, one after another over the threads.
    int ids[3][kLogitIds];
    if (LISTS) {
#pragma unroll
        for (int k = 0; k < LISTS_N; k++)
#pragma unroll
            for (int e = 0; e < (k == 2 ? 1 : kLogitIds); e++) {
                const uint32_t i = (uint32_t)begin[k] + tid + e * kLogitThreads;
                ids[k][e] = i < (uint32_t)end[k] ? list[k][i] : -1;
            }
    }
    if (LISTS) {
        __syncthreads();  // the words are zero
        // Counts entry i of list k, token id, if it lies in the slice.
        auto one = [&](int k, int id, uint32_t i) {
            const uint32_t at = (uint32_t)id - (uint32_t)v0;  // beyond n for ids before the slice
            if (at >= (uint32_t)n) return;
            const uint32_t mark = k == 0 ? kInPrompt : k == 1 ? 1u : kBiased;
            const uint32_t old = k == 1 ? atomicAdd(count + at, mark) : atomicOr(count + at, mark);
            if (old == 0) queue[atomicAdd(&queued, 1)] = (uint16_t)at;
            if (k == 2) later_entry(bias + at, i - (uint32_t)begin[2] + 1u);
        };
#pragma unroll
        for (int k = 0; k < LISTS_N; k++) {
            constexpr int most = kLogitIds;
#pragma unroll
            for (int e = 0; e < (k == 2 ? 1 : most); e++)
                one(k, ids[k][e], (uint32_t)begin[k] + tid + e * kLogitThreads);
#pragma unroll 2
            for (uint32_t i = (uint32_t)begin[k] + tid + (k == 2 ? 1 : most) * kLogitThreads;
                 i < (uint32_t)end[k]; i += kLogitThreads)
                one(k, list[k][i], i);
        }
    }
    // The mask over every group.
#pragma unroll
    for (int k = 0; k <= AHEAD; k++) {  // (a row that does not begin on 16 bytes has one group more)
        const int i0 = (tid + k * kLogitThreads) * VEC - shift;
        if (tid + k * kLogitThreads >= groups) break;
        uint32_t bits = 0xFFFFFFFFu;  // the group's, its first element's in bit 0
        if (r.mask) {
            const int a = max(i0, 0), v = v0 + a, last = min(v + VEC - 1, p.V - 1);
            const uint32_t w0 = r.mask[v >> 5];
            const uint32_t w1 = (last >> 5) != (v >> 5) ? r.mask[last >> 5] : 0u;
            bits = __funnelshift_r(w0, w1, v & 31) << (a - i0);
        }
        if (k < AHEAD && same && i0 >= 0 && i0 + VEC <= n) {
            T e[VEC];
            *reinterpret_cast<uint4 *>(e) = data[k < AHEAD ? k : 0];
#pragma unroll
            for (int q = 0; q < VEC; q++)
                if (!(bits >> q & 1)) logit_store(e + q, __int_as_float(0xff800000));
            *reinterpret_cast<uint4 *>(out + i0) = *reinterpret_cast<const uint4 *>(e);
        } else {
#pragma unroll 1
            for (int q = max(-i0, 0); q < min(VEC, n - i0); q++)
                logit_store(out + i0 + q,
                            bits >> q & 1 ? logit_load(x + i0 + q) : __int_as_float(0xff800000));
        }
    }
    if (LISTS) {
        __syncthreads();  // every count is there, and the mask's values are written
#pragma unroll 2
        for (int i = tid; i < queued; i += kLogitThreads) {
            const int at = queue[i], v = v0 + at;
            const bool allowed = !r.mask || (r.mask[v >> 5] >> (v & 31) & 1);
            logit_store(out + at, adjust(logit_load(x + at), count[at], BIAS ? bias[at] : 0u, allowed, r));
        }
    }
}

template <typename T, bool LISTS, bool BIAS>
static int launch_logits(const LogitParams &p0, int64_t B, int sms, cudaStream_t st) {
    void (*kernel)(LogitParams) = logits_kernel<T, LISTS, BIAS>;
    LogitParams p = p0;
    // Slices of kLogitSlice, or smaller ones while there are too few to fill the GPU.
    const int64_t fill = kLogitPerSm * (int64_t)sms / B;
    int64_t slices = (p.V + kLogitSlice - 1) / kLogitSlice;
    if (slices < fill) slices = fill < (p.V + kLogitLeast - 1) / kLogitLeast ? fill : (p.V + kLogitLeast - 1) / kLogitLeast;
    p.slice = (int)(((p.V + slices - 1) / slices + 31) / 32 * 32);
    const size_t smem = LISTS ? (size_t)p.slice * (BIAS ? 8 : 6) : 0;
    int per_sm;
    if (int e = prepare_kernel((const void *)kernel, kLogitThreads, smem, &per_sm)) return e;
    return launch_pdl(kernel, dim3((unsigned)((p.V + p.slice - 1) / p.slice), (unsigned)B),
                      dim3(kLogitThreads), smem, st, p);
}

template <typename T>
static int dispatch_logits(const LogitParams &p, int64_t B, int sms, cudaStream_t st) {
    if (p.bias_ids) return launch_logits<T, true, true>(p, B, sms, st);
    if (p.prompt_ids || p.output_ids) return launch_logits<T, true, false>(p, B, sms, st);
    return launch_logits<T, false, false>(p, B, sms, st);
}

}  // namespace lb

LB_EXPORT int lb_logits_adjust(const void *logits, int type, int64_t stride, void *out,
                               int64_t out_stride, int64_t B, int64_t V,
                               const lb_logit_rules *rules, void *stream) {
    using namespace lb;
    if (!logits || !out || !rules) return LB_ERR_NULL;
    const lb_logit_rules &r = *rules;
    if ((r.prompt_ids && !r.prompt_start) || (r.output_ids && !r.output_start) ||
        (r.bias_ids && (!r.bias_start || !r.bias_values)))
        return LB_ERR_NULL;
    if ((type != LB_OUT_F32 && type != LB_OUT_BF16) || B < 1 || B > 65535 || V < 1 ||
        V > LB_LOGITS_MAX_V || stride < V || out_stride < V ||
        (r.mask && (r.mask_stride < (V + 31) / 32 || r.mask_rows < (r.mask_row_opt ? 0 : B))))
        return LB_ERR_SHAPE;
    const uintptr_t size = type == LB_OUT_F32 ? 4 : 2;
    if (!aligned_to(logits, size) || !aligned_to(out, size)) return LB_ERR_ALIGN;
    for (const void *q : {(const void *)r.prompt_ids, (const void *)r.prompt_start,
                          (const void *)r.output_ids, (const void *)r.output_start,
                          (const void *)r.repetition, (const void *)r.presence,
                          (const void *)r.frequency, (const void *)r.bias_ids,
                          (const void *)r.bias_values, (const void *)r.bias_start,
                          (const void *)r.mask, (const void *)r.mask_row_opt})
        if (!aligned_to(q, 4)) return LB_ERR_ALIGN;
    DeviceInfo di;
    if (int e = current_device_info(&di)) return e;
    LogitParams p{};
    p.x = logits, p.out = out, p.stride = stride, p.out_stride = out_stride;
    p.mask_stride = r.mask_stride, p.mask_rows = r.mask_rows;
    p.prompt_ids = r.prompt_ids, p.prompt_start = r.prompt_start;
    p.output_ids = r.output_ids, p.output_start = r.output_start;
    p.bias_ids = r.bias_ids, p.bias_start = r.bias_start, p.bias_values = r.bias_values;
    p.repetition = r.repetition, p.presence = r.presence, p.frequency = r.frequency;
    p.mask = r.mask, p.mask_row = r.mask_row_opt, p.V = (int)V;
    return type == LB_OUT_F32 ? dispatch_logits<float>(p, B, di.sms, as_stream(stream))
                              : dispatch_logits<__nv_bfloat16>(p, B, di.sms, as_stream(stream));
}
