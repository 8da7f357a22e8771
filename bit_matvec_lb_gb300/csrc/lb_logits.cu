// lb_logits.cu -- penalties for repeated tokens, biases and grammar masks on logits.
#include <cooperative_groups.h>

#include "lb_kv4.cuh"

namespace lb {
namespace cg = cooperative_groups;

// One row is one thread-block cluster; each CTA owns a slice of the vocabulary and keeps for each
// of its tokens a word of shared memory: bit 31 = in the prompt, the rest = times in the output
// (and a second word, 1 + the last entry of the bias list, if there are biases).  The cluster's
// threads share the lists and count each token in its owner's shared memory (distributed shared
// memory atomics on integers, so the order does not matter); after a cluster barrier every CTA
// passes over its slice once.  Bound by reading and writing the logits: the lists are read once
// and nothing goes through global memory.
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
constexpr int kLogitCluster = 16;
constexpr uint32_t kInPrompt = 0x80000000u;

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
    if (count) {
        x = x > 0.f ? __fdiv_rn(x, r.repetition) : __fmul_rn(x, r.repetition);
        const uint32_t n = count & ~kInPrompt;
        if (n) x = __fsub_rn(__fsub_rn(x, __fmul_rn((float)n, r.frequency)), r.presence);
    }
    if (bias) x = __fadd_rn(x, r.bias[bias - 1]);
    return allowed ? x : __int_as_float(0xff800000);
}

// LISTS: the call has lists (otherwise the kernel has no cluster and no shared memory);
// BIAS: one of them is a bias list.
template <typename T, bool LISTS, bool BIAS>
__global__ void __launch_bounds__(kLogitThreads) logits_kernel(const LogitParams p) {
    extern __shared__ uint4 smem[];
    constexpr int VEC = 16 / sizeof(T);
    const int tid = threadIdx.x;
    const int b = blockIdx.y, rank = blockIdx.x, ranks = gridDim.x;
    const int64_t v0 = (int64_t)rank * p.slice;
    const int n = (int)max((int64_t)0, min((int64_t)p.slice, p.V - v0));
    // Elements before the row's first 16-byte boundary shift everything, so that a group of VEC
    // is one aligned load; slices are a multiple of 32, so the shift is the row's.
    const int64_t row = (int64_t)b * p.stride;
    const int shift = (int)(((reinterpret_cast<uintptr_t>(p.x) / sizeof(T)) + row) % VEC);
    uint32_t *count = reinterpret_cast<uint32_t *>(smem);     // [slice + VEC], element i at i + shift
    uint32_t *bias = count + (BIAS ? p.slice + VEC : 0);
    if (LISTS) {
        const int words = (p.slice + VEC) * (BIAS ? 2 : 1) / 4;
        for (int i = tid; i < words; i += kLogitThreads) smem[i] = make_uint4(0, 0, 0, 0);
    }
    pdl_wait();
    pdl_launch_dependents();
    RowRules r;
    r.repetition = p.repetition ? p.repetition[b] : 1.f;
    r.presence = p.presence ? p.presence[b] : 0.f;
    r.frequency = p.frequency ? p.frequency[b] : 0.f;
    r.bias = BIAS ? p.bias_values + p.bias_start[b] : nullptr;
    r.mask = nullptr;
    if (p.mask) {
        const int64_t m = p.mask_row ? p.mask_row[b] : b;
        if (m >= 0 && m < p.mask_rows) r.mask = p.mask + m * p.mask_stride;
    }
    if (LISTS) {
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();  // every CTA's words are zero
        const int first = rank * kLogitThreads + tid, step = ranks * kLogitThreads;
        if (p.prompt_ids) {
            const int e = p.prompt_start[b + 1];
            for (int64_t i = (int64_t)p.prompt_start[b] + first; i < e; i += step) {
                const int v = p.prompt_ids[i];
                if (v < 0 || v >= p.V) continue;
                const int owner = v / p.slice;
                atomicOr(cluster.map_shared_rank(count, owner) + shift + (v - owner * p.slice), kInPrompt);
            }
        }
        if (p.output_ids) {
            const int e = p.output_start[b + 1];
            for (int64_t i = (int64_t)p.output_start[b] + first; i < e; i += step) {
                const int v = p.output_ids[i];
                if (v < 0 || v >= p.V) continue;
                const int owner = v / p.slice;
                atomicAdd(cluster.map_shared_rank(count, owner) + shift + (v - owner * p.slice), 1u);
            }
        }
        if (BIAS) {
            const int s = p.bias_start[b], e = p.bias_start[b + 1];
            for (int64_t i = (int64_t)s + first; i < e; i += step) {
                const int v = p.bias_ids[i];
                if (v < 0 || v >= p.V) continue;
                const int owner = v / p.slice;
                atomicMax(cluster.map_shared_rank(bias, owner) + shift + (v - owner * p.slice),
                          (uint32_t)(i - s) + 1u);
            }
        }
        cluster.sync();  // every count has arrived; no CTA touches another's memory after this
    }
    const T *x = static_cast<const T *>(p.x) + row + v0;
    T *out = static_cast<T *>(p.out) + (int64_t)b * p.out_stride + v0;
    const bool same = (reinterpret_cast<uintptr_t>(out) & 15) == (reinterpret_cast<uintptr_t>(x) & 15);
    for (int g = tid; n > 0 && g * VEC < n + shift; g += kLogitThreads) {
        const int i0 = g * VEC - shift;  // the group's first element, < 0 in the first group
        uint32_t c[VEC] = {}, bi[VEC] = {};
        if (LISTS) {
#pragma unroll
            for (int k = 0; k < VEC; k += 4) {
                const uint4 w = smem[(g * VEC + k) / 4];
                c[k] = w.x, c[k + 1] = w.y, c[k + 2] = w.z, c[k + 3] = w.w;
            }
        }
        if (BIAS) {
#pragma unroll
            for (int k = 0; k < VEC; k += 4) {
                const uint4 w = reinterpret_cast<const uint4 *>(bias)[(g * VEC + k) / 4];
                bi[k] = w.x, bi[k + 1] = w.y, bi[k + 2] = w.z, bi[k + 3] = w.w;
            }
        }
        // Mask bits of the group, its first element's in bit 0.
        uint32_t bits = 0xFFFFFFFFu;
        const int a = max(i0, 0);
        if (r.mask) {
            const int64_t v = v0 + a;
            const uint32_t w0 = r.mask[v >> 5];
            const int64_t last = min(v + VEC - 1, (int64_t)p.V - 1);
            const uint32_t w1 = (last >> 5) != (v >> 5) ? r.mask[last >> 5] : 0u;
            bits = __funnelshift_r(w0, w1, (int)(v & 31)) << (a - i0);
        }
        if (i0 >= 0 && i0 + VEC <= n) {
            T e[VEC];
            *reinterpret_cast<uint4 *>(e) = *reinterpret_cast<const uint4 *>(x + i0);
#pragma unroll
            for (int k = 0; k < VEC; k++)
                logit_store(e + k, adjust(logit_load(e + k), c[k], bi[k], (bits >> k) & 1, r));
            if (same) {
                *reinterpret_cast<uint4 *>(out + i0) = *reinterpret_cast<const uint4 *>(e);
            } else {
#pragma unroll
                for (int k = 0; k < VEC; k++) out[i0 + k] = e[k];
            }
        } else {
#pragma unroll
            for (int k = 0; k < VEC; k++)
                if (i0 + k >= 0 && i0 + k < n)
                    logit_store(out + i0 + k, adjust(logit_load(x + i0 + k), c[k], bi[k], (bits >> k) & 1, r));
        }
    }
}

template <typename T, bool LISTS, bool BIAS>
static int launch_logits(const LogitParams &p0, int64_t B, cudaStream_t st) {
    constexpr int VEC = 16 / sizeof(T);
    void (*kernel)(LogitParams) = logits_kernel<T, LISTS, BIAS>;
    LogitParams p = p0;
    const int ranks = kLogitCluster;
    p.slice = ((p.V + ranks - 1) / ranks + 31) / 32 * 32;
    const size_t smem = LISTS ? (size_t)(p.slice + VEC) * 4 * (BIAS ? 2 : 1) : 0;
    int per_sm;
    if (int e = prepare_kernel((const void *)kernel, kLogitThreads, smem, &per_sm)) return e;
    if (!LISTS)
        return launch_pdl(kernel, dim3(ranks, (unsigned)B), dim3(kLogitThreads), 0, st, p);
    cudaError_t e = cudaFuncSetAttribute((const void *)kernel,
                                         cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(ranks, (unsigned)B);
        cfg.blockDim = dim3(kLogitThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim = {(unsigned)ranks, 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        e = cudaLaunchKernelEx(&cfg, kernel, p);
    }
    if (e == cudaSuccess) return LB_OK;
    record_cuda_error(e);
    return LB_ERR_LAUNCH;
}

template <typename T>
static int dispatch_logits(const LogitParams &p, int64_t B, cudaStream_t st) {
    if (p.bias_ids) return launch_logits<T, true, true>(p, B, st);
    if (p.prompt_ids || p.output_ids) return launch_logits<T, true, false>(p, B, st);
    return launch_logits<T, false, false>(p, B, st);
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
    return type == LB_OUT_F32 ? dispatch_logits<float>(p, B, as_stream(stream))
                              : dispatch_logits<__nv_bfloat16>(p, B, as_stream(stream));
}
