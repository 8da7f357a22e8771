// lb_attn.cuh -- what the attention kernels over the 4-bit cache share: parameters, the split of
// the work into equal runs of key tiles, and the records of partial results.
#pragma once
#include "lb_kv4.cuh"

namespace lb {

struct AttnParams {
    const void *q;
    void *out;
    float *lse;
    const uint8_t *cache;
    const int32_t *table, *q_start, *kv_len;
    int64_t q_stride, out_stride, pages, width, T;
    int R, heads, kv_heads, group, shift, causal, window;
    float scale;
    int rows_lo, rows_hi;  // this launch takes the requests with rows_lo < queries * group <= rows_hi
    int *error;
    float *part;     // partial sums: [slot][row][D], slot = 2 * CTA + (0: continued, 1: begun)
    float2 *stat;    // [slot][row] {reference exponent, sum of weights}
    float4 *sums;    // sums over parts of an item's keys (prompts in fp32): [CTA][row tile][D / 4][row]
    int4 *record;    // [slot] {request, item of the request, 1 + the CTA that began the item if
                     // this is its last part else 0, rows}; x < 0: none
};

// Many-row requests (lb_attn_tc.cu): scratch bytes and launches.
size_t attn_prompt_workspace(int head_dim);
int attn_prompt(const AttnParams &p, int type, int head_dim, uint8_t *workspace, int sms,
                cudaStream_t st);

// A request as the kernels see it; everything is clamped so that no access leaves its buffer.
struct Request {
    int q0, n;       // first query row, queries
    int len;         // tokens of the cache that may be read
    int base;        // position of query 0 (kv_len - n, may be negative)
};

__device__ __forceinline__ Request load_request(const AttnParams &p, int r) {
    Request q;
    const int T = (int)p.T;
    q.q0 = min(max(p.q_start[r], 0), T);
    q.n = max(min(p.q_start[r + 1], T) - q.q0, 0);
    const int len = p.kv_len[r];
    q.len = (int)min((int64_t)max(len, 0), p.width << p.shift);
    q.base = max(len, 0) - q.n;
    const int64_t rows = (int64_t)q.n * p.group;
    if (rows <= p.rows_lo || rows > p.rows_hi) q.n = 0;
    return q;
}

// First token that the window shows to query i, 0 without one.  (In 64 bits: a request may have more
// queries than tokens, and the window may be as long as "no limit" is written.)
__device__ __forceinline__ int window_start(const AttnParams &p, const Request &q, int i) {
    return p.window ? (int)max((int64_t)q.base + i - p.window + 1, (int64_t)0) : 0;
}

// Tokens [lo, hi) that the queries i0 .. i1 - 1 of a request can see among them.
__device__ __forceinline__ void visible_range(const AttnParams &p, const Request &q, int i0, int i1,
                                              int &lo, int &hi) {
    hi = p.causal ? max(0, min(q.len, q.base + i1)) : q.len;
    lo = min(window_start(p, q, i0), hi);
}

// Orders this thread's ordinary shared-memory accesses before later bulk copies into the same bytes.
__device__ __forceinline__ void fence_proxy_async_shared() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.69314718055994531f;

// The power of two that brings a row whose largest magnitude is `amax` to [2^12, 2^13) (fp16 then
// holds its small values too), and its inverse.  Infinities and NaN are left to spread in their row.
__device__ __forceinline__ void row_power(float amax, float &up, float &down) {
    const int e = max((int)((__float_as_uint(amax) >> 23) & 255), 1);
    const int x = e == 255 ? 0 : min(139 - e, 126);
    up = __uint_as_float((uint32_t)(x + 127) << 23);
    down = __uint_as_float((uint32_t)(127 - x) << 23);
}

// log2 of an fp16 scale, to a small error and at least -24 (a scale of 0 gives weights of 0 whatever
// its score).
__device__ __forceinline__ float scale_log2(float d) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaxf(d, 5.9604645e-8f)));
    return y;
}

__device__ __forceinline__ void store_value(float *p, float x) { *p = x; }
__device__ __forceinline__ void store_value(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

}  // namespace lb
