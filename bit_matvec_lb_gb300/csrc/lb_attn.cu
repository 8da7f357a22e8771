// lb_attn.cu -- attention over the paged 4-bit key/value cache.
#include "lb_kv4.cuh"

#include <math.h>

namespace lb {

struct AttnParams {
    const void *q;
    void *out;
    float *lse;
    const uint8_t *cache;
    const int32_t *table, *q_start, *kv_len;
    int64_t q_stride, out_stride, pages, width, T;
    int R, heads, kv_heads, shift, causal, window;
    float scale;
};

// One warp per query row and head: D / 32 dimensions a lane, one key at a time, running maximum
// and sum.
template <int D, typename T>
__global__ void __launch_bounds__(128) attn_simple_kernel(const AttnParams p) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t t = w / p.heads;
    const int h = (int)(w % p.heads);
    if (t >= p.T) return;
    int r = 0;
    while (r < p.R && !(t >= p.q_start[r] && t < p.q_start[r + 1])) r++;
    if (r == p.R) return;
    const int len = (int)min((int64_t)max(p.kv_len[r], 0), p.width << p.shift);
    const int pos = p.kv_len[r] - (p.q_start[r + 1] - (int)t);
    const int hi = p.causal ? min(len, pos + 1) : len;
    const int lo = p.window ? max(0, pos - p.window + 1) : 0;
    const int kvh = h / (p.heads / p.kv_heads);
    float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
    const T *qr = static_cast<const T *>(p.q) + t * p.q_stride + (int64_t)h * D + lane * E;
    for (int e = 0; e < E; e++) q[e] = (float)qr[e];
    for (int j = lo; j < hi; j++) {
        const int page = p.table[r * p.width + (j >> p.shift)];
        if (page < 0 || page >= p.pages) continue;
        const int in = j & ((1 << p.shift) - 1);
        const uint8_t *c = p.cache + kv4_chunk_offset(page, kvh, in, p.kv_heads, p.shift, D);
        const uint8_t *kc = c + (in & 15) * (D / 2), *vc = kc + kv4_codes_bytes(D);
        const __half2 kd = reinterpret_cast<const __half2 *>(c + 2 * kv4_codes_bytes(D))[in & 15];
        const __half2 vd =
            reinterpret_cast<const __half2 *>(c + 2 * kv4_codes_bytes(D) + kKv4PairBytes)[in & 15];
        float s = 0.f;
        for (int e = 0; e < E; e++) {
            const int i = lane * E + e;
            s += q[e] * (__low2float(kd) * ((float)((kc[i / 2] >> (i % 2 * 4)) & 15) - __high2float(kd)));
        }
        for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
        s *= p.scale;
        const float mn = fmaxf(m, s), f = m == -INFINITY ? 0.f : expf(m - mn), w1 = expf(s - mn);
        m = mn;
        l = l * f + w1;
        for (int e = 0; e < E; e++) {
            const int i = lane * E + e;
            const float v = __low2float(vd) * ((float)((vc[i / 2] >> (i % 2 * 4)) & 15) - __high2float(vd));
            o[e] = o[e] * f + w1 * v;
        }
    }
    T *orow = static_cast<T *>(p.out) + t * p.out_stride + (int64_t)h * D + lane * E;
    for (int e = 0; e < E; e++) orow[e] = (T)(l > 0.f ? o[e] / l : 0.f);
    if (p.lse && lane == 0) p.lse[t * p.heads + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace lb

LB_EXPORT size_t lb_attn_kv4_workspace_bytes(int heads, int kv_heads, int head_dim, int64_t max_q) {
    return heads < 1 || kv_heads < 1 || head_dim < 1 || max_q < 1 ? 0 : 16;
}

LB_EXPORT int lb_attn_kv4(const void *q, int type, int64_t q_stride, const uint8_t *cache,
                          int64_t pages, int page_size, int heads, int kv_heads, int head_dim,
                          const int32_t *block_table, int64_t table_width, const int32_t *q_start,
                          const int32_t *kv_len, int64_t R, int64_t T, int64_t max_q, float scale,
                          int causal, int64_t window, void *out, int64_t out_stride,
                          float *lse_opt, void *workspace, size_t workspace_bytes, void *stream) {
    using namespace lb;
    const int64_t lim = int64_t(1) << 31;
    if (!q || !cache || !block_table || !q_start || !kv_len || !out || !workspace) return LB_ERR_NULL;
    if ((type != LB_OUT_F32 && type != LB_OUT_BF16) ||
        !kv4_shape_ok(pages, page_size, kv_heads, head_dim) || heads < kv_heads ||
        heads % kv_heads || heads / kv_heads > 64 || R < 1 || R > LB_KV_MAX_REQUESTS || T < 0 ||
        T >= lim || table_width < 1 || table_width >= lim / page_size || max_q < 1 || max_q >= lim ||
        !(scale > 0.f) || !(scale < INFINITY) || window < 0 || window >= lim || (window && !causal) ||
        q_stride < (int64_t)heads * head_dim || out_stride < (int64_t)heads * head_dim ||
        workspace_bytes < lb_attn_kv4_workspace_bytes(heads, kv_heads, head_dim, max_q))
        return LB_ERR_SHAPE;
    const int64_t per16 = type == LB_OUT_F32 ? 4 : 8;
    if (!aligned16(q) || !aligned16(cache) || !aligned16(out) || !aligned16(workspace) ||
        q_stride % per16 || out_stride % per16 || !aligned_to(block_table, 4) ||
        !aligned_to(q_start, 4) || !aligned_to(kv_len, 4) || !aligned_to(lse_opt, 4))
        return LB_ERR_ALIGN;
    DeviceInfo di;
    if (int e = current_device_info(&di)) return e;
    if (T == 0) return LB_OK;
    const AttnParams p{q, out, lse_opt, cache, block_table, q_start, kv_len, q_stride, out_stride,
                       pages, table_width, T, (int)R, heads, kv_heads, page_shift_of(page_size),
                       causal, (int)window, scale};
    const dim3 grid((unsigned)((T * heads + 3) / 4));
    cudaStream_t st = as_stream(stream);
    if (type == LB_OUT_F32)
        return head_dim == 64 ? launch_pdl(attn_simple_kernel<64, float>, grid, dim3(128), 0, st, p)
                              : launch_pdl(attn_simple_kernel<128, float>, grid, dim3(128), 0, st, p);
    return head_dim == 64
               ? launch_pdl(attn_simple_kernel<64, __nv_bfloat16>, grid, dim3(128), 0, st, p)
               : launch_pdl(attn_simple_kernel<128, __nv_bfloat16>, grid, dim3(128), 0, st, p);
}
