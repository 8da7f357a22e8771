// lb_q4.cu -- entry points over 4-bit weights with group scales: the product for a few and for many
// tokens, and the experts' feed-forward blocks.
//
// Experts: the gate and up rows are one product that ends in h = silu(gate) * up, kept in binary32 at
// the pairs' places by expert; the down rows' product leaves an output row per pair, in binary32; a last kernel adds
// each token's up in the order of its places (no atomics, so the same inputs give the same bits).  Few pairs per expert:
// three kernels (lb_q4_gemv.cu twice); many: five, with rows for the tensor cores laid out before each product.
#include "lb_q4.cuh"

#include <algorithm>

namespace lb {

constexpr int kCombineThreads = 256;

// y[t] = sum over j of weights[t][j] * part[t k + j].  Bound by memory: k numbers of 4 bytes in for one out.  Eight columns
// of a token per thread.  (The experts' outputs in fp16, scaled for every 32 rows, make this 7 us shorter for 32768 of
// 2048 and the product that leaves them 50 us longer.)
template <typename T>
__global__ void __launch_bounds__(kCombineThreads)
    experts_combine_kernel(const float *part, const int32_t *ids, const float *weights, T *y,
                           int64_t y_stride, int64_t tokens, int k, int columns) {
    pdl_launch_dependents();
    pdl_wait();
    const int eights = columns / 8;
    const int64_t i = blockIdx.x * (int64_t)kCombineThreads + threadIdx.x;
    if (i >= tokens * eights) return;
    const int64_t t = i / eights;
    const int c = (int)(i - t * eights) * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int j = 0; j < k; j++) {
        const int64_t pair = t * k + j;
        if (ids[pair] < 0) continue;
        const float w = weights[pair];
        float a[8];
        load8(part + pair * columns + c, a);
#pragma unroll
        for (int e = 0; e < 8; e++) v[e] = fmaf(w, a[e], v[e]);
    }
    T *to = y + t * y_stride + c;
    if ((reinterpret_cast<uintptr_t>(to) & 15) == 0) {
        store8(to, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; e++) {
            if constexpr (sizeof(T) == 4) to[e] = v[e];
            else to[e] = __float2bfloat16_rn(v[e]);
        }
    }
}

// Arguments that lb_gemv_q4 and lb_gemm_q4 share.
static int check_product(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, int group,
                         const void *x, int type, int64_t x_stride, const void *y, int64_t y_stride,
                         int64_t M, int64_t N, int64_t K) {
    if (!codes || !scales || (M != 0 && (!x || !y))) return LB_ERR_NULL;   // (no tokens: empty tensors lie nowhere)
    if (!q4_group_ok(group) || !q4_type_ok(type) || M < 0 || M > (1 << 20) || N < 1 || N > (1 << 23) ||
        K < group || K > LB_Q4_MAX_K || K % group != 0 || x_stride < K || y_stride < N ||
        x_stride > 0x7fffffff || y_stride > 0x7fffffff)
        return LB_ERR_SHAPE;
    const int size = type == LB_OUT_F32 ? 4 : 2;
    if (!aligned16(codes) || !aligned16(scales) || !aligned16(zeros) || !aligned16(x) ||
        x_stride * size % 16 != 0 || !aligned_to(y, size))
        return LB_ERR_ALIGN;
    return LB_OK;
}

static Q4Params product_of(const uint16_t *scales, const uint8_t *zeros, int group, const void *x,
                           int64_t x_stride, void *y, int64_t y_stride, int64_t M, int64_t N, int64_t K) {
    Q4Params p{};
    p.scales = scales, p.zeros = zeros, p.group = group, p.pitch = q4_pitch(K, group);
    p.x = x, p.x_stride = x_stride, p.y = y, p.y_stride = y_stride;
    p.N = N, p.T = M, p.K = (int)K;
    p.error = device_error_word();
    return p;
}

static size_t align256(size_t n) { return (n + 255) / 256 * 256; }
static int parts_of(int type) { return type == LB_OUT_F32 ? 2 : 1; }

// A piece of a workspace: rows of x as the tensor cores take them.
struct RowsAt {
    uint16_t *to;
    float *scale;
};
static size_t rows_bytes(int64_t n, int64_t K, int type) {
    return align256((size_t)n * K * 2 * parts_of(type)) + align256((size_t)n * 4);
}
static RowsAt rows_at(uint8_t *at, int64_t n, int64_t K, int type) {
    return {reinterpret_cast<uint16_t *>(at),
            reinterpret_cast<float *>(at + align256((size_t)n * K * 2 * parts_of(type)))};
}

// Pairs per expert from which the experts' products run on tcgen05, whose time hardly grows with them; the other kernel
// takes pieces of eight tokens, so its time grows with every one that begins.  64 experts of 2048 x 1024, eight per
// token, 6, 12 and 16 pairs each: fp32 113, 149 and 180 us against tcgen05's 141, 145 and 148; bf16 88, 113 and 133
// against 98, 100 and 101.  Eight of 4096 x 8192, two per token, 8, 12 and 16: fp32 203, 238 and 308 against 195, 215
// and 219; bf16 183, 203 and 265 against 150, 162 and 163.  32 of 1024 x 512, four per token, 12 and 16: fp32 37 and 45
// against 37 and 37; bf16 31 and 37 against 31 and 31.
constexpr int many_pairs(int type) { return type == LB_OUT_F32 ? 13 : 10; }

struct ExpertsAt {
    size_t x, h, h_rows, part, bytes;
};
static ExpertsAt experts_at(int64_t T, int k, int64_t hidden, int64_t ffn, int type) {
    ExpertsAt a;
    const size_t pairs = (size_t)T * k;
    a.x = 0;
    a.h = a.x + rows_bytes(pairs, hidden, type);
    a.h_rows = a.h + align256(pairs * ffn * 4);
    a.part = a.h_rows + rows_bytes(pairs, ffn, type);
    a.bytes = a.part + align256(pairs * hidden * 4) + 256;
    return a;
}

}  // namespace lb

LB_EXPORT int lb_gemv_q4(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros_opt, int group,
                         const void *x, int type, int64_t x_stride, void *y, int64_t y_stride, int64_t N,
                         int64_t K, int B, void *stream) {
    using namespace lb;
    if (int e = check_product(codes, scales, zeros_opt, group, x, type, x_stride, y, y_stride, 1, N, K)) return e;
    if (B < 1 || B > 8) return LB_ERR_BATCH;
    DeviceInfo di;
    if (int e = current_device_info(&di)) return e;
    const Q4Params p = product_of(scales, zeros_opt, group, x, x_stride, y, y_stride, B, N, K);
    if (!p.error) return LB_ERR_LAUNCH;
    return q4_gemv(p, kQ4Dense, type, codes, N, di.sms, as_stream(stream));
}

LB_EXPORT size_t lb_gemm_q4_workspace_bytes(int64_t M, int64_t N, int64_t K, int type) {
    using namespace lb;
    if (M < 0 || M > (1 << 20) || N < 1 || N > (1 << 23) || K < 32 || K > LB_Q4_MAX_K || !q4_type_ok(type))
        return 0;
    return M <= 8 ? 256 : 256 + rows_bytes(M, K, type);
}

LB_EXPORT int lb_gemm_q4(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros_opt, int group,
                         const void *x, int type, int64_t x_stride, void *y, int64_t y_stride, int64_t M,
                         int64_t N, int64_t K, void *workspace, size_t workspace_bytes, void *stream) {
    using namespace lb;
    if (!workspace) return LB_ERR_NULL;
    if (int e = check_product(codes, scales, zeros_opt, group, x, type, x_stride, y, y_stride, M, N, K)) return e;
    if (!aligned16(workspace)) return LB_ERR_ALIGN;
    if (workspace_bytes < lb_gemm_q4_workspace_bytes(M, N, K, type)) return LB_ERR_SHAPE;
    DeviceInfo di;
    if (int e = current_device_info(&di)) return e;
    if (M == 0) return LB_OK;
    const Q4Params p = product_of(scales, zeros_opt, group, x, x_stride, y, y_stride, M, N, K);
    if (!p.error) return LB_ERR_LAUNCH;
    cudaStream_t st = as_stream(stream);
    if (M <= 8) return q4_gemv(p, kQ4Dense, type, codes, N, di.sms, st);
    const RowsAt r = rows_at(static_cast<uint8_t *>(workspace), M, K, type);
    if (int e = q4_rows(x, type == LB_OUT_F32, x_stride, M, (int)K, nullptr, nullptr, 1, parts_of(type), r.to, r.scale, st))
        return e;
    return q4_gemm_dense(p, {r.to, r.scale, M}, type, codes, N, di.sms, st);
}

LB_EXPORT size_t lb_experts_q4_workspace_bytes(int64_t T, int E, int k, int64_t hidden, int64_t ffn,
                                               int type) {
    using namespace lb;
    if (T < 0 || E < 1 || E > LB_ROUTE_MAX_EXPERTS || k < 1 || k > LB_ROUTE_MAX_CHOSEN ||
        T > (1 << 24) / k || hidden < 32 || hidden > LB_Q4_MAX_K || ffn < 32 || ffn > LB_Q4_MAX_K ||
        !q4_type_ok(type))
        return 0;
    return experts_at(T, k, hidden, ffn, type).bytes;
}

LB_EXPORT int lb_experts_q4(const void *x, int type, int64_t x_stride, int64_t T, int E, int k,
                            int64_t hidden, int64_t ffn, int group, const uint8_t *up_codes,
                            const uint16_t *up_scales, const uint8_t *up_zeros_opt,
                            const uint8_t *down_codes, const uint16_t *down_scales,
                            const uint8_t *down_zeros_opt, const int32_t *ids, const float *weights,
                            const int32_t *expert_start, const int32_t *order, void *y, int64_t y_stride,
                            void *workspace, size_t workspace_bytes, void *stream) {
    using namespace lb;
    if (!up_codes || !up_scales || !down_codes || !down_scales || !expert_start || !workspace ||
        (T != 0 && (!x || !ids || !weights || !order || !y)))
        return LB_ERR_NULL;
    if (!q4_group_ok(group) || hidden % group != 0 || ffn % group != 0 || x_stride < hidden ||
        y_stride < hidden || x_stride > 0x7fffffff || y_stride > 0x7fffffff)
        return LB_ERR_SHAPE;
    const size_t need = lb_experts_q4_workspace_bytes(T, E, k, hidden, ffn, type);
    if (!need || workspace_bytes < need) return LB_ERR_SHAPE;
    const int size = type == LB_OUT_F32 ? 4 : 2;
    for (const void *q : {(const void *)x, (const void *)up_codes, (const void *)up_scales,
                          (const void *)up_zeros_opt, (const void *)down_codes, (const void *)down_scales,
                          (const void *)down_zeros_opt, (const void *)workspace})
        if (!aligned16(q)) return LB_ERR_ALIGN;
    for (const void *q : {(const void *)ids, (const void *)weights, (const void *)expert_start,
                          (const void *)order})
        if (!aligned_to(q, 4)) return LB_ERR_ALIGN;
    if (x_stride * size % 16 != 0 || !aligned_to(y, size)) return LB_ERR_ALIGN;
    DeviceInfo di;
    if (int e = current_device_info(&di)) return e;
    if (T == 0) return LB_OK;
    const int64_t pairs = T * k;
    cudaStream_t st = as_stream(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const ExpertsAt at = experts_at(T, k, hidden, ffn, type);
    float *h = reinterpret_cast<float *>(ws + at.h), *part = reinterpret_cast<float *>(ws + at.part);
    Q4Params up = product_of(up_scales, up_zeros_opt, group, x, x_stride, h, ffn, pairs, ffn, hidden);
    if (!up.error) return LB_ERR_LAUNCH;
    up.start = expert_start, up.order = order, up.E = E, up.k = k;
    Q4Params down = product_of(down_scales, down_zeros_opt, group, h, ffn, part, hidden, pairs, hidden, ffn);
    down.start = expert_start, down.order = order, down.E = E, down.k = k;
    if (pairs < (int64_t)many_pairs(type) * E) {
        if (int e = q4_gemv(up, kQ4Up, type, up_codes, E * 2 * ffn, di.sms, st)) return e;
        if (int e = q4_gemv(down, kQ4Down, type, down_codes, E * hidden, di.sms, st)) return e;
    } else {
        const RowsAt xr = rows_at(ws + at.x, pairs, hidden, type), hr = rows_at(ws + at.h_rows, pairs, ffn, type);
        const int parts = parts_of(type);
        if (int e = q4_rows(x, type == LB_OUT_F32, x_stride, pairs, (int)hidden, expert_start + E, order, k, parts, xr.to,
                            xr.scale, st))
            return e;
        if (int e = q4_gemm_experts(up, {xr.to, xr.scale, pairs}, kQ4Up, type, up_codes, E * 2 * ffn, di.sms, st)) return e;
        if (int e = q4_rows(h, true, ffn, pairs, (int)ffn, expert_start + E, nullptr, 1, parts, hr.to, hr.scale, st))
            return e;
        if (int e = q4_gemm_experts(down, {hr.to, hr.scale, pairs}, kQ4Down, type, down_codes, E * hidden, di.sms, st)) return e;
    }
    const int64_t blocks = (T * (hidden / 8) + kCombineThreads - 1) / kCombineThreads;
    if (blocks > 0x7fffffff) return LB_ERR_SHAPE;
    const dim3 grid((unsigned)blocks), block(kCombineThreads);
    if (type == LB_OUT_F32)
        return launch_pdl(experts_combine_kernel<float>, grid, block, 0, st, part, ids, weights, static_cast<float *>(y),
                          y_stride, T, k, (int)hidden);
    return launch_pdl(experts_combine_kernel<__nv_bfloat16>, grid, block, 0, st, part, ids, weights,
                      static_cast<__nv_bfloat16 *>(y), y_stride, T, k, (int)hidden);
}
