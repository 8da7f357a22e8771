// lb_q4_gemm.cu -- 4-bit products for many tokens: rows of x for the tensor cores, and the plain product
// (lb_q4_gemm.cuh has the kernel).
#include "lb_q4_gemm.cuh"

namespace lb {

// ------------------------------------------------------------------------------------------
// Rows of x for the tensor cores (with an order, row i is that of pair order[i], zeros where there is none;
// four-row gathering copies of the tensors' own rows take four times as long as the products): scaled so that the largest lies in [2^14, 2^15), in fp16 (one part, or two
// that hold 22 bits), each eight columns in the order 0 4 1 5 2 6 3 7.
// ------------------------------------------------------------------------------------------
constexpr int kRowThreads = 128;
constexpr int kRowHold = 4;   // groups of eight columns that a thread keeps between its two passes

template <typename X, int PARTS>
__global__ void __launch_bounds__(kRowThreads)
    q4_rows_kernel(const X *x, int64_t x_stride, int64_t n, int K, const int32_t *n_opt,
                   const int32_t *order, int k, uint16_t *to, float *row_scale) {
    __shared__ float most[kRowThreads / 32];
    const int tid = threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = blockIdx.x;
    if (n_opt && row >= min(max(*n_opt, 0), (int)n)) return;
    int64_t from = row;
    if (order) {
        const int pair = order[row];
        from = pair >= 0 && pair < n ? pair / k : -1;
    }
    const X *src = x + max(from, (int64_t)0) * x_stride;
    const int units = K / 8;
    float held[kRowHold][8], m = 0.f;
#pragma unroll
    for (int h = 0; h < kRowHold; h++) {
        const int u = tid + h * kRowThreads;
        if (u >= units) break;
        load8(src + 8 * u, held[h]);
#pragma unroll
        for (int j = 0; j < 8; j++) m = fmaxf(m, fabsf(held[h][j]));
    }
    for (int u = tid + kRowHold * kRowThreads; u < units; u += kRowThreads) {
        float v[8];
        load8(src + 8 * u, v);
#pragma unroll
        for (int j = 0; j < 8; j++) m = fmaxf(m, fabsf(v[j]));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((tid & 31) == 0) most[tid >> 5] = m;
    __syncthreads();
    m = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
    const uint32_t e = q4_power(__float_as_uint(m));
    const float up = __uint_as_float(e << 23);
    if (tid == 0) row_scale[row] = __uint_as_float((254 - e) << 23);
    auto put = [&](int u, const float (&v)[8]) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float a = from < 0 ? 0.f : v[j] * up, b = from < 0 ? 0.f : v[j + 4] * up;
            const __half2 h = __floats2half2_rn(a, b);
            hi[j] = bits_of(h);
            if (PARTS == 2) lo[j] = bits_of(__floats2half2_rn(a - __low2float(h), b - __high2float(h)));
        }
        uint16_t *dst = to + row * K + 8 * u;
        *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if (PARTS == 2) *reinterpret_cast<uint4 *>(dst + n * K) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    };
#pragma unroll
    for (int h = 0; h < kRowHold; h++) {
        const int u = tid + h * kRowThreads;
        if (u >= units) break;
        put(u, held[h]);
    }
    for (int u = tid + kRowHold * kRowThreads; u < units; u += kRowThreads) {
        float v[8];
        load8(src + 8 * u, v);
        put(u, v);
    }
}

int q4_rows(const void *x, bool f32, int64_t x_stride, int64_t n, int K, const int32_t *n_opt,
            const int32_t *order, int k, int parts, uint16_t *to, float *row_scale, cudaStream_t st) {
    const dim3 grid((unsigned)n), block(kRowThreads);
    if (f32) {
        auto kernel = parts == 2 ? q4_rows_kernel<float, 2> : q4_rows_kernel<float, 1>;
        return launch_pdl(kernel, grid, block, 0, st, static_cast<const float *>(x), x_stride, n, K, n_opt, order,
                          k, to, row_scale);
    }
    return launch_pdl(q4_rows_kernel<__nv_bfloat16, 1>, grid, block, 0, st,
                      static_cast<const __nv_bfloat16 *>(x), x_stride, n, K, n_opt, order, k, to,
                      row_scale);
}

int q4_gemm_dense(const Q4Params &p, const Q4Rows &r, int type, const uint8_t *codes, int64_t rows, int sms,
                  cudaStream_t st) {
    if (type == LB_OUT_F32) return dispatch_gemm<kQ4Dense, float, 128>(p, r, codes, rows, sms, st);
    // 256 tokens and one accumulator, or 128 and two in turn: the first expands weights half as often, the second
    // hides what happens behind the last product, which a short K does not.
    if (p.K >= kGmLongK) return dispatch_gemm<kQ4Dense, __nv_bfloat16, 256>(p, r, codes, rows, sms, st);
    return dispatch_gemm<kQ4Dense, __nv_bfloat16, 128>(p, r, codes, rows, sms, st);
}

}  // namespace lb
