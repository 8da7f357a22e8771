// lb_q4_gemm.cu -- 4-bit products for many tokens: rows of x for the tensor cores, and the plain product
// (lb_q4_gemm.cuh has the kernel).
#include "lb_q4_gemm.cuh"

namespace lb {

// ------------------------------------------------------------------------------------------
// Rows of x for the tensor cores (with an order, row i is that of pair order[i], zeros where there is none): scaled so
// that the largest lies in [2^14, 2^15), in fp16 (one part, or two that hold 22 bits), each eight columns in the order
// 0 4 1 5 2 6 3 7.  Bound by memory.
// ------------------------------------------------------------------------------------------
constexpr int kRowThreads = 256;
constexpr int kRowHold = 8;        // groups of eight columns that a thread keeps between its two passes
// A warp takes a row, instead of four, where there are so many rows and a warp's registers hold a row: many rows keep the
// memory busy by themselves and need no barrier, few or longer ones are sooner done by more threads.  With a product of
// 128 weight rows behind them, a warp against four: 32768 x 1024 fp32 73 against 122 us, bf16 37 against 64;
// 2048 x 1024 15.1 against 18.6 and 14.4 against 16.4; 512 x 1024 14.5 both and 14.4 against 13.9; 32768 x 4096
// 290 against 263 and 136 against 134; 64 x 4096 16.5 against 14.5 and 14.5 against 12.4.
constexpr int kRowsMany = 2048;

template <typename X>
struct RawEight;   // eight numbers as they lie in memory
template <>
struct RawEight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
};
template <>
struct RawEight<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; i++)
            v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
};

// PER: threads of a row.
template <typename X, int PARTS, int PER>
__global__ void __launch_bounds__(kRowThreads)
    q4_rows_kernel(const X *x, int64_t x_stride, int64_t n, int K, const int32_t *n_opt,
                   const int32_t *order, int k, uint16_t *to, float *row_scale) {
    __shared__ float most[kRowThreads / 32];
    const int tid = threadIdx.x % PER;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = blockIdx.x * (int64_t)(kRowThreads / PER) + threadIdx.x / PER;
    const int64_t end = n_opt ? min(max(*n_opt, 0), (int)n) : n;
    int64_t from = row < end ? row : -1;
    if (order && from >= 0) {
        const int pair = order[row];
        from = pair >= 0 && pair < n ? pair / k : -1;
    }
    const X *src = x + max(from, (int64_t)0) * x_stride;
    const int units = K / 8;
    RawEight<X> held[kRowHold];
    float m = 0.f;
    auto look = [&](const RawEight<X> &r) {
        float v[8];
        r.get(v);
#pragma unroll
        for (int j = 0; j < 8; j++) m = fmaxf(m, fabsf(v[j]));
    };
    if (from >= 0) {
#pragma unroll
        for (int h = 0; h < kRowHold; h++)
            if (tid + h * PER < units) held[h].load(src + 8 * (tid + h * PER));
#pragma unroll
        for (int h = 0; h < kRowHold; h++)
            if (tid + h * PER < units) look(held[h]);
        for (int u = tid + kRowHold * PER; u < units; u += PER) {
            RawEight<X> r;
            r.load(src + 8 * u);
            look(r);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (PER > 32) {
        if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
        __syncthreads();
        const float *mine = most + threadIdx.x / PER * (PER / 32);
        m = mine[0];
#pragma unroll
        for (int w = 1; w < PER / 32; w++) m = fmaxf(m, mine[w]);
    }
    if (row >= end) return;
    const uint32_t e = q4_power(__float_as_uint(m));
    const float up = __uint_as_float(e << 23);
    if (tid == 0) row_scale[row] = __uint_as_float((254 - e) << 23);
    auto put = [&](int u, const RawEight<X> &r) {
        float v[8];
        r.get(v);
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
    for (int h = 0; h < kRowHold; h++)
        if (tid + h * PER < units) put(tid + h * PER, held[h]);
    for (int u = tid + kRowHold * PER; u < units; u += PER) {
        RawEight<X> r;
        r.load(src + 8 * u);
        put(u, r);
    }
}

template <typename X, int PARTS>
static int launch_rows(const X *x, int64_t x_stride, int64_t n, int K, const int32_t *n_opt, const int32_t *order, int k,
                       uint16_t *to, float *row_scale, cudaStream_t st) {
    const int per = n >= kRowsMany && K <= 32 * 8 * kRowHold ? 32 : 128, rows = kRowThreads / per;
    auto kernel = per == 32 ? q4_rows_kernel<X, PARTS, 32> : q4_rows_kernel<X, PARTS, 128>;
    return launch_pdl(kernel, dim3((unsigned)((n + rows - 1) / rows)), dim3(kRowThreads), 0, st, x, x_stride, n, K, n_opt,
                      order, k, to, row_scale);
}

int q4_rows(const void *x, bool f32, int64_t x_stride, int64_t n, int K, const int32_t *n_opt,
            const int32_t *order, int k, int parts, uint16_t *to, float *row_scale, cudaStream_t st) {
    if (!f32)
        return launch_rows<__nv_bfloat16, 1>(static_cast<const __nv_bfloat16 *>(x), x_stride, n, K, n_opt, order, k, to,
                                             row_scale, st);
    const float *v = static_cast<const float *>(x);
    return parts == 2 ? launch_rows<float, 2>(v, x_stride, n, K, n_opt, order, k, to, row_scale, st)
                      : launch_rows<float, 1>(v, x_stride, n, K, n_opt, order, k, to, row_scale, st);
}

// About the clocks that a call takes with items of so many tokens: rounds of items, each so many clocks a step, and what
// one accumulator cannot hide behind the next item's products, or sums of a cluster cost.
static int64_t gemm_clocks(const Q4Params &p, int tokens, int sms) {
    const int64_t tiles = (p.N + kGmRows - 1) / kGmRows, pieces = (p.T + tokens - 1) / tokens;
    int64_t steps = (p.K + kGmStep - 1) / kGmStep, rounds = 1, sums = 0;
    if (tiles * pieces * 2 <= sms) {
        const int64_t split = std::min<int64_t>({sms / (tiles * pieces), kGmMaxSplit, std::max<int64_t>(steps / 4, 1)});
        steps = (steps + split - 1) / split;
        sums = split > 1 ? 5000 : 0;
    } else {
        rounds = (pieces * tiles + sms - 1) / sms;
    }
    return rounds * (tokens == 128 ? 450 * steps : tokens == 176 ? 490 * steps : 520 * steps + 8000) + sums;
}

int q4_gemm_dense(const Q4Params &p, const Q4Rows &r, int type, const uint8_t *codes, int64_t rows, int sms,
                  cudaStream_t st) {
    if (type == LB_OUT_F32) return dispatch_gemm<kQ4Dense, float, 128>(p, r, codes, rows, sms, st);
    // Items of 256 tokens and one accumulator, or of 176 or 128 and two in turn: large ones expand weights less often, two
    // accumulators hide what happens behind the last product, and items come in rounds.  us with 128, 176 and 256: 4096 x
    // 12288 x 4096 309, 264, 255; 2048 x 4096 with K = 2816 49, 43, 40, with 768 21, 20, 21; 500 x 4096 with K = 2048 16.4,
    // 16.5, 22.6.
    const int64_t t128 = gemm_clocks(p, 128, sms), t176 = gemm_clocks(p, 176, sms), t256 = gemm_clocks(p, 256, sms);
    if (t256 < t128 && t256 < t176) return dispatch_gemm<kQ4Dense, __nv_bfloat16, 256>(p, r, codes, rows, sms, st);
    if (t176 < t128) return dispatch_gemm<kQ4Dense, __nv_bfloat16, 176>(p, r, codes, rows, sms, st);
    return dispatch_gemm<kQ4Dense, __nv_bfloat16, 128>(p, r, codes, rows, sms, st);
}

}  // namespace lb
