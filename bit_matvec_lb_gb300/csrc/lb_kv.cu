// lb_kv.cu -- page plan of a serving step, and the write and read-back of the 4-bit key/value
// cache.
#include "lb_kv4.cuh"

namespace lb {

// ------------------------------------------------------------------------------------------
// Page plan: two prefix sums over the requests (new tokens, new pages), then one independent
// lookup per token.  Every CTA computes both sums over all requests itself (8 B per request from
// L2, at most 64 KB) instead of a second launch that would have to wait for them: the step is one
// launch, bound by its latency (8 requests 2.3 us, 512 with prompts among them 5.7 us).
// ------------------------------------------------------------------------------------------
struct PlanParams {
    const int32_t *past, *fresh, *free_pages, *free_from;
    int32_t *table, *q_start, *kv_len, *position, *counts;
    int64_t *slot;
    int64_t width, T, n_free;
    int R, shift;
};

constexpr int kPlanThreads = 256;
constexpr int kPlanTokens = 1024;  // tokens per CTA and turn

__device__ __forceinline__ int clamp_len(int n) { return n < 0 ? 0 : n; }

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const PlanParams p) {
    extern __shared__ int32_t sm[];
    int32_t *tok = sm;                 // [R + 1] new tokens before request r
    int32_t *pg = sm + p.R + 1;        // [R + 1] new pages before request r
    __shared__ int32_t wsum[2][kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int mask = (1 << p.shift) - 1;
    pdl_wait();
    pdl_launch_dependents();
    for (int r = tid; r < p.R; r += kPlanThreads) {
        const int past = clamp_len(p.past[r]), fresh = clamp_len(p.fresh[r]);
        tok[r] = fresh;
        pg[r] = (int)(((int64_t)past + fresh + mask) >> p.shift) -
                (int)(((int64_t)past + mask) >> p.shift);
        if (r % gridDim.x == blockIdx.x) p.kv_len[r] = past + fresh;
    }
    const int from = p.free_from ? *p.free_from : 0;
    __syncthreads();
    // Exclusive sums: each thread sums its run of requests, the runs are scanned over the CTA.
    const int run = (p.R + kPlanThreads - 1) / kPlanThreads;
    const int r0 = min(tid * run, p.R), r1 = min(r0 + run, p.R);
    int st = 0, sp = 0;
    for (int r = r0; r < r1; r++) st += tok[r], sp += pg[r];
    int it = st, ip = sp;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, it, o), b = __shfl_up_sync(0xffffffffu, ip, o);
        if (lane >= o) it += a, ip += b;
    }
    if (lane == 31) wsum[0][warp] = it, wsum[1][warp] = ip;
    __syncthreads();
    int bt = it - st, bp = ip - sp, total_t = 0, total_p = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; w++) {
        if (w < warp) bt += wsum[0][w], bp += wsum[1][w];
        total_t += wsum[0][w], total_p += wsum[1][w];
    }
    for (int r = r0; r < r1; r++) {
        const int a = tok[r], b = pg[r];
        tok[r] = bt, pg[r] = bp;
        bt += a, bp += b;
    }
    if (tid == 0) tok[p.R] = total_t, pg[p.R] = total_p;
    __syncthreads();

    for (int r = blockIdx.x * kPlanThreads + tid; r <= p.R; r += gridDim.x * kPlanThreads)
        p.q_start[r] = tok[r];
    if (blockIdx.x == 0 && tid == 0) p.counts[0] = total_t, p.counts[1] = from + total_p;

    // Page of column `col` of request r: an old entry of the table, or a free page.
    auto new_page = [&](int r, int64_t i) -> int {
        const int64_t at = (int64_t)from + pg[r] + i;
        return at >= 0 && at < p.n_free ? p.free_pages[at] : -1;
    };
    // New table entries: a warp per request.
    for (int r = blockIdx.x * (kPlanThreads / 32) + warp; r < p.R;
         r += gridDim.x * (kPlanThreads / 32)) {
        const int take = pg[r + 1] - pg[r];
        if (take <= 0) continue;
        const int64_t have = ((int64_t)clamp_len(p.past[r]) + mask) >> p.shift;
        for (int i = lane; i < take; i += 32)
            if (have + i < p.width) p.table[r * p.width + have + i] = new_page(r, i);
    }
    // Tokens: the request by bisection of tok[], the page as above (never through the entries
    // this launch writes).
    for (int64_t t = (int64_t)blockIdx.x * kPlanThreads + tid; t < p.T;
         t += (int64_t)gridDim.x * kPlanThreads) {
        int position = -1;
        int64_t slot = -1;
        if (t < total_t) {
            int lo = 0, hi = p.R - 1;  // the last r with tok[r] <= t (an idle request owns none)
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (tok[mid] <= t) lo = mid;
                else hi = mid - 1;
            }
            const int past = clamp_len(p.past[lo]);
            position = past + (int)(t - tok[lo]);
            const int64_t col = position >> p.shift, have = ((int64_t)past + mask) >> p.shift;
            int page = -1;
            if (col >= 0 && col < p.width)
                page = col < have ? p.table[lo * p.width + col] : new_page(lo, col - have);
            if (page >= 0) slot = ((int64_t)page << p.shift) + (position & mask);
        }
        p.position[t] = position;
        p.slot[t] = slot;
    }
}

// ------------------------------------------------------------------------------------------
// Append and read-back: one row (a token's key or value of one head) per D / 16 lanes, two times 8
// values a lane (of the row's halves), so a row is read once with 16-byte loads, its extremes meet in
// log2(D / 16) shuffles, and a lane's codes are two 4-byte stores.  The bytes allow about 7 us for the
// append of 8191 tokens of 8 heads x 128 in bf16; what bounds it is issue, so values become whole
// numbers and back by additions to 2^23 and 1.5 * 2^23, whose last place is 1, not by conversions (a
// quarter of the rate), and a row's fixed work is shared by 16 values of a lane: append + read-back
// 20.8 us; with 8 values a lane 30.4, with four rows per thread (fewer threads on an SM) 37.5.
// ------------------------------------------------------------------------------------------
struct KvParams {
    const void *k, *v;
    void *k_out, *v_out;
    const int64_t *slot;
    uint8_t *cache;
    int64_t k_stride, v_stride, T, slots;
    int kv_heads, shift, tokens;  // tokens of a CTA
    uint32_t per_inverse;         // ceil(2^32 / (2 kv_heads)): rows of a CTA over rows of a token
};

constexpr int kKvThreads = 256;

// Where a row lies: its token, head and tensor, and its slot (-1 for a row past the end).
template <int D>
struct KvRow {
    int64_t t, slot;
    int h, is_v;
    bool there;

    __device__ __forceinline__ KvRow(const KvParams &p, int row) {
        // (exact while row * 2 kv_heads < 2^32)
        const int tl = (int)__umulhi((uint32_t)row, p.per_inverse), i = row - tl * 2 * p.kv_heads;
        t = (int64_t)blockIdx.x * p.tokens + tl;
        there = tl < p.tokens && t < p.T;
        is_v = i >= p.kv_heads;
        h = i - is_v * p.kv_heads;
        slot = there ? p.slot[t] : -1;
    }
    __device__ __forceinline__ bool stored(const KvParams &p) const {
        return slot >= 0 && slot < p.slots;
    }
    __device__ __forceinline__ void find(const KvParams &p, uint8_t *&codes, uint8_t *&pair) const {
        const int in_page = (int)(slot & ((1 << p.shift) - 1));
        uint8_t *chunk = p.cache + kv4_chunk_offset(slot >> p.shift, h, in_page, p.kv_heads, p.shift, D);
        codes = chunk + is_v * kv4_codes_bytes(D) + (in_page & 15) * (D / 2);
        pair = chunk + 2 * kv4_codes_bytes(D) + is_v * kKv4PairBytes + (in_page & 15) * 4;
    }
};

template <int D, typename T>
__global__ void __launch_bounds__(kKvThreads) kv4_append_kernel(const KvParams p) {
    constexpr int L = D / 16, STEP = kKvThreads / L;  // lanes of a row, rows of a CTA at a time
    const int sub = threadIdx.x % L;
    pdl_wait();
    pdl_launch_dependents();
    const int rows = 2 * p.kv_heads * p.tokens;
    for (int row0 = 0; row0 < rows; row0 += STEP) {
        const KvRow<D> r(p, row0 + threadIdx.x / L);
        float x[2][8] = {};
        if (r.there) {
            const T *src = static_cast<const T *>(r.is_v ? p.v : p.k) +
                           r.t * (r.is_v ? p.v_stride : p.k_stride) + r.h * D + sub * 8;
            load8(src, x[0]);
            load8(src + D / 2, x[1]);
        }
        float2 m = make_float2(0.f, 0.f);  // {-lowest, highest}, 0 among them
#pragma unroll
        for (int e = 0; e < 16; e++) m.x = fmaxf(m.x, -x[e / 8][e % 8]), m.y = fmaxf(m.y, x[e / 8][e % 8]);
        if (sizeof(T) == 2) {  // bf16 extremes are bf16: both in one word
            __nv_bfloat162 w = __floats2bfloat162_rn(m.x, m.y);
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<uint32_t *>(&w), o);
                w = __hmax2(w, *reinterpret_cast<const __nv_bfloat162 *>(&other));
            }
            m = __bfloat1622float2(w);
        } else {
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) {
                m.x = fmaxf(m.x, __shfl_xor_sync(0xffffffffu, m.x, o));
                m.y = fmaxf(m.y, __shfl_xor_sync(0xffffffffu, m.y, o));
            }
        }
        if (!r.stored(p)) continue;
        const __half d = __float2half_rn(fminf(__fdiv_rn(__fadd_rn(m.y, m.x), 15.f), 65504.f));
        const float df = __half2float(d);
        const float id = df > 0.f ? __frcp_rn(df) : 0.f;
        // round-half-even by adding 1.5 * 2^23; values are clamped at whole numbers before
        constexpr float kRound = 12582912.f;
        const float z = fminf(__fadd_rn(__fadd_rn(fminf(__fmul_rn(m.x, id), 64.f), kRound), -kRound), 15.f);
        uint8_t *codes, *pair;
        r.find(p, codes, pair);
#pragma unroll
        for (int half = 0; half < 2; half++) {
            uint32_t c[8];
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float y = fminf(fmaxf(__fmul_rn(x[half][e], id), -z), 15.f - z);
                c[e] = __float_as_uint(__fadd_rn(__fadd_rn(y, kRound), z));  // the last byte is the code
            }
            const uint32_t even = prmt(prmt(c[0], c[2], 0x0040), prmt(c[4], c[6], 0x0040), 0x5410);
            const uint32_t odd = prmt(prmt(c[1], c[3], 0x0040), prmt(c[5], c[7], 0x0040), 0x5410);
            reinterpret_cast<uint32_t *>(codes)[half * L + sub] = even | odd << 4;
        }
        if (sub == 0) *reinterpret_cast<__half2 *>(pair) = __halves2half2(d, __float2half_rn(z));
    }
}

template <int D, typename T>
__global__ void __launch_bounds__(kKvThreads) kv4_dequant_kernel(const KvParams p) {
    constexpr int L = D / 16, STEP = kKvThreads / L;
    const int sub = threadIdx.x % L;
    pdl_wait();
    pdl_launch_dependents();
    const int rows = 2 * p.kv_heads * p.tokens;
    for (int row0 = threadIdx.x / L; row0 < rows; row0 += STEP) {
        const KvRow<D> r(p, row0);
        if (!r.there) continue;
        uint32_t w[2] = {0, 0};
        float d = 0.f, z = 8388608.f;
        if (r.stored(p)) {
            uint8_t *codes, *pair;
            r.find(p, codes, pair);
            w[0] = reinterpret_cast<const uint32_t *>(codes)[sub];
            w[1] = reinterpret_cast<const uint32_t *>(codes)[L + sub];
            const __half2 dz = *reinterpret_cast<const __half2 *>(pair);
            d = __low2float(dz), z += __high2float(dz);
        }
        T *dst = static_cast<T *>(r.is_v ? p.v_out : p.k_out) + (r.t * p.kv_heads + r.h) * D + sub * 8;
#pragma unroll
        for (int half = 0; half < 2; half++) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; e++)  // 2^23 + c, less 2^23 + z
                x[e] = __fmul_rn(d, __uint_as_float(0x4B000000u | ((w[half] >> (4 * e)) & 15)) - z);
            store8(dst + half * (D / 2), x);
        }
    }
}

template <int D, typename T>
static int launch_kv(bool append, KvParams p, cudaStream_t st) {
    // Tokens of a CTA: as many as give each thread one row.
    p.tokens = kKvThreads / (D / 16) / (2 * p.kv_heads);
    if (p.tokens < 1) p.tokens = 1;
    p.per_inverse = (uint32_t)(((uint64_t(1) << 32) + 2 * p.kv_heads - 1) / (2 * p.kv_heads));
    const dim3 grid((unsigned)((p.T + p.tokens - 1) / p.tokens));
    return append ? launch_pdl(kv4_append_kernel<D, T>, grid, dim3(kKvThreads), 0, st, p)
                  : launch_pdl(kv4_dequant_kernel<D, T>, grid, dim3(kKvThreads), 0, st, p);
}

static int dispatch_kv(bool append, int D, int type, const KvParams &p, cudaStream_t st) {
    DeviceInfo di;
    if (int e = current_device_info(&di)) return e;
    if (p.T == 0) return LB_OK;
    if (type == LB_OUT_F32)
        return D == 64 ? launch_kv<64, float>(append, p, st) : launch_kv<128, float>(append, p, st);
    return D == 64 ? launch_kv<64, __nv_bfloat16>(append, p, st)
                   : launch_kv<128, __nv_bfloat16>(append, p, st);
}

}  // namespace lb

LB_EXPORT int lb_kv_plan(const int32_t *past, const int32_t *fresh, int64_t R,
                         const int32_t *free_pages, int64_t n_free, const int32_t *free_from_opt,
                         int page_size, int32_t *block_table, int64_t table_width, int64_t T,
                         int32_t *q_start, int32_t *kv_len, int32_t *position, int64_t *slot,
                         int32_t *counts, void *stream) {
    using namespace lb;
    const int64_t lim = int64_t(1) << 31;
    if (!past || !fresh || !block_table || !q_start || !kv_len || !counts) return LB_ERR_NULL;
    if ((n_free > 0 && !free_pages) || (T > 0 && (!position || !slot))) return LB_ERR_NULL;
    for (const void *q : {(const void *)past, (const void *)fresh, (const void *)free_pages,
                          (const void *)free_from_opt, (const void *)block_table,
                          (const void *)q_start, (const void *)kv_len, (const void *)position,
                          (const void *)counts})
        if (!aligned_to(q, 4)) return LB_ERR_ALIGN;
    if (!aligned_to(slot, 8)) return LB_ERR_ALIGN;
    const int shift = page_shift_of(page_size);
    if (shift < 0 || R < 1 || R > LB_KV_MAX_REQUESTS || n_free < 0 || n_free >= lim || T < 0 ||
        T >= lim || table_width < 1 || table_width >= lim || free_from_opt == counts ||
        free_from_opt == counts + 1)
        return LB_ERR_SHAPE;
    DeviceInfo di;
    if (int e = current_device_info(&di)) return e;
    // The lengths and the free list are read by every CTA, at any time: none of them may be an output.
    struct {
        const void *p;
        size_t bytes;
    } const in[] = {{past, (size_t)R * 4}, {fresh, (size_t)R * 4}, {free_pages, (size_t)n_free * 4},
                    {free_from_opt, 4}},
      written[] = {{block_table, (size_t)R * table_width * 4}, {q_start, (size_t)(R + 1) * 4},
                   {kv_len, (size_t)R * 4}, {position, (size_t)T * 4}, {slot, (size_t)T * 8}, {counts, 8}};
    for (const auto &a : in)
        for (const auto &b : written)
            if (overlap(a.p, a.bytes, b.p, b.bytes)) return LB_ERR_SHAPE;
    const PlanParams p{past,    fresh,  free_pages, free_from_opt, block_table, q_start, kv_len,
                       position, counts, slot,       table_width,   T,           n_free, (int)R,
                       shift};
    const size_t smem = 2 * (size_t)(R + 1) * sizeof(int32_t);
    int per_sm;
    if (int e = prepare_kernel((const void *)kv_plan_kernel, kPlanThreads, smem, &per_sm)) return e;
    const int64_t want = (T + kPlanTokens - 1) / kPlanTokens, want_r = (R + 63) / 64;
    const int64_t ctas = want > want_r ? want : want_r;
    return launch_pdl(kv_plan_kernel, dim3((unsigned)(ctas < di.sms ? ctas : di.sms)),
                      dim3(kPlanThreads), smem, as_stream(stream), p);
}

LB_EXPORT int lb_kv4_append(const void *k, const void *v, int type, int64_t k_stride,
                            int64_t v_stride, const int64_t *slot, int64_t T, uint8_t *cache,
                            int64_t pages, int page_size, int kv_heads, int head_dim,
                            void *stream) {
    using namespace lb;
    if (!cache || (T != 0 && (!k || !v || !slot))) return LB_ERR_NULL;
    if (!kv4_shape_ok(pages, page_size, kv_heads, head_dim) || T < 0 || T >= (int64_t(1) << 31) ||
        (type != LB_OUT_F32 && type != LB_OUT_BF16) || k_stride < (int64_t)kv_heads * head_dim ||
        v_stride < (int64_t)kv_heads * head_dim)
        return LB_ERR_SHAPE;
    const int64_t per16 = type == LB_OUT_F32 ? 4 : 8;
    if (!aligned16(k) || !aligned16(v) || !aligned16(cache) || !aligned_to(slot, 8) ||
        k_stride % per16 || v_stride % per16)
        return LB_ERR_ALIGN;
    KvParams p{};
    p.k = k, p.v = v, p.slot = slot, p.cache = cache, p.k_stride = k_stride, p.v_stride = v_stride;
    p.T = T, p.slots = pages * page_size, p.kv_heads = kv_heads;
    p.shift = page_shift_of(page_size);
    return dispatch_kv(true, head_dim, type, p, as_stream(stream));
}

LB_EXPORT int lb_dequantize_kv4(const uint8_t *cache, int64_t pages, int page_size, int kv_heads,
                                int head_dim, const int64_t *slot, int64_t T, int out_format,
                                void *k, void *v, void *stream) {
    using namespace lb;
    if (!cache || (T != 0 && (!k || !v || !slot))) return LB_ERR_NULL;
    if (!kv4_shape_ok(pages, page_size, kv_heads, head_dim) || T < 0 || T >= (int64_t(1) << 31) ||
        (out_format != LB_OUT_F32 && out_format != LB_OUT_BF16))
        return LB_ERR_SHAPE;
    if (!aligned16(k) || !aligned16(v) || !aligned16(cache) || !aligned_to(slot, 8))
        return LB_ERR_ALIGN;
    KvParams p{};
    p.k_out = k, p.v_out = v, p.slot = slot, p.cache = const_cast<uint8_t *>(cache);
    p.T = T, p.slots = pages * page_size, p.kv_heads = kv_heads;
    p.shift = page_shift_of(page_size);
    return dispatch_kv(false, head_dim, out_format, p, as_stream(stream));
}
