// lb_attn_tc.cu -- attention over the paged 4-bit key/value cache for requests with many query rows
// (prompts, chunks of them) on the 5th-generation tensor cores.
#include "lb_attn.cuh"
#include "lb_tc.cuh"

namespace lb {

// ------------------------------------------------------------------------------------------
// Mathematics.  A key/value head's rows (queries x heads of the group, packed) times 64 keys at a
// time: S = Q K'^T and O += P V', K' and V' the codes less their zero, whole numbers in -15..15 and
// exact in fp16.  The keys' scales act on the scores, x = S kd_t a_r - R_r in powers of two (a_r
// holds the row's own power of two, scale and log2 e), the values' scales on the weights,
// P = 2^x vd_t, which enter the second product as fp16 bounded by the reference R_r (see below).
// fp32 tensors take two fp16 parts of Q and of P: each product twice.
//
// One CTA per SM, 14 warps: two times four for the softmax of two tiles of 128 rows (a thread per
// row), four that turn codes into fp16 operands, one that issues the tensor-core operations and
// one that copies cache chunks in.  Tensor memory holds S twice for each row tile (4 x 64 columns)
// and O (2 x 128); P overwrites S.  The operations are issued QK0(j+1) PV0(j) QK1(j+1) PV1(j), so a
// row tile's next scores are there when it is done with the present ones (128 keys and S once: 0.72
// against 0.66 ms for a bf16 prompt of 8192 tokens with 32 / 8 heads; now 0.67, 825 TFLOP/s).  What
// bounds it are the products and their hand-overs: 0.57 ms are left without softmax and expansion of
// the codes.
// Score products read both operands from shared memory, 72 cycles for 128 x 64 x 16 where the
// multiplications take 32 and one with its first operand in tensor memory 42.
//
// One pass over the scores: the reference is the first tile's largest weight, value scale and all
// (the largest score and the largest scale taken apart may be different keys', and weights pushed down
// by a scale that has no part in the row lose bits), and moves only when it must, when the weights of
// 32 keys could leave fp16's range by their sum and the tile's largest scale.  Then those 32 scores
// are read again for their largest weight, and if that is above the reference, what is already there
// under the old one (the tile's earlier weights, O and the sum) is scaled by a power of two.  (With
// the two maxima taken apart: 0.660 instead of 0.667 ms, but 4e-5 and more in norm with fp32 tensors
// where a key without weight has values 2^14 times the others'; now 3e-7.)
//
// The tensor cores cut, downwards, what lies below an accumulator's last place, once for every 16
// keys and part: over a long item that is far more than fp32 rounding.  With fp32 tensors O
// therefore holds kFlush tiles at most, is then added to a sum in memory (atomics without a return
// value, which nobody waits for; only one thread adds to an address, so the order is fixed) and
// begins anew.  3 x 1021 queries after 1300 to 3800 tokens, error in norm and time: never 2.6e-6
// and 178 us, every 8 tiles 1.0e-6 and 190, 6 0.9e-6 and 194 (197 with later changes), 4 0.8e-6 and 201.
//
// Work is split into equal runs of key tiles over the CTAs, parts of
// an item that several CTAs share are joined by a second kernel.
// ------------------------------------------------------------------------------------------
constexpr int kKeys = 64;            // keys per tile (four chunks, one copy stage)
constexpr int kRows = 128;           // query rows per tile, two tiles per item
constexpr int kPieces = 3;           // copy stages
constexpr int kScales = 8;           // tiles of scales kept
constexpr int kTcThreads = 448;
// An item's queries and outputs take about as long as 6 tiles.  A prompt of 2048 / 8192 tokens, us:
// 128 dimensions bf16 79 / 663 (counted as 3: 90 / 837, as 12: 83 / 685), fp32 115 / 1049 (139 /
// 1353, 120 / 1079); 64 dimensions bf16 69 / 640 (70 / 670, 73 / 663), fp32 90 / 865 (97 / 926, 95 / 898).
constexpr int kItemCost = 6;
constexpr int kTcMaxCtas = 160;
constexpr int kTcWhole = 8;          // items of at most this many tiles are never split
                                     // (8 x 64 queries, 364 keys: 20 us, split 29)
constexpr int kTcMinRun = kItemCost + 1;
constexpr int kFlush = 6;            // fp32: tiles between two additions to the sums in memory
constexpr float kTcLift = 16.f;      // weights at the reference: 2^4
constexpr float kTcMost = 60000.f;   // largest weight a tile may hold

template <int D, int SPLIT>
struct Prompt {
    static constexpr int kBuf = 4 / SPLIT;             // fp16 key and value tiles
    static constexpr int kQ = kRows * D * 2;           // bytes of one part of one row tile
    static constexpr int kTileB = kKeys * D * 2;
    static constexpr int kRaw = kKeys / 16 * kv4_chunk_bytes(D);
    static constexpr int oQ = 0;                       // [2 tiles][SPLIT]
    static constexpr int oK = oQ + 2 * SPLIT * kQ;     // [kBuf]
    static constexpr int oV = oK + kBuf * kTileB;
    static constexpr int oRaw = oV + kBuf * kTileB;    // [kPieces]
    static constexpr int oScale = oRaw + kPieces * kRaw;  // [3][kScales][kKeys] floats
    static constexpr int kSmem = oScale + kScales * 3 * kKeys * 4;
};

struct TcBars {
    uint64_t raw_full[kPieces], raw_empty[kPieces];
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
    uint64_t sc_full[kScales];
    uint64_t q_full[2], s_full[2][2], p_full[2][2], o_full[2][2];  // [row tile][key tile's parity]
};

// Shared-memory matrix descriptors (K-major, no swizzle: core matrices of 8 rows x 16 bytes, 128 B
// apart along K, SBO bytes between groups of 8 rows) are kept as their low words; a step of 16
// along K adds 256 >> 4.  Four steps go out as one statement: the issuing thread's own instructions
// would otherwise set the pace.
constexpr uint32_t desc_high(uint32_t sbo) { return ((sbo >> 4) & 0x3FFF) | 1u << 14; }
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr) {
    return ((saddr >> 4) & 0x3FFF) | (uint32_t)(128 >> 4) << 16;
}
// D[tmem] (+)= A[desc] * B[desc]^T over 64 of K.
template <uint32_t HA, uint32_t HB>
__device__ __forceinline__ void mma4_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p; .reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5}; mov.b64 b, {%2, %6};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
        "setp.eq.b32 p, 0, 0;\n\t"
        "add.s64 a, a, 16; add.s64 b, b, 16;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
        "add.s64 a, a, 16; add.s64 b, b, 16;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
        "add.s64 a, a, 16; add.s64 b, b, 16;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p; }" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(HA), "n"(HB)
        : "memory");
}
// D[tmem] (+)= A[tmem] * B[desc]^T over 64 of K; a step's 8 columns of A lie 16 columns apart.
template <uint32_t HB>
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p; .reg .b64 b; .reg .b32 a;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 b, {%2, %5}; mov.b32 a, %1;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p;\n\t"
        "setp.eq.b32 p, 0, 0;\n\t"
        "add.s32 a, a, 16; add.s64 b, b, 16;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p;\n\t"
        "add.s32 a, a, 16; add.s64 b, b, 16;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p;\n\t"
        "add.s32 a, a, 16; add.s64 b, b, 16;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p; }" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(HB)
        : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t x;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(x));
    return x != 0;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// 16 columns asked for; they are there after tmem_ld16_wait.
__device__ __forceinline__ void tmem_ld16_start(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
    return (uint64_t)__float_as_uint(a) | (uint64_t)__float_as_uint(b) << 32;
}
__device__ __forceinline__ float lo_of(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi_of(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ void pairs_of(const uint32_t (&r)[16], uint64_t (&s)[8]) {
#pragma unroll
    for (int e = 0; e < 8; e++) s[e] = (uint64_t)r[2 * e] | (uint64_t)r[2 * e + 1] << 32;
}
// A chunk's weights: 8 columns (one part) or 16.
__device__ __forceinline__ void tmem_st_weights(uint32_t taddr, const uint32_t (&r)[16]) {
    tmem_st16(taddr, r);
}
__device__ __forceinline__ void tmem_st_weights(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// A pair of -ref: what is added to a row's scores; 0 for a row that has seen nothing yet.
__device__ __forceinline__ uint64_t minus_base(float ref) {
    const float b = ref == -INFINITY ? 0.f : -ref;
    return pair_of(b, b);
}

// Rows [256 b, 256 b + 256) of a request: their visible key tiles.
struct Pair {
    int lo, hi, t0, tiles, rows;
};
__device__ __forceinline__ Pair pair_of_rows(const AttnParams &p, const Request &q, int b) {
    Pair x;
    const int total = q.n * p.group, r0 = b * 2 * kRows;
    x.rows = min(2 * kRows, total - r0);
    visible_range(p, q, r0 / p.group, (r0 + x.rows - 1) / p.group + 1, x.lo, x.hi);
    x.t0 = x.lo / kKeys;
    x.tiles = max((x.hi + kKeys - 1) / kKeys - x.t0, 1);
    return x;
}
__device__ __forceinline__ int pairs_of(const AttnParams &p, const Request &q) {
    return (q.n * p.group + 2 * kRows - 1) / (2 * kRows);
}

// A CTA's items in order; every warp walks them by itself.
struct Walk {
    Request q;
    Pair x;
    int r, b, h;            // request, pair of row tiles, head
    int64_t u, end, begin;  // next unit, end of the run, first unit of the item
    int first, last;        // this CTA's tiles of the item

    __device__ __forceinline__ void set(const AttnParams &p) {
        q = load_request(p, r);
        x = pair_of_rows(p, q, b);
    }
    // The next item this CTA takes part in; false at the end of its run.
    __device__ __forceinline__ bool next(const AttnParams &p) {
        while (u < end) {
            while (u >= begin + x.tiles + kItemCost) {
                begin += x.tiles + kItemCost;
                if (++h < p.kv_heads) continue;
                h = 0;
                if (++b >= pairs_of(p, q)) {
                    b = 0;
                    do q = load_request(p, ++r);
                    while (q.n == 0);
                }
                x = pair_of_rows(p, q, b);
            }
            const bool starts = u == begin;
            first = max((int)(u - begin) - kItemCost, 0);
            const int64_t stop = min(end, begin + x.tiles + kItemCost);
            last = max((int)(stop - begin) - kItemCost, 0);
            u = stop;
            if (x.tiles <= kTcWhole) {  // never split: the CTA in whose run it begins takes it
                first = 0, last = starts ? x.tiles : 0;
            }
            if (last > first) return true;
        }
        return false;
    }
};

template <int D, typename T, int SPLIT>
__global__ void __launch_bounds__(kTcThreads, 1) attn_prompt_kernel(const AttnParams p) {
    using C = Prompt<D, SPLIT>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ TcBars bar;
    __shared__ uint32_t s_tmem, raw_valid[kPieces], sc_valid[kScales];
    __shared__ float sc_max[kScales][4], row_a[2][kRows];
    __shared__ int64_t scan[kTcThreads / 32], s_begin;
    __shared__ int s_r, s_b, s_h;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

    if (tid == 0) {
        for (int i = 0; i < kPieces; i++) mbar_init(&bar.raw_full[i], 1), mbar_init(&bar.raw_empty[i], 4);
        for (int i = 0; i < 4; i++) {
            mbar_init(&bar.k_full[i], 4), mbar_init(&bar.k_empty[i], 1);
            mbar_init(&bar.v_full[i], 4), mbar_init(&bar.v_empty[i], 1);
            mbar_init(&bar.s_full[i >> 1][i & 1], 1), mbar_init(&bar.p_full[i >> 1][i & 1], 4);
            mbar_init(&bar.o_full[i >> 1][i & 1], 1);
        }
        mbar_init(&bar.q_full[0], 4), mbar_init(&bar.q_full[1], 4);
        for (int i = 0; i < kScales; i++) mbar_init(&bar.sc_full[i], 4);
        fence_mbar_init();
    }
    pdl_wait();

    // ---- this CTA's run of units ----
    const int run = (p.R + kTcThreads - 1) / kTcThreads;
    const int ra = min(tid * run, p.R), rb = min(ra + run, p.R);
    int64_t mine = 0;
    for (int r = ra; r < rb; r++) {
        const Request q = load_request(p, r);
        for (int b = 0, n = pairs_of(p, q); b < n; b++)
            mine += (int64_t)(pair_of_rows(p, q, b).tiles + kItemCost) * p.kv_heads;
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += a;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int64_t total = 0, before = incl - mine;
#pragma unroll
    for (int w = 0; w < kTcThreads / 32; w++) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    const int64_t ctas = min((int64_t)gridDim.x, (total + kTcMinRun - 1) / kTcMinRun);
    int4 *record = p.record + 2 * blockIdx.x;
    if (tid < 2) record[tid] = make_int4(-1, 0, 0, 0);
    if (blockIdx.x >= ctas) {
        pdl_launch_dependents();
        return;
    }
    Walk it;
    it.u = total * blockIdx.x / ctas, it.end = total * (blockIdx.x + 1) / ctas;
    if (before <= it.u && it.u < before + mine) {
        int64_t at = before;
        for (int r = ra; r < rb; r++) {
            const Request q = load_request(p, r);
            for (int b = 0, n = pairs_of(p, q); b < n; b++) {
                const int64_t t = pair_of_rows(p, q, b).tiles + kItemCost;
                if (it.u < at + t * p.kv_heads) {
                    const int h = (int)((it.u - at) / t);
                    s_r = r, s_b = b, s_h = h, s_begin = at + h * t;
                    r = rb;
                    break;
                }
                at += t * p.kv_heads;
            }
        }
    }
    // Tensor memory is taken only now, when the kernels before this one have ended, and the next
    // kernel may start only after it: neither waits for the other's columns.
    if (warp == 12) tmem_alloc(&s_tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = s_tmem;
    it.r = s_r, it.b = s_b, it.h = s_h, it.begin = s_begin;
    it.set(p);

    // Bounded: about 2 s (2000 tries of up to a millisecond), after the first that ran out a few tries.
    int tries = 2000;
    auto wait = [&](uint64_t &b, uint32_t parity) {
        int i = 0;
        while (!mbar_try_wait_hint(&b, parity & 1, 1000000u) && i < tries) i++;
        if (i >= tries) {
            *p.error = 1;
            tries = 4;
        }
        __syncwarp();
    };
    float *kd_s = reinterpret_cast<float *>(smem + C::oScale);   // [kScales][kKeys]
    float *vd_s = kd_s + kScales * kKeys, *vl_s = vd_s + kScales * kKeys;  // vl_s: powers of two
    uint32_t gt = 0;  // tiles so far, over all items

    if (warp < 8) {
        // =================== softmax: one row per thread ===================
        const int w = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // lane quarter in the address' upper half
        const uint32_t S0 = tmem + 2 * kKeys * w + lanes, O = tmem + 256 + D * w + lanes;
        uint32_t cw = 0;
        float4 *sums = p.sums + (int64_t)(2 * blockIdx.x + w) * (D / 4) * kRows + row;  // [D / 4][kRows]
        while (it.next(p)) {
            const int n = it.last - it.first;
            const int ncol = it.x.rows - w * kRows;  // rows of this tile
            if (ncol <= 0) {
                gt += n;
                continue;
            }
            const int row0 = it.b * 2 * kRows + w * kRows;
            // ---- queries: a warp's 32 rows, 8 rows x 32 dimensions per step; the loads of
            // several groups of 8 rows first ----
            constexpr int BATCH = 2;
#pragma unroll 1
            for (int g0 = 0; g0 < 4; g0 += BATCH) {
                float x[BATCH][D / 32][8];
#pragma unroll
                for (int g = 0; g < BATCH; g++) {
                    const int cc = row0 + min((warp & 3) * 32 + (g0 + g) * 8 + (lane & 7), ncol - 1);
                    const T *src = static_cast<const T *>(p.q) +
                                   (int64_t)(it.q.q0 + cc / p.group) * p.q_stride +
                                   (int64_t)(it.h * p.group + cc % p.group) * D + (lane >> 3) * 8;
#pragma unroll
                    for (int k = 0; k < D / 32; k++) load8(src + 32 * k, x[g][k]);
                }
#pragma unroll
                for (int g = 0; g < BATCH; g++) {
                    const int rr = (warp & 3) * 32 + (g0 + g) * 8 + (lane & 7);
                    float amax = 0.f;
#pragma unroll
                    for (int k = 0; k < D / 32; k++)
#pragma unroll
                        for (int e = 0; e < 8; e++) amax = fmaxf(amax, fabsf(x[g][k][e]));
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 8));
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 16));
                    float up, down;
                    row_power(amax, up, down);
                    if (lane < 8) row_a[w][rr] = p.scale * kLog2e * down;
#pragma unroll
                    for (int k = 0; k < D / 32; k++) {
                        // order 0 4 1 5 2 6 3 7, as the codes of a word unfold
                        const uint32_t at =
                            (rr >> 3) * (D * 16) + (4 * k + (lane >> 3)) * 128 + (rr & 7) * 16;
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const float a = x[g][k][e] * up, b = x[g][k][e + 4] * up;
                            const __half2 h2 = __floats2half2_rn(a, b);
                            hi[e] = *reinterpret_cast<const uint32_t *>(&h2);
                            lo[e] = half2_bits(a - __low2float(h2), b - __high2float(h2));
                        }
                        uint8_t *dst = smem + C::oQ + w * SPLIT * C::kQ + at;
                        *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        if (SPLIT == 2)
                            *reinterpret_cast<uint4 *>(dst + C::kQ) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.q_full[w]);
            const float a = row_a[w][row];
            const uint64_t a2 = pair_of(a, a);
            // Keys this row sees, and those all rows of the tile see.
            const int qi = (row0 + min(row, ncol - 1)) / p.group;
            int hi = it.x.hi, all_hi = hi;
            if (p.causal) {
                hi = min(hi, it.q.base + qi + 1);
                all_hi = min(all_hi, it.q.base + row0 / p.group + 1);
            }
            const int lo = window_start(p, it.q, qi);
            const int all_lo = window_start(p, it.q, (row0 + ncol - 1) / p.group);
            float ref = -INFINITY, l = 0.f;

            for (int j = 0; j < n; j++, gt++, cw++) {
                const int slot = gt % kScales, j0 = (it.x.t0 + it.first + j) * kKeys;
                // The scores first: a warp that had no rows in the items before counted their tiles
                // without waiting, and could take the slot's phase before last for this one.
                wait(bar.s_full[w][cw & 1], cw >> 1);
                tc_fence_after();
                wait(bar.sc_full[slot], gt / kScales);
                const uint32_t ok = sc_valid[slot], S = S0 + kKeys * (cw & 1);
                const bool inside = ok == 0xFu && j0 >= all_lo && j0 + kKeys <= all_hi;
                float vmax = 0.f;
#pragma unroll
                for (int e = 0; e < 4; e++) vmax = fmaxf(vmax, sc_max[slot][e]);
                const ulonglong2 *kd = reinterpret_cast<const ulonglong2 *>(kd_s + slot * kKeys);
                const ulonglong2 *vd = reinterpret_cast<const ulonglong2 *>(vd_s + slot * kKeys);
                const ulonglong2 *vl = vd + kScales * kKeys / 4;

                // Scores of 16 keys (c), plus more(e) for each four of them, as pairs, from the raw
                // products in s.
                auto scores = [&](int c, uint64_t (&s)[8], auto more) {
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const ulonglong2 k = kd[4 * c + e], m = more(4 * c + e);
                        s[2 * e] = fma2(mul2(s[2 * e], k.x), a2, m.x);
                        s[2 * e + 1] = fma2(mul2(s[2 * e + 1], k.y), a2, m.y);
                    }
                    if (!inside) {
                        const bool there = ok >> c & 1;
#pragma unroll
                        for (int e = 0; e < 8; e++) {
                            const int t = j0 + 16 * c + 2 * e;
                            s[e] = pair_of(there && t >= lo && t < hi ? lo_of(s[e]) : -INFINITY,
                                           there && t + 1 >= lo && t + 1 < hi ? hi_of(s[e]) : -INFINITY);
                        }
                    }
                };
                // The weights of chunk c as fp16 (and, second, what rounding took from them).
                auto weights = [&](int c, uint64_t(&s)[8], uint64_t &sum, uint32_t *ph) {
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const ulonglong2 v = vd[4 * c + e / 2];
                        const uint64_t pr = pair_of(ex2(lo_of(s[e])), ex2(hi_of(s[e])));
                        sum = add2(sum, pr);
                        const uint64_t wv = mul2(pr, e & 1 ? v.y : v.x);
                        const __half2 h2 = __floats2half2_rn(lo_of(wv), hi_of(wv));
                        ph[e] = *reinterpret_cast<const uint32_t *>(&h2);
                        if (SPLIT == 2)
                            ph[8 * (SPLIT - 1) + e] =
                                half2_bits(lo_of(wv) - __low2float(h2), hi_of(wv) - __high2float(h2));
                    }
                };
                // What is added to the scores: -ref, the value scales as powers of two (weights'
                // sizes), or both.
                uint64_t nb = 0;
                auto less = [&](int) { return make_ulonglong2(nb, nb); };
                auto sizes = [&](int e) { return vl[e]; };
                auto sizes_less = [&](int e) {
                    const ulonglong2 v = vl[e];
                    return make_ulonglong2(add2(v.x, nb), add2(v.y, nb));
                };
                auto largest = [&](const uint64_t(&s)[8], float m) {
#pragma unroll
                    for (int e = 0; e < 8; e++) m = fmaxf(m, fmaxf(lo_of(s[e]), hi_of(s[e])));
                    return m;
                };
                uint32_t r0[16], r1[16];
                tmem_ld16_start(S, r0);
                if (j == 0) {  // the first reference: this tile's largest weight
                    float m = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < 4; c++) {
                        tmem_ld16_wait(r0);
                        uint64_t s[8];
                        pairs_of(r0, s);
                        tmem_ld16_start(S + 16 * ((c + 1) & 3), r0);
                        scores(c, s, sizes);
                        m = largest(s, m);
                    }
                    ref = m;  // the last load, of chunk 0, is in flight
                }
                // A chunk's weights as fp16 (and what rounding took from them), 8 columns each, over
                // its 16 scores: P of chunk c lies at columns 16 c.
                nb = minus_base(ref);
#pragma unroll 1  // (unrolled, the instruction cache becomes the limit)
                for (int c2 = 0; c2 < kKeys / 32; c2++) {
                    uint32_t ph[2][8 * SPLIT];
                    uint64_t sum = 0;
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        const int c = 2 * c2 + k;
                        uint32_t(&r)[16] = k ? r1 : r0;
                        tmem_ld16_wait(r);
                        if (c < kKeys / 16 - 1) tmem_ld16_start(S + 16 * (c + 1), k ? r0 : r1);
                        uint64_t s[8];
                        pairs_of(r, s);
                        scores(c, s, less);
                        weights(c, s, sum, ph[k]);
                    }
                    float part = lo_of(sum) + hi_of(sum);
                    bool keep = true;  // the weights just computed
                    if (__any_sync(0xffffffffu, ref == -INFINITY || !(part * vmax <= kTcMost))) {
                        // (r0 holds the next chunk's scores, or is in flight: it stays.)
                        uint32_t t0[16];
                        uint64_t s[8];
                        float m = -INFINITY;
#pragma unroll 1
                        for (int c = 2 * c2; c < 2 * c2 + 2; c++) {
                            tmem_ld16_start(S + 16 * c, t0);
                            tmem_ld16_wait(t0);
                            pairs_of(t0, s);
                            scores(c, s, sizes_less);
                            m = largest(s, m);
                        }
                        float f = 1.f, d = 0.f;  // 2^-d, d a whole number
                        if (ref == -INFINITY) {
                            if (m > -INFINITY) d = ref = m;  // nothing is there to scale
                        } else if (m > 0.f) {
                            d = ceilf(m), ref += d;
                            f = ex2(-d);
                        }
                        // (Else the bound was too wide: a large value scale beside a small weight.)
                        if (__any_sync(0xffffffffu, d != 0.f)) {
                            nb = minus_base(ref);
                            l *= f;
                            // Loads are not ordered behind this thread's own stores without a wait: the
                            // earlier weights must have arrived before they are read back.
                            tmem_wait_st();
#pragma unroll 1
                            for (int c = 0; c < 2 * c2; c++) {
                                tmem_ld16_start(S + 16 * c, t0);
                                tmem_ld16_wait(t0);
#pragma unroll
                                for (int e = 0; e < 8 * SPLIT; e++) {
                                    const float2 v = __half22float2(*reinterpret_cast<__half2 *>(&t0[e]));
                                    t0[e] = half2_bits(v.x * f, v.y * f);  // (f may be below fp16)
                                }
                                tmem_st16(S + 16 * c, t0);
                            }
                            if (j > 0) {
                                wait(bar.o_full[w][(cw - 1) & 1], (cw - 1) >> 1);
                                tc_fence_after();
#pragma unroll 1
                                for (int c = 0; c < D; c += 16) {
                                    tmem_ld16_start(O + c, t0);
                                    tmem_ld16_wait(t0);
#pragma unroll
                                    for (int e = 0; e < 16; e++)
                                        t0[e] = __float_as_uint(__uint_as_float(t0[e]) * f);
                                    tmem_st16(O + c, t0);
                                }
                                if (SPLIT == 2 && j > kFlush) {
#pragma unroll 1
                                    for (int c = 0; c < D / 4; c++) {
                                        const float4 v = __ldcg(sums + c * kRows);
                                        __stcg(sums + c * kRows, make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
                                    }
                                }
                            }
                            tmem_wait_st();
                            sum = 0;
#pragma unroll 1
                            for (int c = 2 * c2; c < 2 * c2 + 2; c++) {
                                uint32_t pw[8 * SPLIT];
                                tmem_ld16_start(S + 16 * c, t0);
                                tmem_ld16_wait(t0);
                                pairs_of(t0, s);
                                scores(c, s, less);
                                weights(c, s, sum, pw);
                                tmem_st_weights(S + 16 * c, pw);
                            }
                            part = lo_of(sum) + hi_of(sum);
                            keep = false;
                        }
                    }
                    l += part;
#pragma unroll
                    for (int k = 0; k < 2; k++)
                        if (keep) tmem_st_weights(S + 32 * c2 + 16 * k, ph[k]);
                }
                if (SPLIT == 2 && j > 0 && j % kFlush == 0) {
                    wait(bar.o_full[w][(cw - 1) & 1], (cw - 1) >> 1);
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t t[32];
                        tmem_ld32(O + c, t);
#pragma unroll
                        for (int e = 0; e < 8; e++) {
                            float4 *at = sums + (c / 4 + e) * kRows;
                            const float4 v = make_float4(__uint_as_float(t[4 * e]), __uint_as_float(t[4 * e + 1]),
                                                         __uint_as_float(t[4 * e + 2]), __uint_as_float(t[4 * e + 3]));
                            if (j == kFlush) __stcg(at, v);
                            else atomicAdd(at, v);
                        }
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_full[w][cw & 1]);
            }

            // ---- outputs, or this CTA's part of them ----
            wait(bar.o_full[w][(cw - 1) & 1], (cw - 1) >> 1);
            tc_fence_after();
            const bool whole = it.first == 0 && it.last == it.x.tiles;
            const int part = 2 * blockIdx.x + (it.first == 0 ? 1 : 0);
            const int cc = row0 + row, head = it.h * p.group + cc % p.group;
            const int64_t t = it.q.q0 + cc / p.group;
            // (a row that has seen nothing has l = 0, and its output is 0)
            const float f = (!whole ? 1.f : l == 0.f ? 0.f : 1.f / l) * (1.f / kTcLift);
#pragma unroll 1
            for (int c = 0; c < D; c += 64) {
                // column 8 e + k of these 64 is dimension 8 k + e
                uint32_t o0[32], o1[32];
                tmem_ld32(O + c, o0);
                tmem_ld32(O + c + 32, o1);
                if (SPLIT == 2 && n > kFlush) {
#pragma unroll
                    for (int e = 0; e < 16; e++) {
                        const float4 v = __ldcg(sums + (c / 4 + e) * kRows);
                        uint32_t *o = e < 8 ? o0 + 4 * e : o1 + 4 * (e - 8);
                        o[0] = __float_as_uint(__uint_as_float(o[0]) + v.x);
                        o[1] = __float_as_uint(__uint_as_float(o[1]) + v.y);
                        o[2] = __float_as_uint(__uint_as_float(o[2]) + v.z);
                        o[3] = __float_as_uint(__uint_as_float(o[3]) + v.w);
                    }
                }
                if (row < ncol) {
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        float y[8];
#pragma unroll
                        for (int e = 0; e < 8; e++) {
                            y[e] = __uint_as_float(e < 4 ? o0[8 * e + k] : o1[8 * (e - 4) + k]) * f;
                            if (whole && l == 0.f) y[e] = 0.f;
                        }
                        if (whole)
                            store8(static_cast<T *>(p.out) + t * p.out_stride + (int64_t)head * D + c + 8 * k, y);
                        else
                            store8(p.part + ((int64_t)part * (2 * kRows) + w * kRows + row) * D + c + 8 * k, y);
                    }
                }
                __syncwarp();
            }
            if (row < ncol) {
                if (!whole)
                    p.stat[part * 2 * kRows + w * kRows + row] = make_float2(ref, l);
                else if (p.lse)
                    p.lse[t * p.heads + head] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
            }
            if (!whole && tid == 0) {
                // the CTA of the item's first tile (of the item, if it is never split)
                const int owner = (int)(((it.begin + kItemCost + 1) * ctas - 1) / total);
                record[it.first == 0 ? 1 : 0] = make_int4(
                    it.r, it.b * p.kv_heads + it.h, it.last == it.x.tiles ? owner + 1 : 0, it.x.rows);
            }
            tc_fence_before();  // O is read before the next item's products write it
        }
    } else if (warp < 12) {
        // =================== codes to fp16 operands: one chunk per warp and piece ===================
        const int q = warp - 8;
        const __half2 k1024 = __half2half2(__ushort_as_half(0x6400)), k64 = __half2half2(__ushort_as_half(0x5400));
        // 8 codes less their zeros: pairs (0,4) (1,5) (2,6) (3,7); z1024 = 1024 + z, z64 = 64 + z.
        auto unfold = [&](uint32_t w, __half2 z1024, __half2 z64, uint32_t (&x)[4]) {
            const uint32_t h = w >> 8;
            uint32_t y[4];
            asm("lop3.b32 %0, %1, 0x000F000F, 0x64006400, 0xEA;" : "=r"(y[0]) : "r"(w));
            asm("lop3.b32 %0, %1, 0x00F000F0, 0x54005400, 0xEA;" : "=r"(y[1]) : "r"(w));
            asm("lop3.b32 %0, %1, 0x000F000F, 0x64006400, 0xEA;" : "=r"(y[2]) : "r"(h));
            asm("lop3.b32 %0, %1, 0x00F000F0, 0x54005400, 0xEA;" : "=r"(y[3]) : "r"(h));
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const __half2 v = __hsub2(*reinterpret_cast<__half2 *>(&y[e]), e & 1 ? z64 : z1024);
                x[e] = *reinterpret_cast<const uint32_t *>(&v);
            }
        };
        while (it.next(p)) {
            const int n = it.last - it.first;
            for (int j = 0; j < n; j++, gt++) {
                const int buf = gt % C::kBuf, slot = gt % kScales;
                const uint32_t turn = gt / C::kBuf;
                uint8_t *K = smem + C::oK + buf * C::kTileB, *V = smem + C::oV + buf * C::kTileB;
                wait(bar.k_empty[buf], turn + 1);
                const int st = gt % kPieces;
                wait(bar.raw_full[st], gt / kPieces);
                const uint8_t *chunk = smem + C::oRaw + st * C::kRaw + q * kv4_chunk_bytes(D);
                const uint32_t valid = raw_valid[st];
                const int j0 = (it.x.t0 + it.first + j) * kKeys + q * 16;
                const int live = valid >> q & 1 ? min(16, it.x.hi - j0) : 0;  // tokens that exist
                const __half2 *pairs = reinterpret_cast<const __half2 *>(chunk + 2 * kv4_codes_bytes(D));
                    {  // scales: lane t < 16 keys, the others values
                        const int t = lane & 15;
                        const float d = t < live ? __low2float(pairs[lane]) : 0.f;
                        const int at = slot * kKeys + q * 16 + t;
                        if (lane < 16) kd_s[at] = d;
                        else vd_s[at] = d * kTcLift, vl_s[at] = scale_log2(d);
                        float m = lane < 16 ? 0.f : d * kTcLift;
#pragma unroll
                        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                        if (lane == 16) sc_max[slot][q] = m;
                        if (lane == 0 && q == 0) sc_valid[slot] = valid;
                    }
                    // ---- keys ----
                    constexpr int QN = D / 32;              // 16-byte quarters of a key row
                    constexpr int TN = 32 / QN;             // tokens per step
#pragma unroll
                    for (int s = 0; s < 16 / TN; s++) {
                        const int t8 = lane & 7, t = s * TN + (lane >> 3) / QN * 8 + t8;
                        // rotated so that both the reads and the writes of 8 lanes miss each other
                        const int kq = ((lane >> 3) % QN + (D == 128 ? t8 >> 1 : t8 >> 2)) % QN;
                        const uint4 wv = *reinterpret_cast<const uint4 *>(chunk + t * (D / 2) + kq * 16);
                        const uint32_t w4[4] = {wv.x, wv.y, wv.z, wv.w};
                        const __half2 z = __half2half2(t < live ? __high2half(pairs[t]) : __ushort_as_half(0));
                        const __half2 za = __hadd2(k1024, z), zb = __hadd2(k64, z);
                        const int tt = q * 16 + t;
                        uint8_t *dst = K + (tt >> 3) * (D * 16) + (kq * 4) * 128 + (tt & 7) * 16;
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            uint32_t x[4];
                            unfold(w4[i], za, zb, x);
                            *reinterpret_cast<uint4 *>(dst + i * 128) = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                    }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.k_full[buf]), mbar_arrive(&bar.sc_full[slot]);
                wait(bar.v_empty[buf], turn + 1);
                {
                    // ---- values: 8 tokens x 8 dimensions per lane, transposed ----
                    constexpr int WN = D / 8;
                    if (lane < 2 * WN) {
                        const int wi = lane % WN, gr = lane / WN;
                        const uint8_t *src = chunk + kv4_codes_bytes(D) + gr * 8 * (D / 2) + wi * 4;
                        uint32_t wa[4], wb[4];
                        __half2 za[4], zb[4];
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            // the second half warp reads a pair's tokens in the other order (banks)
                            wa[i] = *reinterpret_cast<const uint32_t *>(src + (2 * i + gr) * (D / 2));
                            wb[i] = *reinterpret_cast<const uint32_t *>(src + (2 * i + 1 - gr) * (D / 2));
                            const int t = gr * 8 + 2 * i;
                            const __half z0 = t < live ? __high2half(pairs[16 + t]) : __ushort_as_half(0);
                            const __half z1 = t + 1 < live ? __high2half(pairs[16 + t + 1]) : __ushort_as_half(0);
                            const __half2 z = __halves2half2(z0, z1);
                            za[i] = __hadd2(k1024, z), zb[i] = __hadd2(k64, z);
                        }
                        // dimension 8 wi + e is row 64 (wi / 8) + 8 e + wi % 8 of the operand
                        uint8_t *dst = V + (wi >> 3) * (8 * kKeys * 16) + (q * 2 + gr) * 128 + (wi & 7) * 16;
#pragma unroll
                        for (int hw = 0; hw < 2; hw++) {
                            const uint32_t sel = hw ? (gr ? 0x3276 : 0x7632) : (gr ? 0x1054 : 0x5410);
                            uint32_t x[4][4];  // token pair, dimension
#pragma unroll
                            for (int i = 0; i < 4; i++) unfold(prmt(wa[i], wb[i], sel), za[i], zb[i], x[i]);
#pragma unroll
                            for (int e = 0; e < 4; e++)
                                *reinterpret_cast<uint4 *>(dst + (4 * hw + e) * (kKeys * 16)) =
                                    make_uint4(x[0][e], x[1][e], x[2][e], x[3][e]);
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.raw_empty[st]), mbar_arrive(&bar.v_full[buf]);
            }
        }
    } else if (warp == 12) {
        // =================== tensor-core operations ===================
        const uint32_t sb = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t dQ = desc_low(sb + C::oQ), dK = desc_low(sb + C::oK), dV = desc_low(sb + C::oV);
        constexpr uint32_t idS = idesc_f16(128, kKeys), idO = idesc_f16(128, D);
        constexpr uint32_t hQ = desc_high(D * 16), hV = desc_high(kKeys * 16);
        uint32_t cw[2] = {0, 0}, nq[2] = {0, 0};  // key tiles and items of each row tile so far
        auto qk = [&](int w, uint32_t tile, int buf, bool last) {
            if (elect_one()) {
#pragma unroll
                for (int s = 0; s < SPLIT; s++)
#pragma unroll
                    for (int k = 0; k < D / 64; k++)
                        mma4_ss<hQ, hQ>(tm + 2 * kKeys * w + kKeys * (tile & 1),
                                        dQ + (((w * SPLIT + s) * C::kQ + k * 1024) >> 4),
                                        dK + ((buf * C::kTileB + k * 1024) >> 4), idS, s + k > 0);
                mma_commit(&bar.s_full[w][tile & 1]);
                if (last) mma_commit(&bar.k_empty[buf]);
            }
            __syncwarp();
        };
        while (it.next(p)) {
            const int n = __shfl_sync(0xffffffffu, it.last - it.first, 0);
            const int tiles = __shfl_sync(0xffffffffu, it.x.rows > kRows ? 2 : 1, 0);
            wait(bar.k_full[gt % C::kBuf], gt / C::kBuf);
#pragma unroll
            for (int w = 0; w < 2; w++) {
                if (w >= tiles) continue;
                wait(bar.q_full[w], nq[w]++);
                tc_fence_after();
                qk(w, cw[w], gt % C::kBuf, w == tiles - 1);
            }
            for (int j = 0; j < n; j++, gt++) {
                const int buf = gt % C::kBuf, nb = (gt + 1) % C::kBuf;
#pragma unroll
                for (int w = 0; w < 2; w++) {
                    if (w >= tiles) continue;
                    if (j + 1 < n) {
                        if (w == 0) wait(bar.k_full[nb], (gt + 1) / C::kBuf);
                        tc_fence_after();
                        qk(w, cw[w] + 1, nb, w == tiles - 1);
                    }
                    if (w == 0) wait(bar.v_full[buf], gt / C::kBuf);
                    wait(bar.p_full[w][cw[w] & 1], cw[w] >> 1);
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int s = 0; s < SPLIT; s++)
                            mma4_ts<hV>(tm + 256 + D * w, tm + 2 * kKeys * w + kKeys * (cw[w] & 1) + 8 * s,
                                        dV + ((buf * C::kTileB) >> 4), idO,
                                        s > 0 || (SPLIT == 2 ? j % kFlush : j) > 0);
                        mma_commit(&bar.o_full[w][cw[w] & 1]);
                        if (w == tiles - 1) mma_commit(&bar.v_empty[buf]);
                    }
                    __syncwarp();
                    cw[w]++;
                }
            }
        }
        // The last arrivals of the tensor core must not outlive the CTA's shared memory.
        if (gt > 0) {
            wait(bar.k_empty[(gt - 1) % C::kBuf], (gt - 1) / C::kBuf);
            wait(bar.v_empty[(gt - 1) % C::kBuf], (gt - 1) / C::kBuf);
        }
    } else {
        // =================== cache chunks into shared memory ===================
        uint32_t piece = 0;
        const int64_t page_bytes = ((int64_t)p.kv_heads << (p.shift - 4)) * kv4_chunk_bytes(D);
        while (it.next(p)) {
            const int n = it.last - it.first;
            const uint8_t *base = p.cache + ((int64_t)it.h << (p.shift - 4)) * kv4_chunk_bytes(D);
            const int32_t *row = p.table + (int64_t)it.r * p.width;
            int page = -1;
            for (int i = 0; i < n; i++, piece++) {
                const int tok0 = (it.x.t0 + it.first + i) * kKeys;
                if ((i & 7) == 0) {  // the pages of the next 32 chunks, one per lane
                    const int j = tok0 + 16 * lane;
                    const int64_t c = j >> p.shift;
                    page = i + (lane >> 2) < n && j < it.x.hi && c < p.width ? row[c] : -1;
                }
                const int pg = __shfl_sync(0xffffffffu, page, (i & 7) * 4 + (lane & 3));
                const int j = tok0 + 16 * (lane & 3), st = piece % kPieces;
                const bool ok = lane < 4 && pg >= 0 && pg < p.pages && j < it.x.hi && j + 16 > it.x.lo;
                const uint32_t valid = __ballot_sync(0xffffffffu, ok);
                wait(bar.raw_empty[st], piece / kPieces + 1);
                if (lane == 0) {
                    raw_valid[st] = valid;
                    mbar_arrive_expect_tx(&bar.raw_full[st], __popc(valid) * kv4_chunk_bytes(D));
                }
                __syncwarp();
                if (ok)
                    bulk_g2s(smem + C::oRaw + st * C::kRaw + lane * kv4_chunk_bytes(D),
                             base + pg * page_bytes + ((j & ((1 << p.shift) - 1)) >> 4) * kv4_chunk_bytes(D),
                             kv4_chunk_bytes(D), &bar.raw_full[st]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the parts of items that several CTAs shared, a warp per row (see attn_join_kernel).
template <int D, typename T>
__global__ void __launch_bounds__(256) attn_join_rows_kernel(const AttnParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.x, lane = threadIdx.x & 31;
    const int row = blockIdx.y * 8 + (threadIdx.x >> 5);
    const int4 rec = p.record[2 * b];
    if (rec.x < 0 || rec.z == 0 || row >= rec.w) return;
    const int first = rec.z - 1, n = b - first + 1;
    auto at_of = [&](int i) { return (int64_t)(i == 0 ? 2 * first + 1 : 2 * (first + i)) * (2 * kRows) + row; };
    float m = -INFINITY, l = 0.f, x[4] = {};
    for (int i = 0; i < n; i++) m = fmaxf(m, p.stat[at_of(i)].x);
    if (lane * 4 < D) {
        for (int i = 0; i < n; i++) {
            const float2 s = p.stat[at_of(i)];
            const float4 v = *reinterpret_cast<const float4 *>(p.part + at_of(i) * D + lane * 4);
            const float f = s.x == -INFINITY ? 0.f : ex2(s.x - m);
            l = fmaf(f, s.y, l);
            x[0] = fmaf(f, v.x, x[0]), x[1] = fmaf(f, v.y, x[1]);
            x[2] = fmaf(f, v.z, x[2]), x[3] = fmaf(f, v.w, x[3]);
        }
        const Request q = load_request(p, rec.x);
        const int cc = rec.y / p.kv_heads * 2 * kRows + row;
        const int head = rec.y % p.kv_heads * p.group + cc % p.group;
        const int64_t t = q.q0 + cc / p.group;
        T *dst = static_cast<T *>(p.out) + t * p.out_stride + (int64_t)head * D + lane * 4;
#pragma unroll
        for (int e = 0; e < 4; e++) store_value(dst + e, l == 0.f ? 0.f : x[e] / l);
        if (p.lse && lane == 0) p.lse[t * p.heads + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
}

size_t attn_prompt_workspace(int head_dim) {
    return (size_t)kTcMaxCtas * 2 * (16 + 2 * kRows * (8 + (size_t)head_dim * 4) +
                                     kRows * (size_t)head_dim * 4);
}

template <int D, typename T>
static int launch_prompt(AttnParams p, uint8_t *workspace, int sms, cudaStream_t st) {
    constexpr int SPLIT = sizeof(T) == 4 ? 2 : 1;
    using C = Prompt<D, SPLIT>;
    p.record = reinterpret_cast<int4 *>(workspace);
    p.stat = reinterpret_cast<float2 *>(p.record + 2 * kTcMaxCtas);
    p.part = reinterpret_cast<float *>(p.stat + 2 * kTcMaxCtas * 2 * kRows);
    p.sums = reinterpret_cast<float4 *>(p.part + (size_t)2 * kTcMaxCtas * 2 * kRows * D);
    auto kernel = attn_prompt_kernel<D, T, SPLIT>;
    int per_sm;
    if (int e = prepare_kernel((const void *)kernel, kTcThreads, C::kSmem, &per_sm)) return e;
    const int ctas = sms < kTcMaxCtas ? sms : kTcMaxCtas;
    if (int e = launch_pdl(kernel, dim3(ctas), dim3(kTcThreads), C::kSmem, st, p)) return e;
    if ((p.width << p.shift) <= kTcWhole * kKeys) return LB_OK;  // no item can have been split
    return launch_pdl(attn_join_rows_kernel<D, T>, dim3(ctas, 2 * kRows / 8), dim3(256), 0, st, p);
}

int attn_prompt(const AttnParams &p, int type, int head_dim, uint8_t *workspace, int sms,
                cudaStream_t st) {
    if (type == LB_OUT_F32)
        return head_dim == 64 ? launch_prompt<64, float>(p, workspace, sms, st)
                              : launch_prompt<128, float>(p, workspace, sms, st);
    return head_dim == 64 ? launch_prompt<64, __nv_bfloat16>(p, workspace, sms, st)
                          : launch_prompt<128, __nv_bfloat16>(p, workspace, sms, st);
}

}  // namespace lb
