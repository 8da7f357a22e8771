// lb_q4_gemm.cuh -- products of 4-bit weights with group scales for many tokens, on the 5th-generation
// tensor cores.
//
// Mathematics.  D[n][t] = sum_k w[n][k] x[t][k], 128 weight rows (the accumulator's lanes) times up to
// 256 tokens.  The weights are expanded once per item by eight warps, a thread per row, from 16-byte loads
// of codes straight into tensor memory, from where the tensor cores read them as their first operand; x
// comes through shared memory.  Two forms:
//   bf16 tensors: the operand is d (c - z), rounded to fp16's 11 bits (an eighth of a bf16
//     output's own rounding); the accumulator runs over all of K.
//   fp32 tensors: the operand is c - z, exact; x enters as two fp16 parts, one product each; the sums of
//     a group leave the accumulator, of which there are two in turn, and are added to binary32 sums in
//     registers with the group's scale.  (The tensor cores cut what lies below an accumulator's last
//     place downwards at every step of 16: over a long row that is far more than binary32 rounding.)
// Rows of x are scaled by powers of two into fp16's range beforehand (q4_rows), and stored in the order
// in which the codes of a word unfold, pairs (0, 4), (1, 5), (2, 6), (3, 7).
//
// One CTA per SM, 20 warps (one has nothing to do): eight that take the sums out (a quarter of the lanes times half of
// the columns each), eight that expand weights, one that has codes copied in (tensor copies, 128 rows x 128
// columns), one that has x copied in (tensor copies of half of an item's tokens x 64 columns), one that issues the tensor-core
// operations.  Each CTA copies what it multiplies into its own shared memory.  Calls with few tiles are split along K over
// a cluster; the parts are added up through distributed shared memory.
//
// What bounds it: with many tokens the products (4096 x 12288 x 4096 bf16: 235 us, the tensor pipe busy for 78 % of
// them); with few per item, at 460 clocks a step of 64 columns, issue slots (56 %) and latency: the warps that expand
// weights are busy for 300 of them, the one that issues products for 300 (49 tokens for each of 128 experts, DRAM 35 %);
// in fp32 the products' issue and a drain per group, about 900 clocks a step (509 x 6912 x 2560: 38 us).
#pragma once
#include "lb_q4.cuh"
#include "lb_tc.cuh"

#include <algorithm>

namespace lb {

constexpr int kGmRows = 128;
constexpr int kGmStep = 64;              // columns of K of a stage
constexpr int kGmOutWarps = 8, kGmExpandWarps = 8;
constexpr int kGmCodeWarp = kGmOutWarps + kGmExpandWarps, kGmCopyWarp = kGmCodeWarp + 1;
constexpr int kGmMmaWarp = kGmCopyWarp + 1;
constexpr int kGmWarps = kGmMmaWarp + 2;   // (whole groups of four)
constexpr int kGmThreads = 32 * kGmWarps;
constexpr int kGmOutThreads = 32 * kGmOutWarps;
constexpr int kGmC = kGmRows * 64;       // bytes of a stage of codes: two steps

constexpr int kGmMaxSplit = 8;           // a portable cluster
// What depends on the tokens of an item (with two parts: of each).  Of tensor memory's 512 columns two accumulators of 176
// tokens leave as many as five stages of weights take; 256 tokens leave room for one accumulator, whose way out then is
// not hidden (a third of the time of experts' products with 205 tokens a piece, 12 % with K = 4096).
template <int TOKENS, int PARTS>
struct GmShape {
    static constexpr int kB = TOKENS * 128 * PARTS;                // bytes of a stage of x
    static constexpr int kBuffers = TOKENS > 176 ? 1 : 2;          // accumulators
    static constexpr int kABase = kBuffers * TOKENS;               // expanded weights lie behind them, 32 columns a stage
    static constexpr int kStages = kB > 16384 ? 5 : 8;             // of x and of expanded weights
    static constexpr int kCStages = kB == 32768 ? 6 : 10;          // of codes
    static_assert(kABase + 32 * kStages <= 512, "tensor memory");
    static_assert(TOKENS % 16 == 0, "pieces are multiples of 16");
    static constexpr int kSmem = kStages * kB + kCStages * kGmC;
};
constexpr int kGmMaxStages = 8, kGmMaxCStages = 10;

struct GmLaunch {
    int steps;        // of K, of a CTA
    int split;        // CTAs along K, a cluster
    int box;          // tokens of a copy
    int pairs;        // two rows of a bf16 y may be stored as one word
    int tokens;       // of an item, at most (dense)
    int tiles;        // of weight rows
    int fault;        // test hook: CTA 0 copies no codes and waits so many microseconds for the first ones
};

struct GmBars {
    uint64_t full[kGmMaxStages], empty[kGmMaxStages];
    uint64_t c_full[kGmMaxCStages], c_empty[kGmMaxCStages];
    uint64_t d_full[2], d_empty[2], done;
};

// Shared-memory matrix descriptor, K-major rows of 128 bytes under the 128-byte swizzle: eight rows are 1024
// bytes, a step of 16 along K is 32 bytes further.
constexpr uint32_t gm_desc_high() { return (1024 >> 4) | 1u << 14 | 2u << 29; }
__device__ __forceinline__ uint32_t gm_desc_low(uint32_t saddr) { return ((saddr >> 4) & 0x3FFF) | 1u << 16; }
// D[tmem] (+)= A[tmem] * B[desc]^T over 64 of K.
__device__ __forceinline__ void gm_mma4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p; .reg .b64 b; .reg .b32 a;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 b, {%2, %5}; mov.b32 a, %1;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p;\n\t"
        "setp.eq.b32 p, 0, 0;\n\t"
        "add.s32 a, a, 8; add.s64 b, b, 2;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p;\n\t"
        "add.s32 a, a, 8; add.s64 b, b, 2;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p;\n\t"
        "add.s32 a, a, 8; add.s64 b, b, 2;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p; }" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(gm_desc_high())
        : "memory");
}
// The same over 32 of K.
__device__ __forceinline__ void gm_mma2(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p; .reg .b64 b; .reg .b32 a;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 b, {%2, %5}; mov.b32 a, %1;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p;\n\t"
        "setp.eq.b32 p, 0, 0;\n\t"
        "add.s32 a, a, 8; add.s64 b, b, 2;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p; }" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(gm_desc_high())
        : "memory");
}
__device__ __forceinline__ bool gm_elect() {
    uint32_t x;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(x));
    return x != 0;
}
__device__ __forceinline__ void gm_tmem_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// A group of four warps' registers per thread.  640 threads start with 96 (61440); with fp32 tensors 256 have 144 then,
// 256 have 80 and 128 have 32 (61440), and in the end all 96 again.  The others take theirs back only after the
// 256 have given theirs up: a CTA without work would otherwise have nothing left for warps that still wait
// for their 144.
template <int N>
__device__ __forceinline__ void gm_more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void gm_fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// 16 columns asked for; they are there after gm_ld_wait.
__device__ __forceinline__ void gm_ld16_start(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void gm_ld_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

__device__ __forceinline__ void gm_store(float *p, float v) { *p = v; }
__device__ __forceinline__ void gm_store(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float gm_cluster_load(const float *p, uint32_t rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void gm_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// On to the next scales and zeros of a warp that takes every other unit of 128 columns.
template <int GROUP>
__device__ __forceinline__ void q4_rotate(uint4 &d, uint2 &z) {
    if (GROUP == 64) {
        d.x = d.z, d.y = d.w;
        z.x = z.y;
    } else if (GROUP == 128) {
        d.x = d.y, d.y = d.z, d.z = d.w;
        z.x = __funnelshift_r(z.x, z.y, 16), z.y >>= 16;
    }   // (32: a block of eight groups has one unit of the warp's)
}

// A place in a ring of N stages, and the parity of its present phase.
template <int N>
struct GmRing {
    uint32_t i = 0, phase = 0;
    __device__ __forceinline__ void next(uint32_t n = 1) {   // n <= N
        i += n;
        if (i >= N) i -= N, phase ^= 1;
    }
    __device__ __forceinline__ void skip(uint32_t n) {
        i += n;
        phase ^= (i / N) & 1;
        i %= N;
    }
};

// An item: up to kTokens tokens (of one expert) times one tile of weight rows.
struct GmItem {
    int expert, t0, tokens, tile;
};

// T: the tensors' type.  F32: their two-part form.
template <Q4Use USE, typename T, int TOKENS, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(kGmThreads, 1)
    q4_gemm_kernel(const __grid_constant__ CUtensorMap code_map, const __grid_constant__ CUtensorMap x_map,
                   const __grid_constant__ Q4Params p, const __grid_constant__ Q4Rows r,
                   const __grid_constant__ GmLaunch l) {
    constexpr bool F32 = sizeof(T) == 4;
    constexpr int kTokens = TOKENS;
    constexpr int kParts = F32 ? 2 : 1;
    constexpr int kCols = (kTokens / 2 + 15) / 16 * 16;   // of an output warp, at most
    using Shape = GmShape<TOKENS, kParts>;
    constexpr int kGmStages = Shape::kStages, kGmB = Shape::kB, kGmCStages = Shape::kCStages;
    constexpr int kBuffers = Shape::kBuffers, kGmABase = Shape::kABase;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ GmBars bar;
    __shared__ uint32_t s_tmem;
    constexpr int kExperts = USE == kQ4Dense ? 1 : LB_ROUTE_MAX_EXPERTS;
    __shared__ int s_first[kExperts], s_row[kExperts], s_count[kExperts];  // pieces and pairs before an expert's, pairs
    __shared__ int s_part[32];
    __shared__ __align__(16) float col_scale[2][kTokens];   // of an item and the next one
    __shared__ __align__(16) int col_row[2][kTokens];
    // (from the warp's first lane: what is made of it stays in the uniform registers that the operations take)
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int rank = blockIdx.x % l.split;            // along K

    if (tid == 0) {
        // a stage is full when its four warps of weights and the copies of x are there
        for (int i = 0; i < kGmStages; i++) mbar_init(&bar.full[i], 5), mbar_init(&bar.empty[i], 1);
        for (int i = 0; i < kGmCStages; i++) mbar_init(&bar.c_full[i], 1), mbar_init(&bar.c_empty[i], 4);
        for (int i = 0; i < 2; i++) mbar_init(&bar.d_full[i], 1), mbar_init(&bar.d_empty[i], kGmOutWarps);
        mbar_init(&bar.done, 1);
        fence_mbar_init();
    }
    pdl_wait();
    // Pieces of at most kTokens tokens: their number, and where an expert's begin.
    int pieces;
    if constexpr (USE == kQ4Dense) {
        pieces = (int)((p.T + l.tokens - 1) / l.tokens);
    } else {
        constexpr int kEach = (LB_ROUTE_MAX_EXPERTS + kGmThreads - 1) / kGmThreads;
        int n[kEach], sum = 0;
#pragma unroll
        for (int i = 0; i < kEach; i++) {
            const int e = tid * kEach + i;
            n[i] = 0;
            if (e < p.E) {
                const int first = min(max(p.start[e], 0), (int)p.T);
                const int count = max(min(p.start[e + 1], (int)p.T) - first, 0);
                s_row[e] = first, s_count[e] = count;
                n[i] = (count + kTokens - 1) / kTokens;
            }
            sum += n[i];
        }
        int run = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int w = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += w;
        }
        if (lane == 31) s_part[warp] = run;
        __syncthreads();
        int before = run - sum, total = 0;
        for (int w = 0; w < kGmWarps; w++) {
            before += w < warp ? s_part[w] : 0;
            total += s_part[w];
        }
#pragma unroll
        for (int i = 0; i < kEach; i++) {
            if (tid * kEach + i < p.E) s_first[tid * kEach + i] = before;
            before += n[i];
        }
        pieces = total;
    }
    // Tensor memory is taken when the kernels before this one have ended, and the next one may start only after
    // it: neither waits for the other's columns.
    if (warp == kGmMmaWarp) tmem_alloc(&s_tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
    const int items = pieces * l.tiles;
    const int each = gridDim.x / l.split, begin = blockIdx.x / l.split;
    auto item_of = [&](int i) {
        GmItem it;
        const int piece = i / l.tiles;
        it.tile = i - piece * l.tiles;
        if constexpr (USE == kQ4Dense) {
            it.expert = 0;
            it.t0 = piece * l.tokens;
            it.tokens = (int)min((int64_t)l.tokens, p.T - it.t0);
        } else {
            int lo = 0, hi = p.E;   // the last expert whose pieces begin at or before this one
            while (hi - lo > 1) {
                const int m = (lo + hi) / 2;
                if (s_first[m] <= piece) lo = m;
                else hi = m;
            }
            it.expert = lo;
            // pieces of one size, a multiple of 16: a small last one would take as long to expand weights for as the others
            const int count = s_count[lo], n = (count + kTokens - 1) / kTokens;
            const int size = ((count + n - 1) / n + 15) / 16 * 16, at = (piece - s_first[lo]) * size;
            it.t0 = s_row[lo] + at;
            it.tokens = max(min(size, count - at), 0);
        }
        return it;
    };
    // Row of the weights (among all matrices' rows) that a lane of the accumulator holds, and whether it is one.
    const int64_t matrix_rows = USE == kQ4Up ? 2 * p.N : p.N;
    auto row_of = [&](const GmItem &it, int at, bool &in) -> int64_t {
        if (USE == kQ4Up) {   // 16 gate rows, then the same 16 up rows
            const int64_t n = it.tile * (int64_t)(kGmRows / 2) + (at >> 5) * 16 + (at & 15);
            in = n < p.N;
            return it.expert * matrix_rows + (at & 16 ? p.N : 0) + n;
        }
        const int64_t n = it.tile * (int64_t)kGmRows + at;
        in = n < p.N;
        return it.expert * matrix_rows + n;
    };
    const int k0 = rank * l.steps * kGmStep;                             // this CTA's slice of K
    const int columns = min(p.K - k0, l.steps * kGmStep);
    const int steps = (columns + kGmStep - 1) / kGmStep;

    // Bounded: about 2 s, after the first that ran out 0.1 ms.
    const bool starve = l.fault && blockIdx.x == 0;
    int tries = kWaitTries;
    auto wait = [&](uint64_t &b, uint32_t parity) {
        if (!mbar_try_wait(&b, parity & 1)) {
            int i = 0;
            while (!mbar_try_wait_hint(&b, parity & 1, 1000000u) && i < tries) i++;
            if (i >= tries) {
                *p.error = 1;
                tries = wait_tries(100);
            }
        }
        __syncwarp();
    };

    if (warp < kGmOutWarps) {
        // =================== sums out: a lane per weight row ===================
        if constexpr (F32) gm_more_registers<144>();
        const int quarter = warp & 3;
        uint32_t turn = 0;   // accumulators taken so far
        // scale and output row of an item's column tid
        float scale = 0.f;
        int to = 0;
        GmItem ahead{0, 0, 0, 0};
        auto ask = [&](int i) {
            if (i >= items) return;
            ahead = item_of(i);
            if (tid >= ahead.tokens) return;
            scale = r.row_scale[ahead.t0 + tid];
            to = ahead.t0 + tid;
            if (USE == kQ4Down) {
                const int pair = p.order[ahead.t0 + tid];
                to = pair >= 0 && pair < p.T ? pair : -1;
            }
        };
        int buf = 0;
        auto tell = [&]() {
            if (tid < kTokens) col_scale[buf][tid] = scale, col_row[buf][tid] = to;
            __syncwarp();
            named_sync(1, kGmOutThreads);
        };
        ask(begin);
        tell();
#pragma unroll 1
        for (int i = begin; i < items; i += each) {
            const GmItem it = ahead;
            ask(i + each);
            bool in;
            const int64_t row = row_of(it, quarter * 32 + lane, in);
            // half of the columns each, in sixteens
            const int half = (it.tokens + 31) / 32 * 16, c0 = warp < 4 ? 0 : half;
            const int mine = warp < 4 ? min(it.tokens, half) : it.tokens - min(it.tokens, half);
            const uint32_t at_lane = tmem + ((uint32_t)(quarter * 32) << 16) + c0;
            float *park = reinterpret_cast<float *>(smem) + c0 * kGmRows + quarter * 32 + lane;   // [column][128]
            // 16 columns from c (of this warp's) on
            auto emit = [&](int c, const float (&v)[16]) {
                if (USE == kQ4Dense && l.split > 1) {
#pragma unroll
                    for (int j = 0; j < 16; j++)
                        if (c + j < mine) park[(c + j) * kGmRows] = v[j];
                    return;
                }
                float x[16];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const float4 f = *reinterpret_cast<const float4 *>(&col_scale[buf][c0 + c + 4 * j]);
                    x[4 * j] = v[4 * j] * f.x, x[4 * j + 1] = v[4 * j + 1] * f.y;
                    x[4 * j + 2] = v[4 * j + 2] * f.z, x[4 * j + 3] = v[4 * j + 3] * f.w;
                }
                const int left = mine - c;
                if constexpr (USE == kQ4Up) {
                    // gate and up rows of a column pair meet: lanes 0..15 make h of the first column, 16..31 of the second
                    const int64_t n = it.tile * (int64_t)(kGmRows / 2) + quarter * 16 + (lane & 15);
                    float *h = static_cast<float *>(p.y) + (int64_t)(it.t0 + c0 + c + (lane >> 4)) * p.y_stride + n;
                    const int mine_left = n < p.N ? left - (lane >> 4) : 0;
#pragma unroll
                    for (int j = 0; j < 16; j += 2, h += 2 * p.y_stride) {
                        const float other = __shfl_xor_sync(0xffffffffu, lane < 16 ? x[j + 1] : x[j], 16);
                        const float gate = lane < 16 ? x[j] : other, up = lane < 16 ? other : x[j + 1];
                        // (bf16: exp and quotient to a few units of 2^-22, nothing beside an output's rounding)
                        const float silu = F32 ? gate / (1.f + expf(-gate)) : __fdividef(gate, 1.f + __expf(-gate));
                        if (j < mine_left) *h = silu * up;
                    }
                } else if constexpr (USE == kQ4Down) {
                    // (rows of a full sixteen go out without a question each: 4096 tokens' experts in a graph 469 -> 464 us)
                    int at[16], all = 0;
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const int4 q = *reinterpret_cast<const int4 *>(&col_row[buf][c0 + c + 4 * j]);
                        at[4 * j] = q.x, at[4 * j + 1] = q.y, at[4 * j + 2] = q.z, at[4 * j + 3] = q.w;
                        all |= q.x | q.y | q.z | q.w;
                    }
                    uint8_t *y = static_cast<uint8_t *>(p.y) + (row - it.expert * matrix_rows) * 4;
                    const uint32_t pitch = (uint32_t)p.y_stride * 4;
                    const int last = in ? left : 0;
                    if (last >= 16 && all >= 0) {
#pragma unroll
                        for (int j = 0; j < 16; j++) *reinterpret_cast<float *>(y + (uint64_t)(uint32_t)at[j] * pitch) = x[j];
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; j++)
                            if (j < last && at[j] >= 0) *reinterpret_cast<float *>(y + (uint64_t)(uint32_t)at[j] * pitch) = x[j];
                    }
                } else if constexpr (F32) {
                    float *y = static_cast<float *>(p.y) + (it.t0 + c0 + c) * p.y_stride + row;
#pragma unroll
                    for (int j = 0; j < 16; j++, y += p.y_stride)
                        if (j < left && in) *y = x[j];
                } else if (l.pairs) {
                    // rows 2i and 2i + 1 meet: even lanes store both of a pair's first column, odd ones of the second
                    uint16_t *y = static_cast<uint16_t *>(p.y) + (it.t0 + c0 + c + (lane & 1)) * p.y_stride + (row & ~1);
                    const int mine_left = in ? left - (lane & 1) : 0;
#pragma unroll
                    for (int j = 0; j < 16; j += 2, y += 2 * p.y_stride) {
                        const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? x[j] : x[j + 1], 1);
                        const uint32_t two = lane & 1 ? bf16_pair(other, x[j + 1]) : bf16_pair(x[j], other);
                        if (j < mine_left) *reinterpret_cast<uint32_t *>(y) = two;
                    }
                } else {
                    __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(p.y) + (it.t0 + c0 + c) * p.y_stride + row;
#pragma unroll
                    for (int j = 0; j < 16; j++, y += p.y_stride)
                        if (j < left && in) *y = __float2bfloat16_rn(x[j]);
                }
            };
            if constexpr (F32) {
                uint64_t total[kCols / 2];   // pairs of columns
#pragma unroll
                for (int c = 0; c < kCols / 2; c++) total[c] = 0;
                const uint4 *ds = reinterpret_cast<const uint4 *>(p.scales + (in ? row : 0) * p.pitch) + k0 / GROUP / 8;
                const int groups = columns / GROUP;
                uint4 held = ds[0];   // eight groups' scales
                int part = k0 / GROUP % 8;
#pragma unroll 1
                for (int g = 0; g < groups; g++, turn++) {
                    const uint32_t two = part & 4 ? (part & 2 ? held.w : held.z) : (part & 2 ? held.y : held.x);
                    const float d = f16_bits_to_float((uint16_t)(part & 1 ? two >> 16 : two));
                    if (++part == 8 && g + 1 < groups) part = 0, held = *++ds;
                    wait(bar.d_full[turn & 1], turn >> 1);
                    tc_fence_after();
                    const uint64_t d2 = (uint64_t)__float_as_uint(d) << 32 | __float_as_uint(d);
#pragma unroll
                    for (int q = 0; q < kCols / 16; q++) {
                        if (16 * q >= mine) break;
                        uint64_t v[8];
                        tmem_ld16_pairs(at_lane + (turn & 1) * kTokens + 16 * q, v);
#pragma unroll
                        for (int c = 0; c < 8; c++) ffma2p(total[8 * q + c], v[c], d2);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.d_empty[turn & 1]);
                }
#pragma unroll
                for (int q = 0; q < kCols / 16; q++) {
                    if (16 * q >= mine) break;
                    float v[16];
#pragma unroll
                    for (int c = 0; c < 16; c++)
                        v[c] = __uint_as_float((uint32_t)(total[8 * q + c / 2] >> (32 * (c & 1))));
                    emit(16 * q, v);
                }
            } else {
                // 16 columns are asked for while the 16 before them go out (a small loop: results kept in
                // registers, to free the accumulator sooner, took code that pushed the other warps' out of the
                // instruction cache)
                const uint32_t mine_at = at_lane + turn % kBuffers * kTokens, which = turn % kBuffers;
                wait(bar.d_full[which], turn / kBuffers);
                turn++;
                tc_fence_after();
                auto leave = [&]() {   // another item may have the accumulator
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.d_empty[which]);
                };
                uint32_t a[16], b[16];
                auto out = [&](int c, uint32_t (&now)[16], uint32_t (&then)[16]) {
                    gm_ld_wait(now);
                    if (c + 16 < mine) gm_ld16_start(mine_at + c + 16, then);
                    else leave();
                    float v[16];
#pragma unroll
                    for (int j = 0; j < 16; j++) v[j] = __uint_as_float(now[j]);
                    emit(c, v);
                    __syncwarp();
                };
                if (mine > 0) gm_ld16_start(mine_at, a);
                else leave();
#pragma unroll 1
                for (int c = 0; c < mine; c += 32) {
                    out(c, a, b);
                    if (c + 16 < mine) out(c + 16, b, a);
                }
            }
            buf ^= 1;
            tell();
        }
        if constexpr (F32) {
            gm_fewer_registers<96>();
            named_sync(2, kGmThreads);
        }
    } else if (warp < kGmOutWarps + kGmExpandWarps) {
        // =================== weights: a thread per row, every other unit of two steps ===================
        if constexpr (F32) gm_fewer_registers<80>();
        if (starve) tries = wait_tries(l.fault);
        const int quarter = warp & 3, half = (warp - kGmOutWarps) >> 2;
        const uint32_t to = tmem + kGmABase + ((uint32_t)(quarter * 32) << 16);
        constexpr int kBlock = 8 * GROUP / 128;   // units of eight groups, whose scales are held
        // the lane's row of a stage of codes, under the 64-byte swizzle
        const int at = USE == kQ4Up ? (lane & 16) * 4 + quarter * 16 + (lane & 15) : quarter * 32 + lane;
        const uint32_t from = smem_u32(smem) + kGmStages * kGmB + at * 64, swizzle = (at >> 1) & 3;
        GmRing<kGmStages> ring;
        GmRing<kGmCStages> code;
        const int units = (steps + 1) / 2;
        uint32_t turn = 0;   // this CTA's units so far
        // Scales and zeros of eight groups are asked for before the eight before them are used, an item's first ones
        // during the item before it.
        const int u_begin = k0 / 128, end_block = (u_begin + units + kBlock - 1) / kBlock;
        uint4 d_next = make_uint4(0, 0, 0, 0);
        uint2 z_next = make_uint2(0, 0);
        int held = -1, next = 0, asked = -1;   // the item of d_next, the next block, the item that at_row is for
        int64_t at_row = 0;
        auto ask = [&](int i, int block) {
            if (i >= items) return;
            if (asked != i) {
                bool in;
                const int64_t row = row_of(item_of(i), quarter * 32 + lane, in);
                at_row = (in ? row : 0) * p.pitch;
                asked = i;
            }
            held = i;
            if (block >= end_block) return;   // (nothing of the item is this warp's)
            if (!F32) d_next = reinterpret_cast<const uint4 *>(p.scales + at_row)[block];
            if (ZEROS) z_next = reinterpret_cast<const uint2 *>(p.zeros + at_row)[block];
        };
        for (int i = begin; i < items; i += each) {
            const uint32_t parity = (half ^ turn) & 1;   // of the units that are this warp's
            next = (u_begin + (int)parity) / kBlock;
            if (held != i) ask(i, next);
            next++;
            GmRing<kGmStages> at_step = ring;
            GmRing<kGmCStages> at_code = code;
            at_step.next(2 * parity), at_code.next(parity);
            // the block of eight groups that is held: unit `uj` of it is next
            uint4 d8 = make_uint4(0, 0, 0, 0);
            uint2 z8 = make_uint2(0, 0);
            int uj = kBlock;
#pragma unroll 1
            for (int u = parity; u < units; u += 2) {
                if (uj >= kBlock) {
                    d8 = d_next, z8 = z_next;
                    uj = (u_begin + u) % kBlock;
                    if (next < end_block) ask(i, next++);
                    else ask(i + each, (u_begin + (int)((half ^ (turn + units)) & 1)) / kBlock);
                    // (a slice of K may begin inside a block)
                    for (int skip = uj / 2; skip > 0; skip--) q4_rotate<GROUP>(d8, z8);
                }
                const bool odd = uj & 1;
                wait(bar.c_full[at_code.i], at_code.phase);
                uint4 c[4];
#pragma unroll
                for (int h = 0; h < 4; h++)
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(c[h].x), "=r"(c[h].y), "=r"(c[h].z), "=r"(c[h].w)
                                 : "r"(from + at_code.i * kGmC + (h ^ swizzle) * 16)
                                 : "memory");
                // the scales (and zeros) of the unit's four chunks of 32 columns
                uint32_t d[4], z[4] = {8, 8, 8, 8};
                if (GROUP == 32) {
                    const uint32_t w0 = odd ? d8.z : d8.x, w1 = odd ? d8.w : d8.y, v = odd ? z8.y : z8.x;
                    d[0] = w0 & 0xffff, d[1] = w0 >> 16, d[2] = w1 & 0xffff, d[3] = w1 >> 16;
                    if (ZEROS) z[0] = v & 0xff, z[1] = v >> 8 & 0xff, z[2] = v >> 16 & 0xff, z[3] = v >> 24;
                } else if (GROUP == 64) {
                    const uint32_t w = odd ? d8.y : d8.x, v = odd ? z8.x >> 16 : z8.x;
                    d[0] = d[1] = w & 0xffff, d[2] = d[3] = w >> 16;
                    if (ZEROS) z[0] = z[1] = v & 0xff, z[2] = z[3] = v >> 8 & 0xff;
                } else {
                    d[0] = d[1] = d[2] = d[3] = odd ? d8.x >> 16 : d8.x & 0xffff;
                    if (ZEROS) z[0] = z[1] = z[2] = z[3] = (odd ? z8.x >> 8 : z8.x) & 0xff;
                }
                q4_rotate<GROUP>(d8, z8);
                uj += 2;
#pragma unroll
                for (int s = 0; s < 2; s++) {
                    if (2 * u + s >= steps) break;
                    uint32_t v[32];
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const int q = 2 * s + h;
                        const __half2 low = half2_of(0x64006400u + z[q] * 0x10001u);   // 1024 + z
                        // -(64 + z), whose last place is 2^-4
                        const __half2 high = half2_of(0xD400D400u + z[q] * 0x00100010u);
                        const __half2 scale = half2_of(d[q] * 0x10001u);
                        expand_f16<!F32>(c[q].x, low, high, scale, v + 16 * h);
                        expand_f16<!F32>(c[q].y, low, high, scale, v + 16 * h + 4);
                        expand_f16<!F32>(c[q].z, low, high, scale, v + 16 * h + 8);
                        expand_f16<!F32>(c[q].w, low, high, scale, v + 16 * h + 12);
                    }
                    if ((2 * u + s) * kGmStep + 32 >= columns)   // K ends after half a step
#pragma unroll
                        for (int e = 16; e < 32; e++) v[e] = 0;
                    wait(bar.empty[at_step.i], at_step.phase ^ 1);
                    tc_fence_after();
                    gm_tmem_st16(to + at_step.i * 32, v);
                    gm_tmem_st16(to + at_step.i * 32 + 16, v + 16);
                    if (s == 0 && lane == 0) mbar_arrive(&bar.c_empty[at_code.i]);   // (all lanes have theirs: wait)
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.full[at_step.i]);
                    at_step.next();
                }
                at_step.next(2), at_code.next(2);
            }
            turn += units;
            ring.skip(steps);
            code.skip(units);
        }
        __syncwarp();
        if constexpr (F32) {
            named_sync(2, kGmThreads);
            gm_more_registers<96>();
        }
    } else {
      if constexpr (F32) gm_fewer_registers<32>();
      if (warp == kGmCodeWarp) {
        // =================== codes: two copies of 64 rows x 128 columns a stage ===================
        GmRing<kGmCStages> code;
        int used = 0;
        for (int i = begin; i < items && !starve; i += each) {
            const GmItem it = item_of(i);
            const int64_t first = it.expert * matrix_rows + it.tile * (int64_t)(USE == kQ4Up ? kGmRows / 2 : kGmRows);
            const int64_t second = USE == kQ4Up ? first + p.N : first + kGmRows / 2;
#pragma unroll 1
            for (int s = 0; s < steps; s += 2) {
                wait(bar.c_empty[code.i], code.phase ^ 1);
                if (gm_elect()) {
                    uint8_t *dst = smem + kGmStages * kGmB + code.i * kGmC;
                    uint64_t *b = &bar.c_full[code.i];
                    mbar_arrive_expect_tx(b, kGmC);
                    tma_load_2d(dst, &code_map, (k0 + s * kGmStep) / 2, (int)first, b);
                    tma_load_2d(dst + kGmC / 2, &code_map, (k0 + s * kGmStep) / 2, (int)second, b);
                }
                __syncwarp();
                code.next();
                used = min(used + 1, kGmCStages);
            }
        }
        // no copy may still be landing when the CTA exits
        for (int n = 0; n < used; n++) {
            if (code.i == 0) code.i = kGmCStages, code.phase ^= 1;
            code.i--;
            wait(bar.c_full[code.i], code.phase);
        }
    } else if (warp == kGmCopyWarp) {
        // =================== x ===================
        GmRing<kGmStages> ring;
        int used = 0;
        for (int i = begin; i < items; i += each) {
            const GmItem it = item_of(i);
            const int boxes = (it.tokens + l.box - 1) / l.box;
            const uint32_t bytes = (uint32_t)(kParts * boxes * l.box * 128);
#pragma unroll 1
            for (int s = 0; s < steps; s++) {
                wait(bar.empty[ring.i], ring.phase ^ 1);
                // (one thread issues everything: copies of several lanes go out one after the other, slower)
                if (gm_elect()) {
                    uint64_t *b = &bar.full[ring.i];
                    mbar_arrive_expect_tx(b, bytes);
                    const int byte = (k0 + s * kGmStep) * 2;
                    for (int box = 0; box < boxes; box++) {
#pragma unroll
                        for (int part = 0; part < kParts; part++) {
                            uint8_t *to = smem + ring.i * kGmB + part * (kGmB / 2) + box * l.box * 128;
                            const int row = part * (int)r.rows + it.t0 + box * l.box;
                            tma_load_2d(to, &x_map, byte, row, b);
                        }
                    }
                }
                __syncwarp();
                ring.next();
                used = min(used + 1, kGmStages);
            }
        }
        // no copy may still be landing when the CTA exits
        for (int n = 0; n < used; n++) {
            if (ring.i == 0) ring.i = kGmStages, ring.phase ^= 1;
            ring.i--;
            wait(bar.full[ring.i], ring.phase);
        }
    } else if (warp == kGmMmaWarp) {
        // =================== tensor-core operations ===================
        GmRing<kGmStages> ring;
        uint32_t taken = 0;   // accumulators
        for (int i = begin; i < items; i += each) {
            const GmItem it = item_of(i);
            const uint32_t idesc = idesc_f16(kGmRows, (it.tokens + 15) / 16 * 16);
            const uint32_t which = taken % kBuffers, at_d = tmem + which * kTokens;
            if (!F32) wait(bar.d_empty[which], (taken / kBuffers) ^ 1);
#pragma unroll 1
            for (int s = 0; s < steps; s++) {
                wait(bar.full[ring.i], ring.phase);
                tc_fence_after();
                const uint32_t a = tmem + kGmABase + ring.i * 32, b = gm_desc_low(smem_u32(smem) + ring.i * kGmB);
                if constexpr (!F32) {
                    if (gm_elect()) {
                        gm_mma4(at_d, a, b, idesc, s > 0);
                        mma_commit(&bar.empty[ring.i]);
                    }
                } else {
                    constexpr int kTurns = GROUP == 32 ? 2 : 1;   // accumulators of a step
#pragma unroll
                    for (int h = 0; h < kTurns; h++) {
                        if (s * kGmStep + 32 * h >= columns) break;
                        const bool begin = GROUP < 128 || s % 2 == 0;
                        const uint32_t buf = taken & 1, d = tmem + buf * kTokens;
                        if (begin) {
                            wait(bar.d_empty[buf], (taken >> 1) ^ 1);
                            tc_fence_after();
                        }
                        if (gm_elect()) {
                            if (GROUP == 32) {
                                gm_mma2(d, a + 16 * h, b + 4 * h, idesc, 0);
                                gm_mma2(d, a + 16 * h, b + 4 * h + (kGmB / 2 >> 4), idesc, 1);
                            } else {
                                gm_mma4(d, a, b, idesc, !begin);
                                gm_mma4(d, a, b + (kGmB / 2 >> 4), idesc, 1);
                            }
                            if (GROUP < 128 || s % 2 == 1) mma_commit(&bar.d_full[buf]);
                        }
                        if (GROUP < 128 || s % 2 == 1) taken++;
                        __syncwarp();
                    }
                    if (gm_elect()) mma_commit(&bar.empty[ring.i]);
                }
                __syncwarp();
                ring.next();
            }
            if (!F32) {
                if (gm_elect()) mma_commit(&bar.d_full[which]);
                __syncwarp();
                taken++;
            }
        }
        if (gm_elect()) mma_commit(&bar.done);
        __syncwarp();
        wait(bar.done, 0);
        tc_fence_before();
      }
      __syncwarp();
      if constexpr (F32) {
          named_sync(2, kGmThreads);
          gm_more_registers<96>();
      }
    }
    __syncthreads();
    tc_fence_after();
    if constexpr (USE == kQ4Dense) {
        if (l.split > 1) {
            // one item per cluster: its parts' sums, a share of the columns per CTA, a warp per column
            gm_cluster_sync();
            if (begin < items) {
                const GmItem it = item_of(begin);
                const float *park = reinterpret_cast<const float *>(smem);
                for (int c = rank + l.split * warp; c < it.tokens; c += l.split * kGmWarps) {
                    const float scale = col_scale[0][c];
                    T *y = static_cast<T *>(p.y) + col_row[0][c] * p.y_stride;
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const int at = j * 32 + lane;
                        float v = 0.f;
                        for (int q = 0; q < l.split; q++) v += gm_cluster_load(park + c * kGmRows + at, q);
                        bool in;
                        const int64_t row = row_of(it, at, in);
                        if (in) gm_store(y + row, v * scale);
                    }
                }
            }
            gm_cluster_sync();
        }
    }
    if (warp == kGmMmaWarp) tmem_dealloc(tmem, 512);
}

template <Q4Use USE, typename T, int TOKENS, int GROUP>
static int launch_gemm(const CUtensorMap &code_map, const CUtensorMap &x_map, const Q4Params &p, const Q4Rows &r,
                       const GmLaunch &l, unsigned grid, cudaStream_t st) {
    auto kernel = p.zeros ? q4_gemm_kernel<USE, T, TOKENS, GROUP, true> : q4_gemm_kernel<USE, T, TOKENS, GROUP, false>;
    constexpr int kSmem = GmShape<TOKENS, sizeof(T) == 4 ? 2 : 1>::kSmem;
    int per_sm;
    if (int e = prepare_kernel((const void *)kernel, kGmThreads, kSmem, &per_sm)) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid), cfg.blockDim = dim3(kGmThreads), cfg.dynamicSmemBytes = kSmem, cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)l.split, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr, cfg.numAttrs = l.split > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, code_map, x_map, p, r, l);
    if (e == cudaSuccess) return LB_OK;
    record_cuda_error(e);
    return LB_ERR_LAUNCH;
}

template <Q4Use USE, typename T, int TOKENS>
static int dispatch_gemm(const Q4Params &p, const Q4Rows &r, const uint8_t *codes, int64_t code_rows, int sms,
                         cudaStream_t st) {
    const int rows = USE == kQ4Up ? kGmRows / 2 : kGmRows;
    GmLaunch l;
    const int64_t tiles = (p.N + rows - 1) / rows, pieces = (p.T + TOKENS - 1) / TOKENS;
    l.tokens = (int)((p.T + pieces - 1) / pieces + 15) / 16 * 16;
    l.tiles = (int)tiles;
    const int steps = (p.K + kGmStep - 1) / kGmStep;
    l.split = 1, l.steps = steps;
    l.pairs = p.N % 2 == 0 && p.y_stride % 2 == 0 && aligned_to(p.y, 4);
    l.box = p.T <= 16 ? 16 : p.T <= 32 ? 32 : TOKENS / 2;   // (small items need one of the two)
    int64_t items = tiles * pieces;
    if (USE != kQ4Dense) items = tiles * std::min(p.T, std::min((int64_t)p.E, p.T) + p.T / TOKENS);
    if (USE == kQ4Dense && items * 2 <= sms) {
        // slices of an even number of steps (whole groups), at least four
        l.split = (int)std::min<int64_t>({(int64_t)sms / items, (int64_t)kGmMaxSplit, (int64_t)std::max(steps / 4, 1)});
        l.steps = (steps + l.split - 1) / l.split;
        l.steps = (l.steps + 1) / 2 * 2;
        l.split = (steps + l.steps - 1) / l.steps;
    }
    l.fault = take_injected_wait_fault();
    const unsigned grid = (unsigned)(l.split > 1 ? items * l.split : std::min<int64_t>(items, sms));
    CUtensorMap codes_map, x_map;
    if (int e = encode_rows_map(&codes_map, codes, (uint64_t)p.K / 2, (uint64_t)code_rows, 64, kGmRows / 2, 64)) return e;
    if (int e = encode_rows_map(&x_map, r.x, (uint64_t)p.K * 2, (uint64_t)r.rows * (sizeof(T) == 4 ? 2 : 1), 128,
                                (uint32_t)l.box, 128))
        return e;
    switch (p.group) {
        case 32: return launch_gemm<USE, T, TOKENS, 32>(codes_map, x_map, p, r, l, grid, st);
        case 64: return launch_gemm<USE, T, TOKENS, 64>(codes_map, x_map, p, r, l, grid, st);
        default: return launch_gemm<USE, T, TOKENS, 128>(codes_map, x_map, p, r, l, grid, st);
    }
}

}  // namespace lb
