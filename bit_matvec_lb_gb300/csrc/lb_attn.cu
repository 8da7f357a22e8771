// lb_attn.cu -- attention over the paged 4-bit key/value cache for requests with few query rows
// (decode, verification of drafted tokens), and the entry point.
#include "lb_attn.cuh"

#include <float.h>
#include <math.h>

namespace lb {

// ------------------------------------------------------------------------------------------
// Mathematics.  For one key/value head, the rows that read it (queries x heads of the group) are
// the columns of two products with the code matrices: with k_t = kd_t (kc_t - kz_t),
//   s_t = scale * kd_t * (sum_i q_i kc_ti - kz_t sum_i q_i),
//   out = sum_t p_t vd_t (vc_t - vz_t) / sum_t p_t,   p_t = 2^(s_t log2 e - R),
// so codes enter the tensor cores as whole numbers, exact in fp16, and the scales act on the scores
// and weights.  R runs over max_t(s_t + log2 vd_t), which bounds the
// weights w_t = p_t vd_t themselves (not the p_t): they enter the second product as fp16 in
// [0, 2^15], whatever the sizes of the scales.
//
// Bound: reading the cache (D + 8 bytes per token and head), and close to it the integer pipe.  A code
// costs 5/8 (keys) or 3/4 (values) of an integer operation to become fp16: masked in place, 4-bit
// fields at bits 0 and 16 of a word are the mantissas' last bits of an fp16 pair, at bits 4 and 20
// the next four.  Two neighbouring tokens' words are interleaved by 16 bits to pair tokens for the
// second product.  mma.sync serves here: rows are 8 to 16 wide, the products
// are a third of the issue slots at full bandwidth, and tcgen05 would need the fp16 codes written
// to shared memory, four times the cache's bytes.
//
// Items (request, head, 4 to 16 rows) are cut into equal runs of tiles over the CTAs, three per SM by
// registers; each warp keeps kStages tiles in flight and its own sums, which the CTA merges.  Of a
// call that splits its items over all CTAs about 11 us are fixed (launches, requests and pages, first
// tiles, merge, join; calls with less work skip some of it and take 5 us or more in all); beyond 131k
// tokens more ones are read at 5.6 TB/s.  Measured (32 / 8 heads of 128): one request of 131k
// tokens in bf16 37 us (3.9 TB/s), 64 requests of 4096 tokens 68 us in bf16 (4.2 TB/s) and 73 in fp32.
// ------------------------------------------------------------------------------------------
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 32;            // tokens of one warp step (two chunks)
constexpr int kStages = 4;           // tiles in flight per warp
// Items of at most kWhole tiles are never split (64 / 256 requests of 300 tokens: 14 / 37 us, split
// 20 / 52), nor are those of half a CTA's run or less, up to kWholeMost (256 requests of 700 tokens: 58
// against 67 us; one of 1000 tokens, whose run is 4 tiles: split 8.2, whole 12.1; 33 requests of up to
// 1000 tokens and 20 rows, whose run is 31: split 28, those below it whole 30).
constexpr int kWhole = 16, kWholeMost = 28;
// Tiles per CTA below which no more CTAs are used (one request of 127 / 2047 / 4095 tokens with 4:
// 5.1 / 8.5 / 9.9 us, 8: 7.4 / 9.0 / 9.6, 2: 5.2 / 9.5 / 11.3).
constexpr int kMinRun = 4;
constexpr int kMaxCtas = 608;
// Query rows per head up to which this file's kernel is used.  32 requests of 1000 tokens, us here
// against the other:  rows         24         32         40         48
//      128 dimensions, bf16     38 / 58    44 / 58    57 / 58    59 / 58
//                      fp32     54 / 74    68 / 75    81 / 75    91 / 76
//      64 dimensions,  bf16     31 / 57    35 / 58    45 / 58    46 / 58
//                      fp32     39 / 68    48 / 68    58 / 69    65 / 69
// and one of 30000 tokens alike (128, bf16: 32 / 41 at 32 rows, 45 / 42 at 40).  One bound for all:
// 64 dimensions would take this kernel up to 48 rows, too (bf16: a fifth of the time).
constexpr int kFewRows = 32;
// Batches this small run as one launch.  The host knows neither the lengths nor how many of the
// requests have few rows, so the rule sees their number alone: it saves the second launch and its
// join for prompts and short contexts and costs decode requests of long contexts beside a prompt
// whole row tiles.  us in one launch against two, bf16 (fp32):
//      three chunks of 500 queries, no decode       72 /  79  (104 / 109)
//      beside a chunk of 256, decode contexts of
//               300 tokens: 3 requests 18 / 27 (25 / 36),    7  18 /  29 (25 /  38),  11  24 /  29  (36 /  38)
//              1000                    23 / 35 (31 / 42),       33 /  41 (47 /  47),      38 /  43  (55 /  49)
//              4000                    35 / 41 (51 / 48),       49 /  47 (75 /  54),      69 /  53 (104 /  59)
//             32000                   126 / 71 (198 / 77),     258 / 114 (408 / 117),    380 / 154 (597 / 156).
constexpr int kFewRequests = 8;
constexpr float kLift = 256.f;       // weights are lifted by 2^8 ...
constexpr float kSlack = 7.f;        // ... and may pass the reference by 2^7 before it moves

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// c += a * b.  FRESH: the product is summed from zero and added in binary32, rounded to nearest (the
// tensor cores would cut the sum downwards at every step: fp32, 192k tokens, 8 rows 3.7e-6 in norm).
template <bool FRESH>
__device__ __forceinline__ void mma_add(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    if (FRESH) {
        float t[4] = {};
        mma16816(t, a0, a1, a2, a3, b0, b1);
#pragma unroll
        for (int e = 0; e < 4; e++) c[e] += t[e];
    } else {
        mma16816(c, a0, a1, a2, a3, b0, b1);
    }
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Four fp16 pairs of a word of eight codes, by pairs of places {0,4}, {1,5}, {2,6}, {3,7}: as
// subnormals, c * 2^-24 and, the odd pairs, 16 c * 2^-24, or (NORMAL) c - 8 as normal numbers, by
// the mantissas of 1024 and 64.  The tensor cores align a product by its factors' exponent fields and
// cut, downwards, what lies below the last place of a sum's largest term; subnormal factors lose ten
// of its 24 bits that way.  Values are always normal: sums over thousands of tokens nearly cancel
// (131k tokens with subnormals: 3e-5 of an output, with normal numbers 7e-7).  Keys are with fp32
// tensors; with bf16 ones the cut is alike for all tokens and far below the outputs' rounding, and
// the subtraction would cost a tenth.
template <bool NORMAL>
__device__ __forceinline__ void spread_codes(uint32_t w, uint32_t (&x)[4]) {
    const uint32_t h = w >> 8;
    if (NORMAL) {
        asm("lop3.b32 %0, %1, 0x000F000F, 0x64006400, 0xEA;" : "=r"(x[0]) : "r"(w));
        asm("lop3.b32 %0, %1, 0x00F000F0, 0x54005400, 0xEA;" : "=r"(x[1]) : "r"(w));
        asm("lop3.b32 %0, %1, 0x000F000F, 0x64006400, 0xEA;" : "=r"(x[2]) : "r"(h));
        asm("lop3.b32 %0, %1, 0x00F000F0, 0x54005400, 0xEA;" : "=r"(x[3]) : "r"(h));
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const __half2 less = __half2half2(__ushort_as_half(e & 1 ? 0x5480 : 0x6408));  // 72, 1032
            const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&x[e]), less);
            x[e] = *reinterpret_cast<const uint32_t *>(&v);
        }
    } else {
        x[0] = and_imm<0x000F000Fu>(w);
        x[1] = and_imm<0x00F000F0u>(w);
        x[2] = and_imm<0x000F000Fu>(h);
        x[3] = and_imm<0x00F000F0u>(h);
    }
}
template <int D, int SPLIT, int NT>
struct Decode {
    static constexpr int kCols = 8 * NT / SPLIT;   // query rows of one item
    static constexpr int kChunk = kv4_chunk_bytes(D);
    static constexpr int kStage = 2 * kChunk;
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kMerge = kWarps * kCols * (D + 4) * 4;
    static constexpr size_t kSmem = kRing > kMerge ? kRing : kMerge;
};

// Work of one request in units of one tile of one item (an item: one key/value head and up to
// kCols rows); at least one tile, so that rows that see nothing are visited and written.
struct Units {
    int lo, hi;    // visible tokens
    int t0, tiles; // first tile, tiles
    int groups;    // items per head
};

template <int COLS>
__device__ __forceinline__ int64_t request_units(const AttnParams &p, const Request &q, Units &u) {
    visible_range(p, q, 0, q.n, u.lo, u.hi);
    u.t0 = u.lo / kTile;
    u.tiles = max((u.hi + kTile - 1) / kTile - u.t0, 1);
    u.groups = (q.n * p.group + COLS - 1) / COLS;
    return (int64_t)u.tiles * u.groups * p.kv_heads;
}

template <int D, typename T, int SPLIT, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2) attn_decode_kernel(const AttnParams p) {
    using C = Decode<D, SPLIT, NT>;
    constexpr int COLS = C::kCols;
    constexpr int W = D / 32;             // words of eight codes per thread and key row
    constexpr int VW = D / 64;            // words of eight codes per thread and value row
    constexpr bool NORMAL = sizeof(T) == 4;  // key codes; what they are of themselves in the products
    constexpr float UNIT = NORMAL ? 1.f : 1.f / 16777216.f, ODD = NORMAL ? 1.f : 16.f, LESS = NORMAL ? 8.f : 0.f;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[kWarps][kStages];
    __shared__ int64_t scan[kWarps];
    __shared__ int64_t s_start;
    __shared__ int s_r;
    __shared__ float m_ref[kWarps][COLS], m_sum[kWarps][COLS], m_zero[kWarps][COLS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, tg = lane & 3;

    if (lane < kStages) mbar_init(&full[warp][lane], 1);
    fence_mbar_init();
    pdl_wait();
    pdl_launch_dependents();

    // ---- this CTA's run of units [u0, u1) and the request it begins in ----
    int64_t mine = 0;
    const int run = (p.R + kThreads - 1) / kThreads;
    const int ra = min(tid * run, p.R), rb = min(ra + run, p.R);
    Units un;
    for (int r = ra; r < rb; r++) mine += request_units<COLS>(p, load_request(p, r), un);
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
    for (int w = 0; w < kWarps; w++) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    const int64_t ctas = min((int64_t)gridDim.x, (total + kMinRun - 1) / kMinRun);
    int4 *record = p.record + 2 * blockIdx.x;
    if (tid < 2) record[tid] = make_int4(-1, 0, 0, 0);
    if (blockIdx.x >= ctas) return;
    const int unsplit = (int)max((int64_t)kWhole, min((int64_t)kWholeMost, total / (2 * ctas)));
    const int64_t u0 = total * blockIdx.x / ctas, u1 = total * (blockIdx.x + 1) / ctas;
    if (before <= u0 && u0 < before + mine) {
        int64_t at = before;
        for (int r = ra; r < rb; r++) {
            const int64_t n = request_units<COLS>(p, load_request(p, r), un);
            if (u0 < at + n) {
                s_r = r, s_start = at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();

    uint32_t count = 0;        // tiles this warp has taken from its ring, over all items
    uint64_t limit = 2000000000ull;
    uint8_t *ring = smem + warp * (kStages * C::kStage);
    int r = s_r;
    Request rq = load_request(p, r);
    int64_t r_units = request_units<COLS>(p, rq, un), r_begin = s_start;

    for (int64_t u = u0; u < u1;) {
        while (u >= r_begin + r_units) {  // requests without work have no units
            r_begin += r_units;
            rq = load_request(p, ++r);
            r_units = request_units<COLS>(p, rq, un);
        }
        const int item = (int)((u - r_begin) / un.tiles);
        const int first = (int)((u - r_begin) - (int64_t)item * un.tiles);  // tile within the item
        int last = (int)min((int64_t)un.tiles, first + (u1 - u));
        u += last - first;
        if (un.tiles <= unsplit) {  // never split: the CTA in whose run it begins takes it
            if (first > 0) continue;
            last = un.tiles;
        }
        const int h = item / un.groups, col0 = item % un.groups * COLS;
        const int ncol = min(COLS, rq.n * p.group - col0);

        // ---- query columns: this thread's D / 4 dimensions of column g, asked for before the
        // copies, behind which they would wait in the memory's queues ----
        float qx[NT][8 * W];
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            const int c = SPLIT == 2 ? nt * 4 + g / 2 : nt * 8 + g;
            const int cc = col0 + (c < ncol ? c : 0);
            const int qi = cc / p.group, head = h * p.group + cc % p.group;
            const T *src = static_cast<const T *>(p.q) + (int64_t)(rq.q0 + qi) * p.q_stride +
                           (int64_t)head * D + tg * (D / 4);
#pragma unroll
            for (int i = 0; i < W; i++) {
                float y[8];
                load8(src + 8 * i, y);
#pragma unroll
                for (int e = 0; e < 8; e++) qx[nt][8 * i + e] = c < ncol ? y[e] : 0.f;
            }
        }

        // ---- pages and first copies ----
        const int n = last - first - warp;                  // this warp: tiles first + warp + 4 i
        const int tiles = n > 0 ? (n + kWarps - 1) / kWarps : 0;
        int pg0 = -1, pg1 = -1, pg_base = -32;
        uint32_t valid = 0;                                 // two bits per stage
        const int64_t page_bytes = ((int64_t)p.kv_heads << (p.shift - 4)) * C::kChunk;
        const uint8_t *head_base = p.cache + ((int64_t)h << (p.shift - 4)) * C::kChunk;
        auto tile_token = [&](int i) { return (un.t0 + first + warp + kWarps * i) * kTile; };
        auto load_pages = [&](int base) {
            pg_base = base;
            const int j = tile_token(base + lane);
            const int64_t c0 = j >> p.shift, c1 = (j + 16) >> p.shift;
            const int32_t *row = p.table + (int64_t)r * p.width;
            pg0 = base + lane < tiles && c0 < p.width ? row[c0] : -1;
            pg1 = c1 == c0 ? pg0 : base + lane < tiles && c1 < p.width ? row[c1] : -1;
        };
        auto issue = [&](int i) {  // tile i of this warp into stage (count + i) % kStages
            const uint32_t slot = count + i;
            const int stage = slot % kStages, j = tile_token(i);
            const int a = __shfl_sync(0xffffffffu, pg0, i - pg_base);
            const int b = __shfl_sync(0xffffffffu, pg1, i - pg_base);
            const bool va = a >= 0 && a < p.pages && j < un.hi && j + 16 > un.lo;
            const bool vb = b >= 0 && b < p.pages && j + 16 < un.hi && j + 32 > un.lo;
            valid = (valid & ~(3u << (2 * stage))) | ((uint32_t)va | (uint32_t)vb << 1) << (2 * stage);
            if (lane == 0) {
                uint8_t *dst = ring + stage * C::kStage;
                uint64_t *bar = &full[warp][stage];
                const int in = j & ((1 << p.shift) - 1);
                mbar_arrive_expect_tx(bar, ((int)va + (int)vb) * C::kChunk);
                if (va) {
                    bulk_g2s(dst, head_base + a * page_bytes + (in >> 4) * C::kChunk,
                             vb && p.shift > 4 ? 2 * C::kChunk : C::kChunk, bar);
                }
                if (vb && !(va && p.shift > 4))
                    bulk_g2s(dst + C::kChunk,
                             head_base + b * page_bytes + (p.shift > 4 ? (in >> 4) + 1 : 0) * C::kChunk,
                             C::kChunk, bar);
            }
        };
        if (tiles > 0) load_pages(0);
        for (int i = 0; i < min(tiles, kStages); i++) issue(i);

        // ---- fp16 parts of the queries, and the columns' constants ----
        uint32_t qb[NT][2 * W][2];
        float col_a[NT][2], col_sum[NT][2];  // of the columns 2 tg, 2 tg + 1 (SPLIT: parts of one)
        int col_hi[NT][2], col_lo[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            const int part = SPLIT == 2 ? g & 1 : 0;
            const int c = SPLIT == 2 ? nt * 4 + g / 2 : nt * 8 + g;
            const int qi = (col0 + (c < ncol ? c : 0)) / p.group;
            float(&x)[8 * W] = qx[nt];
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < 8 * W; i++) amax = fmaxf(amax, fabsf(x[i]));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            float up, down, sum = 0.f;
            row_power(amax, up, down);
#pragma unroll
            for (int i = 0; i < 8 * W; i++) {
                x[i] *= up;
                sum += x[i];
                if (part) x[i] -= __half2float(__float2half_rn(x[i]));
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
            for (int i = 0; i < W; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float s = e & 1 ? 1.f / ODD : 1.f;
                    qb[nt][2 * i + e / 2][e & 1] = half2_bits(x[8 * i + e] * s, x[8 * i + e + 4] * s);
                }
            // (finite for the largest queries too: keys whose scale is 0 score 0)
            const float a = fminf(p.scale * kLog2e * down * (1.f / UNIT), FLT_MAX);
            sum *= UNIT;
            int hi = un.hi;
            if (p.causal) hi = min(hi, rq.base + qi + 1);
            const int lo = window_start(p, rq, qi);
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int from = (2 * tg + e) * 4;
                col_a[nt][e] = __shfl_sync(0xffffffffu, a, from);
                col_sum[nt][e] = __shfl_sync(0xffffffffu, sum, from);
                col_hi[nt][e] = __shfl_sync(0xffffffffu, hi, from);
                col_lo[nt][e] = __shfl_sync(0xffffffffu, lo, from);
            }
        }
        // Tokens that every column sees: no mask in a tile inside them.
        int all_hi = un.hi;
        if (p.causal) all_hi = min(all_hi, rq.base + col0 / p.group + 1);
        const int all_lo = window_start(p, rq, (col0 + ncol - 1) / p.group);

        float o[D / 16][NT][4];
        float ref[NT][2], base[NT][2], sum[NT][2], zero[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
#pragma unroll
            for (int m = 0; m < D / 16; m++)
#pragma unroll
                for (int e = 0; e < 4; e++) o[m][nt][e] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; e++) ref[nt][e] = -INFINITY, base[nt][e] = sum[nt][e] = zero[nt][e] = 0.f;
        }

        for (int i = 0; i < tiles; i++) {
            const int stage = count % kStages;
            if (!mbar_wait(&full[warp][stage], (count / kStages) & 1, limit)) {
                *p.error = 1;
                limit = 1000000ull;
            }
            const int j0 = tile_token(i);
            const uint32_t bits = (valid >> (2 * stage)) & 3u;
            const bool inside = bits == 3u && j0 >= all_lo && j0 + kTile <= all_hi;
            const uint8_t *tile = ring + stage * C::kStage;
            // Row g of the first product is token g ^ (bit 1 of g) of a chunk, so that both the key
            // rows of eight lanes and the value rows of 16 lanes lie in different banks (or two).
            const int tok = g ^ ((g >> 1) & 1);
            constexpr int E = SPLIT == 2 ? 1 : 2;
            // Tokens of this thread: 2 * half and 2 * half + 1 are tok and tok + 8 of a chunk.
            float2 kd[4], vd[4];
            float s[NT][E][4];
#pragma unroll
            for (int half = 0; half < 2; half++) {
                const uint8_t *chunk = tile + half * C::kChunk;
                const __half2 *kp = reinterpret_cast<const __half2 *>(chunk + 2 * kv4_codes_bytes(D));
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    kd[2 * half + e] = __half22float2(kp[tok + 8 * e]);
                    vd[2 * half + e] = __half22float2(kp[LB_KV4_CHUNK + tok + 8 * e]);
                }
                float acc[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int e = 0; e < 4; e++) acc[nt][e] = 0.f;
                uint32_t wa[W], wb[W];
                const uint8_t *row = chunk + tok * (D / 2) + tg * (D / 8);
                if (D == 128) {
                    const uint4 a = *reinterpret_cast<const uint4 *>(row);
                    const uint4 b = *reinterpret_cast<const uint4 *>(row + 8 * (D / 2));
                    wa[0] = a.x, wa[1] = a.y, wa[W - 2] = a.z, wa[W - 1] = a.w;
                    wb[0] = b.x, wb[1] = b.y, wb[W - 2] = b.z, wb[W - 1] = b.w;
                } else {
                    const uint2 a = *reinterpret_cast<const uint2 *>(row);
                    const uint2 b = *reinterpret_cast<const uint2 *>(row + 8 * (D / 2));
                    wa[0] = a.x, wa[1] = a.y, wb[0] = b.x, wb[1] = b.y;
                }
#pragma unroll
                for (int k = 0; k < W; k++) {
                    uint32_t xa[4], xb[4];
                    spread_codes<NORMAL>(wa[k], xa);
                    spread_codes<NORMAL>(wb[k], xb);
#pragma unroll
                    for (int nt = 0; nt < NT; nt++) {
                        mma16816(acc[nt], xa[0], xb[0], xa[1], xb[1], qb[nt][2 * k][0], qb[nt][2 * k][1]);
                        mma16816(acc[nt], xa[2], xb[2], xa[3], xb[3], qb[nt][2 * k + 1][0],
                                 qb[nt][2 * k + 1][1]);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int e = 0; e < E; e++) {
                        s[nt][e][2 * half] = SPLIT == 2 ? acc[nt][0] + acc[nt][1] : acc[nt][e];
                        s[nt][e][2 * half + 1] = SPLIT == 2 ? acc[nt][2] + acc[nt][3] : acc[nt][2 + e];
                    }
            }
            int tj[4];
            if (!inside) {  // what lies behind the request's end is not read as a number
#pragma unroll
                for (int x = 0; x < 4; x++) {
                    tj[x] = bits >> (x / 2) & 1 ? j0 + 16 * (x / 2) + 8 * (x & 1) + tok : 0x7fffffff;
                    if (tj[x] >= un.hi) kd[x] = vd[x] = make_float2(0.f, 0.f);
                }
            }
            // Scores in powers of two, and the bound of the weights' size.
            float vl[4];
            bool move = false;
#pragma unroll
            for (int x = 0; x < 4; x++) vl[x] = scale_log2(vd[x].x);
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int e = 0; e < E; e++) {
                    float top = -INFINITY;
#pragma unroll
                    for (int x = 0; x < 4; x++) {
                        float y = (kd[x].x * col_a[nt][e]) * fmaf(LESS - kd[x].y, col_sum[nt][e], s[nt][e][x]);
                        if (!inside && (tj[x] >= col_hi[nt][e] || tj[x] < col_lo[nt][e])) y = -INFINITY;
                        s[nt][e][x] = y;
                        top = fmaxf(top, y + vl[x]);
                    }
                    move |= top > ref[nt][e] + kSlack;
                }
            if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int e = 0; e < E; e++) {
                        float m = ref[nt][e];
#pragma unroll
                        for (int x = 0; x < 4; x++) m = fmaxf(m, s[nt][e][x] + vl[x]);
#pragma unroll
                        for (int k = 4; k < 32; k <<= 1)
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
                        const float f = m == ref[nt][e] ? 1.f : ex2(ref[nt][e] - m);
                        ref[nt][e] = m;
                        // a column that has seen nothing yet: any finite base gives weights of 0
                        base[nt][e] = m == -INFINITY ? 0.f : m;
                        sum[nt][e] *= f, zero[nt][e] *= f;
#pragma unroll
                        for (int d = 0; d < D / 16; d++) {
                            o[d][nt][e] *= f, o[d][nt][2 + e] *= f;
                            if (SPLIT == 2) o[d][nt][1] *= f, o[d][nt][3] *= f;
                        }
                    }
            }
            uint32_t pb[NT][4];
#pragma unroll
            for (int x = 0; x < 4; x++) {
                const float lift = vd[x].x * kLift;
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    float w[2];
#pragma unroll
                    for (int e = 0; e < E; e++) {
                        const float pr = ex2(s[nt][e][x] - base[nt][e]);
                        sum[nt][e] += pr;
                        w[e] = pr * lift;
                    }
                    __half2 q2;
                    if (SPLIT == 2) {  // two parts: the second holds what rounding took from the first
                        const __half hi = __float2half_rn(w[0]);
                        q2 = __halves2half2(hi, __float2half_rn(w[0] - __half2float(hi)));
                        zero[nt][0] = fmaf(w[0], vd[x].y - 8.f, zero[nt][0]);
                    } else {
                        // The zero's share uses the weights as rounded, so that an error of a
                        // weight acts on d (c - z), not on d c and d z apart.
                        q2 = __floats2half2_rn(w[0], w[1]);
                        const float2 f = __half22float2(q2);
                        zero[nt][0] = fmaf(f.x, vd[x].y - 8.f, zero[nt][0]);
                        zero[nt][E - 1] = fmaf(f.y, vd[x].y - 8.f, zero[nt][E - 1]);
                    }
                    pb[nt][x] = transpose8x8(*reinterpret_cast<const uint32_t *>(&q2));
                }
            }
            // Second product: this thread's dimensions g * D/8 .. of tokens (k order) 2 tg,
            // 2 tg + 1, 2 tg + 8, 2 tg + 9 of each chunk.
            const int t0 = (2 * tg) ^ (tg & 1), t1 = (2 * tg + 1) ^ (tg & 1);
#pragma unroll
            for (int half = 0; half < 2; half++) {
                const uint8_t *vr = tile + half * C::kChunk + kv4_codes_bytes(D) + g * (D / 16);
                uint32_t v0[VW], v1[VW], v2[VW], v3[VW];
                if (D == 128) {
                    const uint2 a = *reinterpret_cast<const uint2 *>(vr + t0 * (D / 2));
                    const uint2 b = *reinterpret_cast<const uint2 *>(vr + t1 * (D / 2));
                    const uint2 c = *reinterpret_cast<const uint2 *>(vr + (t0 + 8) * (D / 2));
                    const uint2 d = *reinterpret_cast<const uint2 *>(vr + (t1 + 8) * (D / 2));
                    v0[0] = a.x, v0[VW - 1] = a.y, v1[0] = b.x, v1[VW - 1] = b.y;
                    v2[0] = c.x, v2[VW - 1] = c.y, v3[0] = d.x, v3[VW - 1] = d.y;
                } else {
                    v0[0] = *reinterpret_cast<const uint32_t *>(vr + t0 * (D / 2));
                    v1[0] = *reinterpret_cast<const uint32_t *>(vr + t1 * (D / 2));
                    v2[0] = *reinterpret_cast<const uint32_t *>(vr + (t0 + 8) * (D / 2));
                    v3[0] = *reinterpret_cast<const uint32_t *>(vr + (t1 + 8) * (D / 2));
                }
#pragma unroll
                for (int k = 0; k < VW; k++)
#pragma unroll
                    for (int hw = 0; hw < 2; hw++) {
                        uint32_t x[4], y[4];
                        spread_codes<true>(prmt(v0[k], v1[k], hw ? 0x7632 : 0x5410), x);
                        spread_codes<true>(prmt(v2[k], v3[k], hw ? 0x7632 : 0x5410), y);
#pragma unroll
                        for (int nt = 0; nt < NT; nt++) {
                            mma_add<NORMAL>(o[k * 4 + hw * 2][nt], x[0], x[1], y[0], y[1], pb[nt][2 * half],
                                     pb[nt][2 * half + 1]);
                            mma_add<NORMAL>(o[k * 4 + hw * 2 + 1][nt], x[2], x[3], y[2], y[3], pb[nt][2 * half],
                                     pb[nt][2 * half + 1]);
                        }
                    }
            }
            __syncwarp();
            count++;
            const int nx = i + kStages;
            if (nx < tiles) {
                if (nx >= pg_base + 32) load_pages(nx);
                // issue() counts from this item's first tile
                count -= i + 1;
                issue(nx);
                count += i + 1;
            }
        }

        // ---- merge the warps ----
        float *mo = reinterpret_cast<float *>(smem);  // [warp][COLS][D + 4], over the idle ring
        constexpr int MS = D + 4;
        __syncthreads();                              // every warp's ring is empty
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            constexpr int E = SPLIT == 2 ? 1 : 2;
#pragma unroll
            for (int e = 0; e < E; e++) {
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) {
                    sum[nt][e] += __shfl_xor_sync(0xffffffffu, sum[nt][e], k);
                    zero[nt][e] += __shfl_xor_sync(0xffffffffu, zero[nt][e], k);
                }
                const int c = SPLIT == 2 ? nt * 4 + tg : nt * 8 + 2 * tg + e;
                if (g == 0) m_ref[warp][c] = ref[nt][e], m_sum[warp][c] = sum[nt][e], m_zero[warp][c] = zero[nt][e];
                float *dst = mo + (warp * COLS + c) * MS + g * (D / 8);
#pragma unroll
                for (int m = 0; m < D / 16; m++) {
                    const float a = SPLIT == 2 ? o[m][nt][0] + o[m][nt][1] : o[m][nt][e];
                    const float b = SPLIT == 2 ? o[m][nt][2] + o[m][nt][3] : o[m][nt][2 + e];
                    // m-tile m: dimensions 2 m and 2 m + 1 of this thread's D / 8
                    *reinterpret_cast<float2 *>(dst + 2 * m) = make_float2(a, b);
                }
            }
        }
        __syncthreads();
        const bool whole = first == 0 && last == un.tiles;
        const int slot = 2 * blockIdx.x + (first == 0 ? 1 : 0);
        for (int c = tid / (D / 4); c < ncol; c += kThreads / (D / 4)) {
            const int d = tid % (D / 4) * 4;
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; w++) m = fmaxf(m, m_ref[w][c]);
            float l = 0.f, z = 0.f, x[4] = {};
#pragma unroll
            for (int w = 0; w < kWarps; w++) {
                const float f = m_ref[w][c] == -INFINITY ? 0.f : ex2(m_ref[w][c] - m);
                l += f * m_sum[w][c], z += f * m_zero[w][c];
                const float4 v = *reinterpret_cast<const float4 *>(mo + (w * COLS + c) * MS + d);
                x[0] += f * v.x, x[1] += f * v.y, x[2] += f * v.z, x[3] += f * v.w;
            }
#pragma unroll
            for (int e = 0; e < 4; e++) x[e] = (x[e] - z) * (1.f / kLift);
            if (whole) {
                const int cc = col0 + c, head = h * p.group + cc % p.group;
                const int64_t t = rq.q0 + cc / p.group;
                const float inv = l == 0.f ? 0.f : 1.f / l;
                T *dst = static_cast<T *>(p.out) + t * p.out_stride + (int64_t)head * D + d;
#pragma unroll
                for (int e = 0; e < 4; e++) store_value(dst + e, l == 0.f ? 0.f : x[e] * inv);
                if (p.lse && d == 0) p.lse[t * p.heads + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            } else {
                *reinterpret_cast<float4 *>(p.part + ((int64_t)slot * COLS + c) * D + d) =
                    make_float4(x[0], x[1], x[2], x[3]);
                if (d == 0) p.stat[slot * COLS + c] = make_float2(m, l);
            }
        }
        if (!whole && tid == 0) {
            // The CTA the item begins in: the last one whose run starts at or before its first unit.
            const int64_t begin = r_begin + (int64_t)item * un.tiles;
            const int owner = (int)(((begin + 1) * ctas - 1) / total);
            record[first == 0 ? 1 : 0] = make_int4(r, item, last == un.tiles ? owner + 1 : 0, ncol);
        }
        fence_proxy_async_shared();  // the merge's writes come before the next item's copies
        __syncthreads();
    }
}

// Joins the parts of items that several CTAs shared.  The record of the CTA that took an item's
// last part names the CTA that began it; the parts in between are the CTAs' between them.  One
// block per CTA record and row, D / 4 threads per part.  Bound by the way from the record to the
// parts and out again: references, parts and the request are loaded together (64 requests of up to
// 4096 tokens: 55 us for both kernels; references, sums and parts one after another 63).
constexpr int kJoin = 128;
template <int D, typename T, int COLS>
__global__ void __launch_bounds__(kJoin) attn_join_kernel(const AttnParams p) {
    constexpr int L = D / 4, GROUPS = kJoin / L, AHEAD = 4;
    __shared__ float acc[GROUPS][D];
    const int tid = threadIdx.x, lane = tid & 31;
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.x, c = blockIdx.y;
    const int4 rec = p.record[2 * b];
    if (rec.x < 0 || rec.z == 0 || c >= rec.w) return;
    const int first = rec.z - 1, n = b - first + 1;
    auto stat_of = [&](int i) { return p.stat[(i == 0 ? 2 * first + 1 : 2 * (first + i)) * COLS + c]; };
    auto part_of = [&](int i) {
        const int64_t slot = i == 0 ? 2 * first + 1 : 2 * (first + i);
        return *reinterpret_cast<const float4 *>(p.part + (slot * COLS + c) * D + tid % L * 4);
    };
    auto share = [](float ref, float m) { return ref == -INFINITY ? 0.f : ex2(ref - m); };
    // All that does not depend on each other is asked for first; every warp reduces the references
    // and sums for itself.
    float2 s[AHEAD];
    float ref[AHEAD];
    float4 v[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; k++) {
        const int i = k * 32 + lane, j = k * GROUPS + tid / L;
        s[k] = i < n ? stat_of(i) : make_float2(-INFINITY, 0.f);
        ref[k] = j < n ? stat_of(j).x : -INFINITY;
        v[k] = j < n ? part_of(j) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const Request q = load_request(p, rec.x);
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int k = 0; k < AHEAD; k++) m = fmaxf(m, s[k].x);
    for (int i = AHEAD * 32 + lane; i < n; i += 32) m = fmaxf(m, stat_of(i).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
    for (int k = 0; k < AHEAD; k++) l = fmaf(share(s[k].x, m), s[k].y, l);
    for (int i = AHEAD * 32 + lane; i < n; i += 32) {
        const float2 t = stat_of(i);
        l = fmaf(share(t.x, m), t.y, l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    float x[4] = {};
    auto add = [&](float f, const float4 &y) {
        x[0] = fmaf(f, y.x, x[0]), x[1] = fmaf(f, y.y, x[1]);
        x[2] = fmaf(f, y.z, x[2]), x[3] = fmaf(f, y.w, x[3]);
    };
#pragma unroll
    for (int k = 0; k < AHEAD; k++) add(share(ref[k], m), v[k]);
#pragma unroll 4
    for (int i = AHEAD * GROUPS + tid / L; i < n; i += GROUPS) add(share(stat_of(i).x, m), part_of(i));
    *reinterpret_cast<float4 *>(&acc[tid / L][tid % L * 4]) = make_float4(x[0], x[1], x[2], x[3]);
    __syncthreads();
    const int groups = (q.n * p.group + COLS - 1) / COLS;
    const int cc = rec.y % groups * COLS + c, head = rec.y / groups * p.group + cc % p.group;
    const int64_t t = q.q0 + cc / p.group;
    if (tid < D) {
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < GROUPS; i++) y += acc[i][tid];
        store_value(static_cast<T *>(p.out) + t * p.out_stride + (int64_t)head * D + tid,
                    l == 0.f ? 0.f : y / l);
    }
    if (p.lse && tid == 0) p.lse[t * p.heads + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int D, typename T, int SPLIT, int NT>
static int launch_decode(AttnParams p, uint8_t *workspace, int sms, cudaStream_t st) {
    using C = Decode<D, SPLIT, NT>;
    p.record = reinterpret_cast<int4 *>(workspace);
    p.stat = reinterpret_cast<float2 *>(p.record + 2 * kMaxCtas);
    p.part = reinterpret_cast<float *>(p.stat + 2 * kMaxCtas * C::kCols);
    auto kernel = attn_decode_kernel<D, T, SPLIT, NT>;
    int per_sm;
    if (int e = prepare_kernel((const void *)kernel, kThreads, C::kSmem, &per_sm)) return e;
    const int ctas = sms * per_sm < kMaxCtas ? sms * per_sm : kMaxCtas;
    if (int e = launch_pdl(kernel, dim3(ctas), dim3(kThreads), C::kSmem, st, p)) return e;
    if ((p.width << p.shift) <= kWhole * kTile) return LB_OK;  // no item can have been split
    return launch_pdl(attn_join_kernel<D, T, C::kCols>, dim3(ctas, C::kCols), dim3(kJoin), 0, st,
                      p);
}

// One fp16 part needs 11 bits (bf16 tensors); fp32 tensors take two.  Up to four rows per head
// take two parts in either type: the eight columns of a product hold them anyway, and a thread
// then has one row's scores instead of two, half of them of empty columns.
template <int D>
static int dispatch_decode(const AttnParams &p, int type, int64_t max_q, uint8_t *workspace,
                           int sms, cudaStream_t st) {
    const int64_t rows = max_q * p.group;
    // Row groups of one product's eight columns: two together take about as long as one after the
    // other, so three go one by one (bf16, 20 rows of 1000 tokens, 32 requests: 38 against 42 us;
    // two or four together: 28 against 30 and 45 against 48).
    const int64_t groups = (rows + (type == LB_OUT_F32 ? 3 : 7)) / (type == LB_OUT_F32 ? 4 : 8);
    const bool one = groups == 1 || groups == 3;
    if (type == LB_OUT_F32)
        return one ? launch_decode<D, float, 2, 1>(p, workspace, sms, st)
                   : launch_decode<D, float, 2, 2>(p, workspace, sms, st);
    if (rows <= 4) return launch_decode<D, __nv_bfloat16, 2, 1>(p, workspace, sms, st);
    return one ? launch_decode<D, __nv_bfloat16, 1, 1>(p, workspace, sms, st)
               : launch_decode<D, __nv_bfloat16, 1, 2>(p, workspace, sms, st);
}

}  // namespace lb

LB_EXPORT size_t lb_attn_kv4_workspace_bytes(int heads, int kv_heads, int head_dim, int64_t max_q) {
    if (heads < 1 || kv_heads < 1 || head_dim < 1 || max_q < 1) return 0;
    const size_t few = (size_t)lb::kMaxCtas * 2 * (16 + 16 * (8 + (size_t)head_dim * 4));
    const size_t many = lb::attn_prompt_workspace(head_dim);
    return max_q * (heads / kv_heads) <= lb::kFewRows || few > many ? few : many;
}

LB_EXPORT int lb_attn_kv4(const void *q, int type, int64_t q_stride, const uint8_t *cache,
                          int64_t pages, int page_size, int heads, int kv_heads, int head_dim,
                          const int32_t *block_table, int64_t table_width, const int32_t *q_start,
                          const int32_t *kv_len, int64_t R, int64_t T, int64_t max_q, float scale,
                          int causal, int64_t window, void *out, int64_t out_stride,
                          float *lse_opt, void *workspace, size_t workspace_bytes, void *stream) {
    using namespace lb;
    const int64_t lim = int64_t(1) << 31;
    if (!cache || !block_table || !q_start || !kv_len || !workspace || (T != 0 && (!q || !out)))
        return LB_ERR_NULL;
    if ((type != LB_OUT_F32 && type != LB_OUT_BF16) ||
        !kv4_shape_ok(pages, page_size, kv_heads, head_dim) || heads < kv_heads ||
        heads % kv_heads || heads / kv_heads > 64 || R < 1 || R > LB_KV_MAX_REQUESTS || T < 0 ||
        T * (heads / kv_heads) >= lim || table_width < 1 ||
        table_width > (lim >> 1) / page_size || max_q < 1 || max_q >= lim ||
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
    AttnParams p{};
    p.q = q, p.out = out, p.lse = lse_opt, p.cache = cache, p.table = block_table;
    p.q_start = q_start, p.kv_len = kv_len, p.q_stride = q_stride, p.out_stride = out_stride;
    p.pages = pages, p.width = table_width, p.T = T, p.R = (int)R, p.heads = heads;
    p.kv_heads = kv_heads, p.group = heads / kv_heads, p.shift = page_shift_of(page_size);
    p.causal = causal != 0, p.window = (int)window, p.scale = scale;
    p.rows_lo = 0, p.rows_hi = 0x7fffffff;
    p.error = device_error_word();
    if (!p.error) return LB_ERR_LAUNCH;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    cudaStream_t st = as_stream(stream);
    if (max_q * p.group > kFewRows) {
        // A few requests go together; in a larger batch those with few rows (decode steps beside
        // prompts) take the other kernel.
        if (R > kFewRequests) p.rows_lo = kFewRows;
        if (int e = attn_prompt(p, type, head_dim, ws, di.sms, st)) return e;
        if (R <= kFewRequests) return LB_OK;
        p.rows_lo = 0, p.rows_hi = kFewRows;
        max_q = kFewRows / p.group > 1 ? kFewRows / p.group : 1;
    }
    return head_dim == 64 ? dispatch_decode<64>(p, type, max_q, ws, di.sms, st)
                          : dispatch_decode<128>(p, type, max_q, ws, di.sms, st);
}
