// lb_q4_gemv.cu -- products of 4-bit weights with group scales for a few tokens.
//
// Mathematics.  y[t][n] = sum over groups g of d[n][g] * sum_{k in g} (c[n][k] - z[n][g]) x[t][k].  The
// inner sums run on mma.sync m16n8k16 (fp16 operands, binary32 sums): 16 weight rows times 8 tokens.
// c - z is a whole number, exact in fp16; a token's slice of x is scaled by a power of two into fp16's range, where a
// bf16 x has all its bits and an fp32 one takes two parts (22 bits).  The scale d acts
// on a group's sum in binary32: a fused multiply-add per group, row and token.
//
// Work: units of 256 rows (of a token piece), each split along K over a cluster of up to eight CTAs; a cluster
// takes an equal run of units, so x is laid out once (experts: once per piece) and weights keep coming across the units' borders.
// One CTA per SM.  One warp copies blocks of 256 rows x 256 columns (32 KB, tensor copies, with their scales and zeros)
// into a ring; the first ones start before the previous kernel in the stream has ended.  16 warps take 16 rows
// each (experts' up products: 8 gate and the same 8 up rows): ldmatrix hands a lane whole words of eight
// consecutive columns of its row, which are four operand registers after logic operations that put the codes
// under the exponent of 1024 and a subtraction of 1024 + z (the upper codes of a byte: times 1/16, less 64 + z).  The eight
// columns of a word enter as pairs (0, 4), (1, 5), (2, 6), (3, 7); x is laid out in shared memory in that
// order, so a 16-byte read is the other operand of two steps.  A warp sends its sums to the CTA of the
// cluster that is to finish its rows, and that CTA adds them up, in the order of the ranks, after its next unit.
//
// What bounds it: in the steady state the issue slots (a warp issues about 60 instructions for 512 weights with two-part x,
// 51 to 59 % of the slots over a call), before HBM (20 to 31 %); in short calls the fixed parts: about 3000 clocks to the
// first product and 2000 to 4000 for x.  128 columns are in flight at a time, on four accumulators, since the products'
// latency would otherwise set the pace (one accumulator: 190 cycles for 512 weights).  1 x 12288 x 4096 fp32 in groups
// of 32: 12.7 us, 5 x 4096 x 12288 bf16: 13.0; 43 tokens' eight of 64 experts of 2048 x 1024, fp32: 94 to 100 with their sum.
#include "lb_q4.cuh"

#include <algorithm>
#include <map>
#include <mutex>
#include <tuple>
#include <type_traits>

namespace lb {

constexpr int kMvRows = 256;                     // of a unit
constexpr int kMvBlock = 256;                    // columns of a ring stage
constexpr int kMvBox = kMvRows * 64;             // bytes of a copy: 128 columns
constexpr int kMvStage = kMvRows * kMvBlock / 2;
constexpr int kMvWarps = 16;
constexpr int kMvThreads = 32 * (kMvWarps + 1);
constexpr int kMvTokens = 8;
constexpr int kMvMaxSplit = 8;
constexpr int kMvSums = 21;                      // most of split * ceil(kMvWarps / split)
constexpr int kMvMaxStages = 5;
constexpr size_t kMvShared = 226 * 1024;         // shared memory of a CTA, static and dynamic

struct MvLaunch {
    int blocks;    // blocks of K of a CTA
    int stages;
    int tokens;    // most tokens of a piece
    int split;     // CTAs along K, a cluster
    int tiles;     // of kMvRows rows (up: of half as many pairs)
    int fault;     // test hook: the first CTA with a unit copies no weights and waits so many microseconds for them
};

// (volatile: stays behind the wait for its stage)
__device__ __forceinline__ void ldmatrix4(uint32_t *r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void mma_f16_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same onto nothing.
__device__ __forceinline__ void mma_f16_begin(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, int bytes) {
    if (bytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else if (bytes == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// The address of this CTA's shared memory's p in another CTA of the cluster.
__device__ __forceinline__ uint32_t address_in(const void *p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void store_in(uint32_t a, float x, float y) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ void arrive_in(uint32_t a) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(a) : "memory");
}
__device__ __forceinline__ bool mv_try_wait_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3; "
        "selp.u32 %0, 1, 0, p; }"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(1000u)
        : "memory");
    return ok != 0;
}
// (apart, so that what the test hook needs takes no registers beside the products)
__device__ __noinline__ static bool mv_wait_weights(uint64_t *bar, uint32_t parity, const int *fault) {
    return mbar_wait_slow(bar, parity, *fault ? (uint64_t)*fault * 1000u : 2000000000ull);
}
// cp.async's of this thread so far arrive once on bar when they have landed (counted in the barrier's number).
__device__ __forceinline__ void copies_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void store_y(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_y(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// The first of the warps whose rows the CTA of a rank finishes (warp w's is w * split / kMvWarps).
__device__ __forceinline__ int first_warp(int rank, int split) { return (kMvWarps * rank + split - 1) / split; }

// T: the type of x (dense, up; h is fp32) and of a dense y; PARTS: fp16 parts of an x.
template <Q4Use USE, typename T, int PARTS, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(kMvThreads, 1)
    q4_gemv_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ Q4Params p,
                   const __grid_constant__ MvLaunch l) {
    using X = typename std::conditional<USE == kQ4Down, float, T>::type;
    constexpr int kPer = kMvBlock / GROUP;                       // groups of a block
    constexpr int kExperts = USE == kQ4Dense ? 1 : LB_ROUTE_MAX_EXPERTS;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint64_t full[kMvMaxStages], empty[kMvMaxStages], sums_full[2];
    __shared__ __align__(16) uint16_t ds[kMvMaxStages][kMvRows][kPer];
    __shared__ __align__(16) uint8_t zs[ZEROS ? kMvMaxStages : 1][kMvRows][kPer < 4 ? 4 : kPer];
    __shared__ __align__(16) float sums[2][kMvSums][16][kMvTokens];   // [rank, own warp][row][column]
    __shared__ int row_of[2][kMvTokens];
    __shared__ uint16_t s_first[kExperts];                       // pieces before an expert's
    __shared__ int s_part[kMvThreads / 32], s_fault;
    __shared__ volatile int s_lost;                              // a wait for sums has run out
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slice = l.blocks * kMvBlock, rank = blockIdx.x % l.split;
    const int k0 = rank * slice, columns = min(p.K - k0, slice);
    const int blocks = max((columns + kMvBlock - 1) / kMvBlock, 0);   // (the last CTAs along K may have none)
    const int x_pitch = 2 * slice + 64;
    uint8_t *ring = smem;
    float *back = reinterpret_cast<float *>(ring + l.stages * kMvStage);   // takes scaling back: [256 columns][operand column]
    uint8_t *xs = reinterpret_cast<uint8_t *>(back + l.blocks * kMvTokens);

    pdl_launch_dependents();
    if (tid == 0) {
        s_lost = 0;
        // a stage is full when the copies of codes and the 32 lanes' copies of scales have landed
        for (int i = 0; i < kMvMaxStages; i++) mbar_init(&full[i], 33), mbar_init(&empty[i], kMvWarps);
        // from every CTA come the sums of the warps whose rows are finished here, in two halves
        const int arrivals = 2 * l.split * (first_warp(rank + 1, l.split) - first_warp(rank, l.split));
        mbar_init(&sums_full[0], arrivals), mbar_init(&sums_full[1], arrivals);
        fence_mbar_init();
    }
    // Pieces of at most l.tokens tokens (of one expert).
    int pieces;
    if constexpr (USE == kQ4Dense) {
        pieces = (int)((p.T + l.tokens - 1) / l.tokens);
    } else {
        pdl_wait();
        constexpr int kEach = (LB_ROUTE_MAX_EXPERTS + kMvThreads - 1) / kMvThreads;
        int n[kEach], mine = 0;
#pragma unroll
        for (int i = 0; i < kEach; i++) {
            const int e = tid * kEach + i;
            n[i] = 0;
            if (e < p.E) {
                const int first = min(max(p.start[e], 0), (int)p.T);
                n[i] = (max(min(p.start[e + 1], (int)p.T) - first, 0) + l.tokens - 1) / l.tokens;
            }
            mine += n[i];
        }
        int run = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int w = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += w;
        }
        if (lane == 31) s_part[warp] = run;
        __syncthreads();
        int before = run - mine;
        pieces = 0;
#pragma unroll
        for (int w = 0; w < kMvThreads / 32; w++) {
            before += w < warp ? s_part[w] : 0;
            pieces += s_part[w];
        }
        pieces = min(pieces, 65535);
#pragma unroll
        for (int i = 0; i < kEach; i++) {
            if (tid * kEach + i < p.E) s_first[tid * kEach + i] = (uint16_t)min(before, 65535);
            before += n[i];
        }
    }
    // (everybody's barriers are there before anybody's sums are sent: waited for then)
    if (l.split > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    __syncthreads();
    struct Piece {
        int expert, t0, tokens, slot;   // slot: of row_of
    };
    auto piece_of = [&](int i) {
        Piece q;
        q.slot = 0;
        if constexpr (USE == kQ4Dense) {
            q.expert = 0, q.t0 = i * l.tokens;
            q.tokens = (int)min((int64_t)l.tokens, p.T - q.t0);
        } else {
            int lo = 0, hi = p.E;   // the last expert whose pieces begin at or before this one
            while (hi - lo > 1) {
                const int m = (lo + hi) / 2;
                if (s_first[m] <= i) lo = m;
                else hi = m;
            }
            const int first = min(max(p.start[lo], 0), (int)p.T), end = min(p.start[lo + 1], (int)p.T);
            q.expert = lo, q.t0 = first + (i - s_first[lo]) * l.tokens;
            q.tokens = min(l.tokens, end - q.t0);
        }
        return q;
    };
    // This cluster's units.
    const int64_t units = (int64_t)pieces * l.tiles, clusters = gridDim.x / l.split, c = blockIdx.x / l.split;
    const int u_begin = (int)(units * c / clusters), u_end = (int)(units * (c + 1) / clusters);
    constexpr int kTileRows = USE == kQ4Up ? kMvRows / 2 : kMvRows;

    if (warp == kMvWarps) {
        // =================== copies ===================
        int stage = 0, used = 0;
        uint32_t phase = 0;
        bool ok = true;
        int at_piece = -1;
        Piece q{0, 0, 0, 0};
        if (l.fault && rank == 0 && u_begin == 0) ok = false;
        for (int u = u_begin; u < u_end && ok; u++) {
            const int piece = u / l.tiles;
            const int64_t n0 = (int64_t)(u - piece * l.tiles) * kTileRows;
            if (piece != at_piece) q = piece_of(piece), at_piece = piece;
            const int64_t matrix = (int64_t)q.expert * (USE == kQ4Up ? 2 * p.N : p.N);
            const int64_t last = matrix + (USE == kQ4Up ? 2 * p.N : p.N);
            const int64_t upper = matrix + (USE == kQ4Up ? p.N + n0 : n0 + kMvRows / 2);   // the tile's row 64
            for (int b = 0; b < blocks; b++) {
                ok = __all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1));
                if (!ok) {
                    if (lane == 0) atomicOr(p.error, 1);
                    break;
                }
                uint64_t *bar = &full[stage];
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, kMvStage);
                    uint8_t *dst = ring + stage * kMvStage;
#pragma unroll
                    for (int j = 0; j < kMvBlock / 128; j++) {
                        const int at = (k0 + b * kMvBlock) / 2 + 64 * j;
                        tma_load_2d(dst + j * kMvBox, &map, at, (int)(matrix + n0), bar);
                        tma_load_2d(dst + j * kMvBox + kMvBox / 2, &map, at, (int)upper, bar);
                    }
                }
                __syncwarp();
                // (a row's entries reach to a multiple of eight; copies have four bytes at least, so where a block has two
                // zeros, the next or last block's come along)
                const int first = k0 / GROUP + b * kPer;
#pragma unroll
                for (int j = 0; j < kMvRows / 32; j++) {
                    const int r = j * 32 + lane;
                    const int64_t row = r < kMvRows / 2 ? matrix + n0 + r : upper + r - kMvRows / 2;
                    if (row >= last) continue;   // the products of rows behind the matrix go nowhere
                    const int64_t from = row * p.pitch + first;
                    copy_async(smem_u32(&ds[stage][r][0]), p.scales + from, 2 * kPer);
                    if (ZEROS)
                        copy_async(smem_u32(&zs[ZEROS ? stage : 0][r][0]), p.zeros + (kPer == 2 ? from & ~3 : from),
                                   kPer < 4 ? 4 : kPer);
                }
                copies_arrive(bar);
                if (++stage == l.stages) stage = 0, phase ^= 1;
                used = min(used + 1, l.stages);
            }
        }
        // no copy may still be landing when the CTA exits
        asm volatile("cp.async.wait_all;" ::: "memory");
        for (int i = 0; i < used; i++) {
            if (stage == 0) stage = l.stages, phase ^= 1;
            stage--;
            mbar_wait(&full[stage], phase);
        }
        if (USE == kQ4Dense) pdl_wait();
        if (l.split > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    } else {
        // =================== products ===================
        if (tid == 0) s_fault = rank == 0 && u_begin == 0 ? l.fault : 0;   // (read behind the first barrier below)
        if (USE == kQ4Dense) pdl_wait();
        const int g = lane >> 2, t = lane & 3;
        // the row this lane points ldmatrix at, and the two rows of its sums, in the tile
        const int row = USE == kQ4Up ? warp * 8 + (lane & 7) + (lane & 8) * (kMvRows / 16) : warp * 16 + (lane & 15);
        const int row0 = USE == kQ4Up ? warp * 8 + g : warp * 16 + g, row1 = USE == kQ4Up ? row0 + kMvRows / 2 : row0 + 8;
        const uint32_t at_row = smem_u32(ring) + row * 64, turn = (row >> 1) & 3;
        const int pitch = (kMvWarps + l.split - 1) / l.split;   // of a rank's sums
        const int first_own = first_warp(rank, l.split), own = first_warp(rank + 1, l.split) - first_own;
        const uint32_t owner = warp * l.split / kMvWarps;
        const uint32_t send_to = address_in(&sums[0][rank * pitch + warp - first_warp(owner, l.split)][g][2 * t], owner);
        const uint32_t tell[2] = {address_in(&sums_full[0], owner), address_in(&sums_full[1], owner)};
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;   // no wait for weights has run out
        int at_piece = -1, cols = 0, planes = 1;
        Piece q{0, 0, 0, 0};
        // The parts of few tokens lie in one operand's eight columns, of more in an operand each.
        auto packed = [](const Piece &a) { return a.tokens * PARTS <= kMvTokens; };
        // What a finished unit leaves to be done after the next one's products.
        Piece q_done{0, 0, 0, 0};
        int64_t n_done = 0;
        // a finished sum of row `row_n` of the matrix (up: gate and up rows')
        auto store = [&](const Piece &a, int64_t row_n, int tk, float v0, float v1) {
            if (row_n >= p.N) return;
            if (USE == kQ4Dense) {
                store_y(static_cast<T *>(p.y) + (a.t0 + tk) * p.y_stride + row_n, v0);
            } else if (USE == kQ4Up) {
                static_cast<float *>(p.y)[(int64_t)(a.t0 + tk) * p.y_stride + row_n] = v0 / (1.f + expf(-v0)) * v1;
            } else {
                const int pair = row_of[a.slot][tk];
                if (pair >= 0 && pair < p.T) static_cast<float *>(p.y)[(int64_t)pair * p.y_stride + row_n] = v0;
            }
        };
        // a lane's two rows' sums
        auto put = [&](const Piece &a, int64_t row_n, int tk, float v0, float v1) {
            store(a, row_n, tk, v0, v1);
            if (USE != kQ4Up) store(a, row_n + 8, tk, v1, 0.f);
        };
        // the sums of unit number n (of this cluster's), added up over the ranks and stored
        auto finish = [&](int n) {
            if (!__any_sync(0xffffffffu, s_lost)) {   // (the whole warp waits, or none of it)
                const uint64_t t_0 = global_ns();
                bool there = mv_try_wait_cluster(&sums_full[n & 1], (uint32_t)(n >> 1) & 1u);
                for (uint32_t i = 1; !there; i++) {
                    there = mv_try_wait_cluster(&sums_full[n & 1], (uint32_t)(n >> 1) & 1u);
                    if ((i & 15u) == 0 && global_ns() - t_0 > 2000000000ull) break;
                }
                if (!__all_sync(0xffffffffu, there)) {
                    if (lane == 0) atomicOr(p.error, 1), s_lost = 1;
                    __syncwarp();
                }
            }
            const int parts = packed(q_done) ? PARTS : 1;
            constexpr int per_warp = USE == kQ4Up ? 8 : 16;
            const uint32_t rows = own * per_warp;
            for (uint32_t i = tid; i < q_done.tokens * rows; i += 32 * kMvWarps) {
                const int tk = i / rows, r = i - tk * rows, w = r / per_warp, rr = r % per_warp;
                const int64_t row_n = n_done + (first_own + w) * per_warp + rr;
                float v[2] = {0.f, 0.f};
#pragma unroll
                for (int h = 0; h < (USE == kQ4Up ? 2 : 1); h++)
                    for (int k = 0; k < parts; k++)
                        for (int s = 0; s < l.split; s++)
                            v[h] += sums[n & 1][s * pitch + w][rr + 8 * h][tk * parts + k];
                store(q_done, row_n, tk, v[0], v[1]);
            }
        };
        int n = 0;
        for (int u = u_begin; u < u_end; u++, n++) {
            const int piece = u / l.tiles;
            if (piece != at_piece) {
                // x of the slice: operand row (packed: token * PARTS + part, else part * tokens + token), columns in
                // the order of the codes' pairs, zeros behind K
                const int slot = q.slot ^ 1;   // (the last piece's rows may still be asked for)
                q = piece_of(piece), at_piece = piece, q.slot = slot;
                named_sync(1, 32 * kMvWarps);   // the last piece's x is done with
                if (USE != kQ4Dense && tid < q.tokens) row_of[slot][tid] = p.order[q.t0 + tid];
                named_sync(1, 32 * kMvWarps);
                const bool pack = packed(q);
                cols = pack ? q.tokens * PARTS : q.tokens, planes = pack ? 1 : PARTS;
                // A warp takes a block of a token, eight columns a lane, scaled so that the largest comes to lie in [2^14,
                // 2^15).  Four blocks are asked for together.
                const int each = max(blocks, 0), all = q.tokens * each;
                for (int c0 = warp; c0 < all; c0 += 4 * kMvWarps) {
                    float v[4][8];
                    bool in[4];
                    int tok[4], blk[4];
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const int c2 = c0 + k * kMvWarps;
                        tok[k] = c2 / each, blk[k] = c2 - tok[k] * each;
                        const int at = blk[k] * kMvBlock + lane * 8;
                        in[k] = c2 < all && at < columns;
                        int64_t from = q.t0 + tok[k];
                        if (USE != kQ4Dense) {
                            const int pair = in[k] ? row_of[slot][tok[k]] : -1;
                            in[k] = pair >= 0 && pair < p.T;
                            if (USE == kQ4Up) from = pair / p.k;
                        }
                        load8(static_cast<const X *>(p.x) + (in[k] ? from * p.x_stride + k0 + at : 0), v[k]);
                    }
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        if (c0 + k * kMvWarps >= all) break;
                        float m = 0.f;
#pragma unroll
                        for (int j = 0; j < 8; j++) {
                            v[k][j] = in[k] ? v[k][j] : 0.f;
                            m = fmaxf(m, fabsf(v[k][j]));
                        }
                        const uint32_t e = q4_power(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
                        const float up = __uint_as_float(e << 23);
                        uint32_t w[PARTS][4];
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const float a = v[k][j] * up, c2 = v[k][j + 4] * up;
                            const __half2 h = __floats2half2_rn(a, c2);
                            w[0][j] = bits_of(h);
                            if (PARTS == 2)
                                w[PARTS - 1][j] = bits_of(__floats2half2_rn(a - __low2float(h), c2 - __high2float(h)));
                        }
#pragma unroll
                        for (int part = 0; part < PARTS; part++) {
                            const int to = pack ? tok[k] * PARTS + part : part * q.tokens + tok[k];
                            *reinterpret_cast<uint4 *>(xs + to * x_pitch + blk[k] * (2 * kMvBlock) + 16 * lane) =
                                make_uint4(w[part][0], w[part][1], w[part][2], w[part][3]);
                            const int col = pack ? to : tok[k];
                            if (lane == 0) back[blk[k] * kMvTokens + col] = __uint_as_float((254u - e) << 23);
                        }
                    }
                }
                named_sync(1, 32 * kMvWarps);
            }
            const uint8_t *xrow = xs + min(g, cols - 1) * x_pitch + 16 * t;   // (columns without a token repeat one)
            const int plane = q.tokens * x_pitch;
            float total[4] = {0.f, 0.f, 0.f, 0.f};
            for (int b = 0; b < blocks && ok; b++) {
                if (!__all_sync(0xffffffffu, mbar_try_wait(&full[stage], phase) || mv_wait_weights(&full[stage], phase, &s_fault))) {
                    if (lane == 0) atomicOr(p.error, 1);
                    ok = false;
                    break;
                }
                const int chunks = min(kMvBlock, columns - b * kMvBlock) / 32;   // of 32 columns (K is a multiple)
                const int z_at = kPer == 2 ? (k0 / GROUP + b * kPer) & 2 : 0;
                // 128 columns at a time; where K ends inside, x is zero and a group behind K is left out.  (Whole blocks
                // without a branch, so that their parts' chains of operations run side by side.)
                auto columns128 = [&](int j, auto whole) {
                    constexpr bool all = decltype(whole)::value;
                    uint32_t w[2][4];   // the lane's two rows of chunks 0 and 1, then of 2 and 3
#pragma unroll
                    for (int h = 0; h < 2; h++)
                        ldmatrix4(w[h], at_row + stage * kMvStage + j * kMvBox +
                                            (((uint32_t)(2 * h) + (lane >> 4)) ^ turn) * 16);
                    const uint8_t *xc = xrow + (b * (kMvBlock / 32) + 4 * j) * 64;
                    constexpr int kGroups = 128 / GROUP, kEach = GROUP / 32;   // groups of 128 columns, chunks of a group
                    float sum[4][4];   // of each chunk; a group of four chunks takes two
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int gi = j * kGroups + e / kEach;
                        __half2 low[2], high[2];
#pragma unroll
                        for (int r = 0; r < 2; r++) {
                            const uint32_t z = ZEROS ? zs[ZEROS ? stage : 0][r ? row1 : row0][gi + z_at] : 8u;
                            low[r] = half2_of(0x64006400u + z * 0x10001u);
                            high[r] = half2_of(0xD400D400u + z * 0x00100010u);
                        }
                        uint32_t a[2][4];
                        const __half2 none = half2_of(0);
                        expand_f16<false>(w[e >> 1][2 * (e & 1)], low[0], high[0], none, a[0]);
                        expand_f16<false>(w[e >> 1][2 * (e & 1) + 1], low[1], high[1], none, a[1]);
                        const int at = kEach == 4 ? e & 1 : e;
                        const uint4 x = *reinterpret_cast<const uint4 *>(xc + e * 64);
                        if (at == e) mma_f16_begin(sum[at], a[0][0], a[1][0], a[0][1], a[1][1], x.x, x.y);
                        else mma_f16_16x8x16(sum[at], a[0][0], a[1][0], a[0][1], a[1][1], x.x, x.y);
                        mma_f16_16x8x16(sum[at], a[0][2], a[1][2], a[0][3], a[1][3], x.z, x.w);
                        if (PARTS == 2 && planes == 2) {
                            const uint4 rest = *reinterpret_cast<const uint4 *>(xc + plane + e * 64);
                            mma_f16_16x8x16(sum[at], a[0][0], a[1][0], a[0][1], a[1][1], rest.x, rest.y);
                            mma_f16_16x8x16(sum[at], a[0][2], a[1][2], a[0][3], a[1][3], rest.z, rest.w);
                        }
                    }
                    float part[4] = {0.f, 0.f, 0.f, 0.f};
                    // the two rows' scales of these 128 columns
                    uint2 d_row[2] = {make_uint2(0, 0), make_uint2(0, 0)};
#pragma unroll
                    for (int r = 0; r < 2; r++) {
                        const uint16_t *d = &ds[stage][r ? row1 : row0][j * kGroups];
                        if (kGroups == 4) d_row[r] = *reinterpret_cast<const uint2 *>(d);
                        else if (kGroups == 2) d_row[r].x = *reinterpret_cast<const uint32_t *>(d);
                        else d_row[r].x = *d;
                    }
                    auto scale_of = [](const uint2 &d, int i) { return (uint16_t)((i & 2 ? d.y : d.x) >> (16 * (i & 1))); };
#pragma unroll
                    for (int i = 0; i < kGroups; i++) {
                        if (!all && 4 * j + i * kEach >= chunks) break;
                        const int at = i * (kEach == 4 ? 1 : kEach);
                        const float d0 = f16_bits_to_float(scale_of(d_row[0], i)), d1 = f16_bits_to_float(scale_of(d_row[1], i));
                        if (kEach > 1)
#pragma unroll
                            for (int c2 = 0; c2 < 4; c2++) sum[at][c2] += sum[at + 1][c2];
                        part[0] = fmaf(d0, sum[at][0], part[0]), part[1] = fmaf(d0, sum[at][1], part[1]);
                        part[2] = fmaf(d1, sum[at][2], part[2]), part[3] = fmaf(d1, sum[at][3], part[3]);
                    }
                    const float2 f = *reinterpret_cast<const float2 *>(back + b * kMvTokens + 2 * t);
                    total[0] = fmaf(part[0], f.x, total[0]), total[1] = fmaf(part[1], f.y, total[1]);
                    total[2] = fmaf(part[2], f.x, total[2]), total[3] = fmaf(part[3], f.y, total[3]);
                };
                if (chunks >= kMvBlock / 32) {
#pragma unroll
                    for (int j = 0; j < kMvBlock / 128; j++) columns128(j, std::true_type{});
                } else {
#pragma unroll 1
                    for (int j = 0; 4 * j < chunks; j++) columns128(j, std::false_type{});
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[stage]);
                if (++stage == l.stages) stage = 0, phase ^= 1;
            }
            const int64_t n0 = (int64_t)(u - piece * l.tiles) * kTileRows;
            if (l.split == 1) {
                // alone: out of the registers, nobody waits for anybody
                const bool pack = packed(q);
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    if (PARTS == 2 && pack && i == 1) break;
                    const int tk = PARTS == 2 && pack ? t : 2 * t + i;
                    if (tk >= q.tokens) continue;
                    const float v0 = PARTS == 2 && pack ? total[0] + total[1] : total[i];
                    const float v1 = PARTS == 2 && pack ? total[2] + total[3] : total[2 + i];
                    put(q, n0 + row0, tk, v0, v1);
                }
                continue;
            }
            if (n > 0) finish(n - 1);
            else asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
            // (a CTA that has sent has done with the unit before the last one: its sums' place may be written to)
            named_sync(1, 32 * kMvWarps);
            // rows g and g + 8, columns 2t and 2t + 1, to the CTA that finishes them
            const uint32_t to = send_to + (n & 1) * (uint32_t)(sizeof(sums) / 2);
            store_in(to, total[0], total[1]);
            store_in(to + 8 * kMvTokens * 4, total[2], total[3]);
            __syncwarp();
            if (lane < 2) arrive_in(tell[n & 1]);
            q_done = q;
            n_done = n0;
        }
        if (l.split > 1) {
            if (n > 0) finish(n - 1);
            else asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
            // A CTA may go when nobody writes to it any more.  One whose waits for sums succeeded has by now all that are sent
            // to it (one without weights sends what it has; each sum arrives once, even from a CTA that gave its wait up and
            // ran ahead).  One that gave such a wait up does not know: it stays until every thread of the cluster has got
            // here or gone.  (All of them always waiting for each other: 13.4 us for 13.0, 5 x 4096 x 12288.)
            if (s_lost) asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
        }
    }
}

// How a call of given sizes is cut up.
struct MvPlan {
    MvLaunch l;
    int64_t clusters = 0;
    size_t smem = 0;
};

// The split whose longest run is the shortest; of equal ones the smallest.  `fixed`: static shared memory.
static MvPlan plan_gemv(const void *kernel, int64_t tokens, int tiles, int64_t pieces, int K, int parts, size_t fixed, int sms) {
    const int blocks = (K + kMvBlock - 1) / kMvBlock;
    MvPlan best;
    int64_t best_time = 0;
    for (int split = 1; split <= kMvMaxSplit; split++) {
        MvLaunch l{};
        l.blocks = (blocks + split - 1) / split;
        l.split = split, l.tiles = tiles;
        // Tokens: eight, or as many as their parts' slices fit beside two stages.
        const size_t pitch = 2 * (size_t)l.blocks * kMvBlock + 64, scales = (size_t)l.blocks * kMvTokens * 4;
        l.tokens = (int)tokens;
        const size_t most = kMvShared - fixed - 2 * kMvStage - scales;
        if (parts * l.tokens * pitch > most && split < kMvMaxSplit) continue;
        while (parts * l.tokens * pitch > most && l.tokens > 1) l.tokens--;
        // As many stages as fit.
        size_t smem = 2 * kMvStage + scales + parts * l.tokens * pitch;
        for (l.stages = 2; l.stages < kMvMaxStages && smem + kMvStage + fixed <= kMvShared; l.stages++) smem += kMvStage;
        int per_sm;
        if (prepare_kernel(kernel, kMvThreads, smem, &per_sm)) continue;
        int held = sms * per_sm;
        if (split > 1) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = (unsigned)split, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.gridDim = dim3((unsigned)split), cfg.blockDim = dim3(kMvThreads), cfg.dynamicSmemBytes = smem;
            cfg.attrs = attr, cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&held, kernel, &cfg) != cudaSuccess) {
                cudaGetLastError();
                continue;
            }
        }
        if (held < 1) continue;
        const int64_t units = (pieces ? pieces : (tokens + l.tokens - 1) / l.tokens) * tiles;
        const int64_t clusters = std::min<int64_t>(units, held);
        // in halves of a block's: a unit takes one by itself, three with sums that go through the cluster
        const int64_t time = (units + clusters - 1) / clusters * (2 * l.blocks + (split > 1 ? 3 : 1));
        if (!best.clusters || time < best_time) best.l = l, best.clusters = clusters, best.smem = smem, best_time = time;
    }
    return best;
}

template <Q4Use USE, typename T, int PARTS, int GROUP>
static int launch_gemv(const Q4Params &p, const CUtensorMap &map, int64_t pieces, int sms, cudaStream_t st) {
    auto kernel = p.zeros ? q4_gemv_kernel<USE, T, PARTS, GROUP, true> : q4_gemv_kernel<USE, T, PARTS, GROUP, false>;
    // (asking the driver for each split takes longer than the launch: remembered by what a plan depends on)
    static std::mutex mutex;
    static std::map<std::tuple<int, bool, int64_t, int64_t, int64_t, int>, MvPlan> known;
    int dev = 0;
    cudaGetDevice(&dev);
    const int64_t tokens = std::min<int64_t>(p.T, kMvTokens);
    MvPlan plan;
    try {
        std::lock_guard<std::mutex> lock(mutex);
        MvPlan &at = known[std::make_tuple(dev, p.zeros != nullptr, tokens, pieces, p.N, p.K)];
        if (!at.clusters) {
            constexpr int kTileRows = USE == kQ4Up ? kMvRows / 2 : kMvRows;
            cudaFuncAttributes fa{};
            const cudaError_t e = cudaFuncGetAttributes(&fa, (const void *)kernel);
            if (e != cudaSuccess) {
                record_cuda_error(e);
                return LB_ERR_LAUNCH;
            }
            at = plan_gemv((const void *)kernel, tokens, (int)((p.N + kTileRows - 1) / kTileRows), pieces, p.K, PARTS,
                           fa.sharedSizeBytes + 1024, sms);
        }
        plan = at;
    } catch (...) {   // (no memory on the host: nothing may be thrown through a C entry)
        return LB_ERR_LAUNCH;
    }
    if (!plan.clusters) return LB_ERR_LAUNCH;
    plan.l.fault = take_injected_wait_fault();
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)plan.l.split, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(plan.clusters * plan.l.split)), cfg.blockDim = dim3(kMvThreads);
    cfg.dynamicSmemBytes = plan.smem, cfg.stream = st, cfg.attrs = attr, cfg.numAttrs = plan.l.split > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, map, p, plan.l);
    if (e == cudaSuccess) return LB_OK;
    record_cuda_error(e);
    return LB_ERR_LAUNCH;
}

template <Q4Use USE, typename T, int PARTS>
static int dispatch_gemv(const Q4Params &p, const uint8_t *codes, int64_t rows, int sms, cudaStream_t st) {
    CUtensorMap map;
    if (int e = encode_rows_map(&map, codes, (uint64_t)p.K / 2, (uint64_t)rows, 64, kMvRows / 2, 64)) return e;
    // (experts: as many pieces as experts, if there are that many pairs)
    const int64_t pieces = USE == kQ4Dense ? 0 : std::min<int64_t>(p.T, p.E);
    switch (p.group) {
        case 32: return launch_gemv<USE, T, PARTS, 32>(p, map, pieces, sms, st);
        case 64: return launch_gemv<USE, T, PARTS, 64>(p, map, pieces, sms, st);
        default: return launch_gemv<USE, T, PARTS, 128>(p, map, pieces, sms, st);
    }
}

int q4_gemv(const Q4Params &p, Q4Use use, int type, const uint8_t *codes, int64_t rows, int sms,
            cudaStream_t st) {
    const bool f32 = type == LB_OUT_F32;
    if (use == kQ4Dense)
        return f32 ? dispatch_gemv<kQ4Dense, float, 2>(p, codes, rows, sms, st)
                   : dispatch_gemv<kQ4Dense, __nv_bfloat16, 1>(p, codes, rows, sms, st);
    if (use == kQ4Up)
        return f32 ? dispatch_gemv<kQ4Up, float, 2>(p, codes, rows, sms, st)
                   : dispatch_gemv<kQ4Up, __nv_bfloat16, 1>(p, codes, rows, sms, st);
    // (with bf16 tensors h is rounded to 11 bits, an eighth of an output's rounding)
    return f32 ? dispatch_gemv<kQ4Down, float, 2>(p, codes, rows, sms, st)
               : dispatch_gemv<kQ4Down, float, 1>(p, codes, rows, sms, st);
}

}  // namespace lb
