// lb_q4_gemv.cu -- products of 4-bit weights with group scales for a few tokens.
//
// Mathematics.  y[t][n] = sum over groups g of d[n][g] * sum_{k in g} (c[n][k] - z[n][g]) x[t][k].  The
// inner sums run on mma.sync m16n8k16 (bf16 operands, binary32 sums): 16 weight rows times 8 tokens.
// c - z is a whole number of at most eight bits, exact in bf16; a bf16 x is its own operand, an fp32 x is cut into
// three bf16 parts, which together are all its 24 bits, so the products are exact.  The scale acts
// on a group's sum in binary32: a fused multiply-add per group, row and token.
//
// A CTA takes 128 rows and a slice of K; up to eight CTAs along K form a cluster and add their sums
// up through distributed shared memory in a fixed order.  One warp copies blocks of 128 rows x
// 512 columns (32 KB) with tensor copies into a ring; they start before the previous kernel in the
// stream has ended.  Eight warps take 16 rows each: ldmatrix hands a lane whole words of eight
// consecutive columns of its row, which are four operand registers after a shift, a logic
// operation that puts the codes under the exponent of 128, and a subtraction of 128 + z.  The eight
// columns of a word enter as pairs (0, 4), (1, 5), (2, 6), (3, 7); x is laid out in shared memory in that
// order, so a 16-byte read is the other operand of two steps.
//
// What bounds it: HBM.  Per 512 weights a warp issues about 30 instructions, 0.6 of what the SM has at
// the rate the weights come in.
#include "lb_q4.cuh"

#include <algorithm>
#include <type_traits>

namespace lb {

constexpr int kMvRows = 128;                     // of a CTA
constexpr int kMvBlock = 512;                    // columns of a ring stage
constexpr int kMvBox = kMvRows * 64;             // bytes of a copy: 128 columns
constexpr int kMvStage = kMvRows * kMvBlock / 2;
constexpr int kMvWarps = 8;
constexpr int kMvThreads = 32 * (kMvWarps + 1);
constexpr int kMvTokens = 8;
constexpr int kMvMaxSplit = 8;
constexpr int kMvMaxStages = 3;

struct MvLaunch {
    int blocks;    // blocks of K of a CTA
    int stages;
    int tokens;    // most tokens of a CTA
    int split;     // CTAs along K
    int packed;    // the parts of all tokens lie in one operand's eight columns
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Eight codes of a word less the zero: pairs (0, 4), (1, 5), (2, 6), (3, 7) of bf16.  bias: 128 + z twice.
__device__ __forceinline__ void expand_bf16(uint32_t w, uint32_t bias, uint32_t (&r)[4]) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t s = i ? w >> (4 * i) : w;
        uint32_t v;
        asm("lop3.b32 %0, %1, 0x000F000F, 0x43004300, 0xEA;" : "=r"(v) : "r"(s));  // (s & m) | 128
        const __nv_bfloat162 h = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&v),
                                         *reinterpret_cast<const __nv_bfloat162 *>(&bias));
        r[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
}
// The high halves of two binary32 numbers: their first eight bits, cut off.
__device__ __forceinline__ uint32_t high_halves(float a, float b) {
    return prmt(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float rest_of(float v) {
    return v - __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
}
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, int bytes) {
    if (bytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else if (bytes == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cluster_arrive_wait() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float load_cluster(const float *p, uint32_t rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void store_y(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_y(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// The item'th piece of at most `tokens` pairs of one expert: its expert, first pair and pairs (0: none).
__device__ __forceinline__ void find_piece(const Q4Params &p, int item, int tokens, int *found) {
    const int tid = threadIdx.x, lane = tid & 31;
    __shared__ int sums[kMvThreads / 32];
    constexpr int kEach = (LB_ROUTE_MAX_EXPERTS + kMvThreads - 1) / kMvThreads;
    int first[kEach], count[kEach], pieces = 0;
    if (tid == 0) found[2] = 0;
#pragma unroll
    for (int i = 0; i < kEach; i++) {
        const int e = tid * kEach + i;
        first[i] = count[i] = 0;
        if (e < p.E) {
            first[i] = min(max(p.start[e], 0), (int)p.T);
            count[i] = max(min(p.start[e + 1], (int)p.T) - first[i], 0);
        }
        pieces += (count[i] + tokens - 1) / tokens;
    }
    int run = pieces;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int w = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += w;
    }
    if (lane == 31) sums[tid >> 5] = run;
    __syncthreads();
    int before = run - pieces;
#pragma unroll
    for (int w = 0; w < kMvThreads / 32; w++) before += w < (tid >> 5) ? sums[w] : 0;
    if (item >= before && item < before + pieces) {
#pragma unroll
        for (int i = 0; i < kEach; i++) {
            const int n = (count[i] + tokens - 1) / tokens;
            if (item >= before && item < before + n) {
                const int at = (item - before) * tokens;
                found[0] = tid * kEach + i;
                found[1] = first[i] + at;
                found[2] = min(tokens, count[i] - at);
            }
            before += n;
        }
    }
    __syncthreads();
}

// T: the type of x (dense, up; h is fp32) and of a dense y; PARTS: bf16 parts of an x.
template <Q4Use USE, typename T, int PARTS, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(kMvThreads, 2)
    q4_gemv_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ Q4Params p,
                   const __grid_constant__ MvLaunch l) {
    using X = typename std::conditional<USE == kQ4Down, float, T>::type;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint64_t full[kMvMaxStages], empty[kMvMaxStages];
    __shared__ int found[3], row_of[kMvTokens];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slice = l.blocks * kMvBlock, rank = blockIdx.x % l.split;
    const int64_t tile = blockIdx.x / l.split;
    const int k0 = rank * slice, columns = min(p.K - k0, slice);   // (columns <= 0: nothing to add)
    const int blocks = max((columns + kMvBlock - 1) / kMvBlock, 0);
    const int groups = l.blocks * (kMvBlock / GROUP);              // of the slice
    const int x_pitch = 2 * slice + 64;
    uint8_t *ring = smem;
    uint8_t *xs = ring + l.stages * kMvStage;
    uint16_t *ds = reinterpret_cast<uint16_t *>(xs + (l.packed ? kMvTokens : PARTS * l.tokens) * x_pitch);
    uint8_t *zs = reinterpret_cast<uint8_t *>(ds + kMvRows * groups);

    pdl_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < kMvMaxStages; i++) mbar_init(&full[i], 1), mbar_init(&empty[i], kMvWarps);
        fence_mbar_init();
    }
    // experts: which one, and which of its pairs
    int64_t matrix = 0;   // first row of the matrix among all rows
    int t0, tokens;
    if (USE == kQ4Dense) {
        t0 = blockIdx.y * l.tokens;
        tokens = (int)min((int64_t)l.tokens, p.T - t0);
        __syncthreads();
    } else {
        pdl_wait();
        find_piece(p, blockIdx.y, l.tokens, found);
        t0 = found[1], tokens = found[2];
        if (!tokens) return;  // the whole cluster's
        matrix = (int64_t)found[0] * (USE == kQ4Up ? 2 * p.N : p.N);
    }
    // The CTA's 128 rows: an up product's are 64 of the gate and the same 64 of the up rows.
    const int64_t n0 = tile * (USE == kQ4Up ? kMvRows / 2 : kMvRows);
    const int64_t upper = USE == kQ4Up ? p.N + n0 : n0 + kMvRows / 2;   // row of the CTA's row 64
    auto issue = [&](int b) {
        uint64_t *bar = &full[b % l.stages];
        mbar_arrive_expect_tx(bar, kMvStage);
        uint8_t *dst = ring + (b % l.stages) * kMvStage;
#pragma unroll
        for (int j = 0; j < kMvBlock / 128; j++) {
            const int at = (k0 + b * kMvBlock) / 2 + 64 * j;
            tma_load_2d(dst + j * kMvBox, &map, at, (int)(matrix + n0), bar);
            tma_load_2d(dst + j * kMvBox + kMvBox / 2, &map, at, (int)(matrix + upper), bar);
        }
    };
    if (tid == 32 * kMvWarps)
        for (int b = 0; b < min(l.stages, blocks); b++) issue(b);
    // scales and zeros of the slice (they are weights too)
    {
        constexpr int per = kMvBlock / GROUP;      // a block's, of one row
        const int64_t last = USE == kQ4Up ? matrix + 2 * p.N : matrix + p.N;
        for (int i = tid; i < kMvRows * blocks; i += kMvThreads) {
            const int r = i / blocks, b = i % blocks;
            const int64_t row = matrix + (r < kMvRows / 2 ? n0 + r : upper + r - kMvRows / 2);
            if (row >= last) continue;   // the products of rows behind the matrix go nowhere
            const int64_t from = row * p.pitch + k0 / GROUP + b * per;
            const int to = r * groups + b * per;
            // (a row's entries reach to a multiple of eight, a block's may be four)
            if (per == 4) copy_async(smem_u32(ds + to), p.scales + from, 8);
            else
                for (int j = 0; j < per; j += 8)
                    if (k0 / GROUP + b * per + j < p.pitch)
                        copy_async(smem_u32(ds + to + j), p.scales + from + j, 16);
            if (ZEROS) {
                if (per == 4) copy_async(smem_u32(zs + to), p.zeros + from, 4);
                else
                    for (int j = 0; j < per; j += 8)
                        if (k0 / GROUP + b * per + j < p.pitch)
                            copy_async(smem_u32(zs + to + j), p.zeros + from + j, 8);
            }
        }
    }
    if (USE == kQ4Dense) pdl_wait();
    if (USE != kQ4Dense) {
        if (tid < tokens) row_of[tid] = p.order[t0 + tid];
        __syncthreads();
    }
    // x of the slice: operand row (packed ? token * PARTS + part : part * tokens + token), columns in
    // the order of the codes' pairs, zeros behind K
    const int units = blocks * (kMvBlock / 8);
    for (int i = tid; i < tokens * units; i += kMvThreads) {
        const int t = i / units, u = i % units;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        int64_t from = t0 + t;
        bool in = 8 * u < columns;
        if (USE != kQ4Dense) {
            const int pair = row_of[t];
            in = in && pair >= 0 && pair < p.T;
            if (USE == kQ4Up) from = pair / p.k;
        }
        if (in) load8(static_cast<const X *>(p.x) + from * p.x_stride + k0 + 8 * u, v);
#pragma unroll
        for (int part = 0; part < PARTS; part++) {
            const int row = l.packed ? t * PARTS + part : part * tokens + t;
            *reinterpret_cast<uint4 *>(xs + row * x_pitch + 16 * u) =
                make_uint4(high_halves(v[0], v[4]), high_halves(v[1], v[5]), high_halves(v[2], v[6]),
                           high_halves(v[3], v[7]));
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = rest_of(v[j]);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();

    float total[4] = {0.f, 0.f, 0.f, 0.f};
    const int cols = l.packed ? tokens * PARTS : tokens;
    if (warp == kMvWarps) {
        if (lane == 0) {
            int b = min(l.stages, blocks);
            for (; b < blocks; b++) {
                if (!mbar_wait(&empty[b % l.stages], (uint32_t)(b / l.stages - 1) & 1u)) {
                    atomicOr(p.error, 1);
                    break;
                }
                issue(b);
            }
            // no copy may still be landing when the ring is written to or the CTA exits
            for (int i = max(0, b - l.stages); i < b; i++)
                mbar_wait(&full[i % l.stages], (uint32_t)(i / l.stages) & 1u);
        }
    } else {
        const int g = lane >> 2, t = lane & 3;
        const int row = warp * 16 + (lane & 15);      // the row this lane points ldmatrix at
        const uint32_t at_row = smem_u32(ring) + row * 64, turn = (row >> 1) & 3;
        const int scale_row = (warp * 16 + g) * groups;
        const int planes = l.packed ? 1 : PARTS;
        const uint8_t *xrow = xs + g * x_pitch + 16 * t;
        const int plane = tokens * x_pitch;
        const bool have = g < cols;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        for (int b = 0; b < blocks; b++) {
            const int s = b % l.stages;
            if (!__all_sync(0xffffffffu, mbar_wait(&full[s], (uint32_t)(b / l.stages) & 1u))) {
                if (lane == 0) atomicOr(p.error, 1);
                break;
            }
            const int chunks = min(kMvBlock, columns - b * kMvBlock) / 32;   // of 32 columns
#pragma unroll
            for (int j = 0; j < kMvBlock / 128; j++) {
                if (4 * j >= chunks) break;
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    if (4 * j + 2 * h >= chunks) break;
                    uint32_t w[4];   // rows g and g + 8 of chunk 2h, then of chunk 2h + 1
                    ldmatrix4(w, at_row + s * kMvStage + j * kMvBox +
                                     (((uint32_t)(2 * h) + (lane >> 4)) ^ turn) * 16);
#pragma unroll
                    for (int c = 0; c < 2; c++) {
                        const int chunk = 4 * j + 2 * h + c;
                        if (chunk >= chunks) break;   // (K is a multiple of 32)
                        const int gi = b * (kMvBlock / GROUP) + chunk / (GROUP / 32);
                        uint32_t bias[2] = {0x43084308u, 0x43084308u};
                        if (ZEROS) {
                            bias[0] = 0x43004300u | zs[scale_row + gi] * 0x10001u;
                            bias[1] = 0x43004300u | zs[scale_row + 8 * groups + gi] * 0x10001u;
                        }
                        uint32_t a[2][4];
                        expand_bf16(w[2 * c], bias[0], a[0]);
                        expand_bf16(w[2 * c + 1], bias[1], a[1]);
                        const uint8_t *xc = xrow + (b * (kMvBlock / 32) + chunk) * 64;
#pragma unroll
                        for (int q = 0; q < PARTS; q++) {
                            if (q >= planes) break;
                            uint4 x = make_uint4(0, 0, 0, 0);
                            if (have) x = *reinterpret_cast<const uint4 *>(xc + q * plane);
                            mma_bf16(sum, a[0][0], a[1][0], a[0][1], a[1][1], x.x, x.y);
                            mma_bf16(sum, a[0][2], a[1][2], a[0][3], a[1][3], x.z, x.w);
                        }
                        if ((chunk + 1) % (GROUP / 32) == 0) {
                            const float d0 = f16_bits_to_float(ds[scale_row + gi]);
                            const float d1 = f16_bits_to_float(ds[scale_row + 8 * groups + gi]);
                            total[0] = fmaf(d0, sum[0], total[0]);
                            total[1] = fmaf(d0, sum[1], total[1]);
                            total[2] = fmaf(d1, sum[2], total[2]);
                            total[3] = fmaf(d1, sum[3], total[3]);
                            sum[0] = sum[1] = sum[2] = sum[3] = 0.f;
                        }
                    }
                }
            }
            if (b + l.stages < blocks) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[s]);
            }
        }
    }
    // The sums, [operand column][row], where the weights were.
    __syncthreads();
    float *out = reinterpret_cast<float *>(ring);
    constexpr int out_pitch = kMvRows + 4;
    if (warp < kMvWarps) {
        const int r = warp * 16 + (lane >> 2), c = 2 * (lane & 3);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int col = c + (i & 1);
            if (col < cols) out[col * out_pitch + r + 8 * (i >> 1)] = total[i];
        }
    }
    if (l.split > 1) cluster_arrive_wait();
    else __syncthreads();
    auto sum_of = [&](int t, int r) {
        const int parts = l.packed ? PARTS : 1;
        float v = 0.f;
        for (int q = 0; q < parts; q++) {
            const float *at = out + (t * parts + q) * out_pitch + r;
            if (l.split > 1)
                for (int c = 0; c < l.split; c++) v += load_cluster(at, c);
            else
                v += *at;
        }
        return v;
    };
    const int rows = USE == kQ4Up ? kMvRows / 2 : kMvRows;
    const int share = (rows + l.split - 1) / l.split;
    for (int i = tid; i < tokens * share; i += kMvThreads) {
        const int t = i / share, r = rank * share + i % share;
        if (r >= rows || n0 + r >= p.N) continue;
        if (USE == kQ4Dense) {
            store_y(static_cast<T *>(p.y) + (t0 + t) * p.y_stride + n0 + r, sum_of(t, r));
        } else if (USE == kQ4Up) {
            const float gate = sum_of(t, r), up = sum_of(t, r + kMvRows / 2);
            static_cast<float *>(p.y)[(int64_t)(t0 + t) * p.y_stride + n0 + r] =
                gate / (1.f + expf(-gate)) * up;
        } else {
            const int pair = row_of[t];
            if (pair >= 0 && pair < p.T)
                static_cast<float *>(p.y)[(int64_t)pair * p.y_stride + n0 + r] = sum_of(t, r);
        }
    }
    if (l.split > 1) cluster_arrive_wait();   // nobody's sums go before all have read them
}

template <Q4Use USE, typename T, int PARTS, int GROUP>
static int launch_gemv(const Q4Params &p, const CUtensorMap &map, const MvLaunch &l, dim3 grid, size_t smem,
                       cudaStream_t st) {
    auto kernel = p.zeros ? q4_gemv_kernel<USE, T, PARTS, GROUP, true> : q4_gemv_kernel<USE, T, PARTS, GROUP, false>;
    int per_sm;
    if (int e = prepare_kernel((const void *)kernel, kMvThreads, smem, &per_sm)) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid, cfg.blockDim = dim3(kMvThreads), cfg.dynamicSmemBytes = smem, cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)l.split, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr, cfg.numAttrs = l.split > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, map, p, l);
    if (e == cudaSuccess) return LB_OK;
    record_cuda_error(e);
    return LB_ERR_LAUNCH;
}

template <Q4Use USE, typename T, int PARTS>
static int dispatch_gemv(const Q4Params &p, const uint8_t *codes, int64_t rows, int sms, cudaStream_t st) {
    const int64_t tiles = (p.N + (USE == kQ4Up ? kMvRows / 2 : kMvRows) - 1) / (USE == kQ4Up ? kMvRows / 2 : kMvRows);
    const int blocks = (p.K + kMvBlock - 1) / kMvBlock;
    MvLaunch l;
    // Slices of K: one block each where that gives at most eight.
    l.blocks = (blocks + kMvMaxSplit - 1) / kMvMaxSplit;
    l.split = (blocks + l.blocks - 1) / l.blocks;
    l.stages = std::min(l.blocks, kMvMaxStages);
    // Tokens: eight, or as many as their parts' slices fit beside the rest.
    const size_t pitch = 2 * (size_t)l.blocks * kMvBlock + 64;
    const size_t fixed = (size_t)l.stages * kMvStage +
                         (size_t)kMvRows * l.blocks * (kMvBlock / p.group) * (p.zeros ? 3 : 2);
    constexpr size_t kMost = 220 * 1024;
    const int64_t most = USE == kQ4Dense ? p.T : kMvTokens;
    l.tokens = (int)std::min(most, (int64_t)kMvTokens);
    l.packed = l.tokens * PARTS <= kMvTokens;
    while (!l.packed && fixed + (size_t)PARTS * l.tokens * pitch > kMost) {
        l.tokens--;
        l.packed = l.tokens * PARTS <= kMvTokens;
    }
    const size_t smem = fixed + (size_t)(l.packed ? kMvTokens : PARTS * l.tokens) * pitch;
    const int64_t items = USE == kQ4Dense ? (p.T + l.tokens - 1) / l.tokens
                                          : std::min(p.T, std::min((int64_t)p.E, p.T) + p.T / l.tokens);
    CUtensorMap map;
    if (int e = encode_rows_map(&map, codes, (uint64_t)p.K / 2, (uint64_t)rows, 64, kMvRows / 2, 64)) return e;
    // (grid y holds 65535 pieces at most)
    if (items > 65535 || tiles * l.split > 0x7fffffff) return LB_ERR_SHAPE;
    const dim3 grid((unsigned)(tiles * l.split), (unsigned)items);
    switch (p.group) {
        case 32: return launch_gemv<USE, T, PARTS, 32>(p, map, l, grid, smem, st);
        case 64: return launch_gemv<USE, T, PARTS, 64>(p, map, l, grid, smem, st);
        default: return launch_gemv<USE, T, PARTS, 128>(p, map, l, grid, smem, st);
    }
}

int q4_gemv(const Q4Params &p, Q4Use use, int type, const uint8_t *codes, int64_t rows, int sms,
            cudaStream_t st) {
    const bool f32 = type == LB_OUT_F32;
    if (use == kQ4Dense)
        return f32 ? dispatch_gemv<kQ4Dense, float, 3>(p, codes, rows, sms, st)
                   : dispatch_gemv<kQ4Dense, __nv_bfloat16, 1>(p, codes, rows, sms, st);
    if (use == kQ4Up)
        return f32 ? dispatch_gemv<kQ4Up, float, 3>(p, codes, rows, sms, st)
                   : dispatch_gemv<kQ4Up, __nv_bfloat16, 1>(p, codes, rows, sms, st);
    // h in two parts: 16 bits, 2^-8 of a bf16 output's rounding
    return f32 ? dispatch_gemv<kQ4Down, float, 3>(p, codes, rows, sms, st)
               : dispatch_gemv<kQ4Down, float, 2>(p, codes, rows, sms, st);
}

}  // namespace lb
