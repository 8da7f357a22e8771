// lb_route.cu -- routing of tokens to experts: scores, the chosen experts and their weights, and the
// tokens of each expert.
//
// Mathematics.  A warp takes a token, lane l the experts l, l + 32, ...  Without a bias the scores
// grow with the logits, so the order of the logits is the order of the experts and only the chosen
// ones' scores are needed; with one the keys s + bias are compared.  Two of them may lie closer
// together than binary32 tells apart: the keys carry a bound of their error, and a token of which two
// neighbours in the order (or the last kept and the first dropped group) lie within it is chosen
// again with binary64 keys (about one token in 500 of sigmoid scores of 256 experts), so the experts
// are those of the 64-bit definition while the FP64 units (1/64 of the FP32 rate) stay out of the way.
//
// By expert: up to 64 tokens are one CTA's, which marks each token in its experts' 64-bit masks; a
// pair's place is its expert's start plus the marks below its token, whatever order the marks came in.
// More tokens take a second kernel: the first leaves each CTA's counts per expert, the second adds
// up the counts of the CTAs before its own and places its tokens by the same masks.
//
// What bounds it: instructions.  A token of 256 experts takes about 1500 of a warp (counted over 8191 with sigmoid
// scores, a bias and eight groups).  Each lane keeps its best two keys, so a
// round of the selection is two warp reductions and a few operations of the lane that loses its best; all of its
// keys are looked through again only when that happens to it a second time.
#include "lb_kv4.cuh"

#include <algorithm>
#include <cfloat>

namespace lb {

constexpr int kRouteTile = 64;         // tokens whose marks fit a mask
constexpr int kRouteMaxCtas = 256;     // of the first kernel: bounds what the second adds up
constexpr int kPlaceThreads = 512;
constexpr int kPlaceSums = 4096;        // partial counts: as many as fit

struct RouteParams {
    const void *logits;
    int64_t stride;
    const float *bias;
    const int32_t *live;
    int32_t *ids, *start, *order;
    float *weights;
    uint16_t *counts;  // [CTA][pitch]
    int T, E, k, sigmoid, groups, keep, best, renormalize, tile, pitch;
    int per, inverse;  // experts of a group, and 2^20 / per
    float scale;
    // e / per: inverse is at most 1 (of 2^20 / per) too large, e below 2^10, so the quotient's error is below 1 / per
    __device__ __forceinline__ int group_of(int e) const { return min((uint32_t)(e * inverse) >> 20, 31u); }
};

__device__ __forceinline__ float route_load(const float *p) { return *p; }
__device__ __forceinline__ float route_load(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <typename R>
__device__ __forceinline__ R warp_add(R v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The largest of the lanes' values and, of equal ones, the lowest index; -inf everywhere leaves
// index INT_MAX.  (No value is NaN or -0.)
__device__ __forceinline__ void warp_best(float &v, int &i) {
    const uint32_t b = __float_as_uint(v);
    const uint32_t u = b & 0x80000000u ? ~b : b | 0x80000000u;
    const uint32_t m = __reduce_max_sync(0xffffffffu, u);
    v = __uint_as_float(m & 0x80000000u ? m & 0x7fffffffu : ~m);
    i = (int)__reduce_min_sync(0xffffffffu, u == m && v != -INFINITY ? (uint32_t)i : 0x7fffffffu);
}
// Binary64 numbers (none NaN or -0) as whole ones of the same order, 0 for none: the FP64 units take 64 times as long to
// compare them.
__device__ __forceinline__ uint64_t order_of(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double number_of(uint64_t u) {
    return __longlong_as_double((long long)(u >> 63 ? u & ~(1ull << 63) : ~u));
}
// The largest of the lanes' and, of equal ones, the lowest index.
__device__ __forceinline__ void warp_best(uint64_t &u, int &i) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(u >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(u >> 32) == hi ? (uint32_t)u : 0u);
    const uint64_t best = (uint64_t)hi << 32 | lo;
    i = (int)__reduce_min_sync(0xffffffffu, u == best && u ? (uint32_t)i : 0x7fffffffu);
    u = best;
}

// exp(x - m), with what the difference's rounding left out.
__device__ __forceinline__ float exp_difference(float x, float m) {
    const float t = x - m, back = x - t;
    const float rest = (x - (t + back)) + (back - m);
    const float s = expf(t);
    return t < -100.f ? s : fmaf(s, rest, s);  // (infinite differences leave no rest)
}

struct Chosen {
    int id;        // lane j's expert, -1 without
    bool close;    // binary32 does not tell the order
    float sum;     // softmax: sum of exp(x - max)
};

// Binary64 key of expert e.
template <typename T>
__device__ __forceinline__ double exact_key(const RouteParams &p, const T *row, int e, float m, double sum) {
    const float x = fminf(route_load(row + e), FLT_MAX);
    const double v = exp(p.sigmoid ? -(double)x : (double)x - m);
    return (p.sigmoid ? 1 / (1 + v) : v / sum) + (p.bias ? p.bias[e] : 0.f) + 0.0;
}
// The first k of n <= 32 experts by their binary64 keys, a lane each.
template <typename T>
__device__ __noinline__ int order_again(const RouteParams &p, const T *row, float m, const int *list, int n, int lane) {
    double sum = 0;
    if (!p.sigmoid) {
#pragma unroll 4
        for (int e = lane; e < p.E; e += 32) {
            const float x = route_load(row + e), b = p.bias ? p.bias[e] : 0.f;
            if (x > -INFINITY && b > -INFINITY) sum += exp((double)fminf(x, FLT_MAX) - m);
        }
        sum = warp_add(sum);
    }
    const int e = list[lane < n ? lane : 0];
    uint64_t key = lane < n ? order_of(exact_key(p, row, e, m, sum)) : 0;
    int id = -1;
#pragma unroll 1
    for (int j = 0; j < p.k; j++) {
        uint64_t v = key;
        int at = e;
        warp_best(v, at);
        if (!v) break;
        if (lane == j) id = at;
        if (lane < n && e == at) key = 0;
    }
    return id;
}

// The k experts of a token, one per lane.  x: the lane's logits (-inf: not to be chosen), b: their biases, m: the warp's
// largest logit.
template <int EL, typename T>
__device__ __forceinline__ Chosen choose(const RouteParams &p, const T *row, const float (&x)[EL], const float (&b)[EL], float m,
                                         float *keys, int lane) {
    const bool plain = !p.bias && p.best == 1;
    const float none = -INFINITY;
    Chosen c{-1, false, 0.f};
    bool groups = false;   // two groups lie too close together
    float key[EL], tol = 0.f;
    if (plain) {
#pragma unroll
        for (int i = 0; i < EL; i++) key[i] = x[i] + 0.f;  // -0 and 0 are the same number
        if (!p.sigmoid && !p.renormalize) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < EL; i++) s += x[i] > -INFINITY ? exp_difference(x[i], m) : 0.f;
            c.sum = warp_add(s);
        }
    } else {
        float s = 0.f, most = 0.f;
#pragma unroll
        for (int i = 0; i < EL; i++) {
            const bool in = x[i] > -INFINITY;
            most = fmaxf(most, in ? fabsf(b[i]) : 0.f);
            if (p.sigmoid) key[i] = __fdividef(1.f, 1.f + __expf(-x[i]));
            else key[i] = in ? exp_difference(x[i], m) : 0.f, s += key[i];
        }
        float by = 1.f;
        if (!p.sigmoid) {
            s = warp_add(s);
            c.sum = s;
            by = __fdividef(1.f, s);
        }
#pragma unroll
        for (int i = 0; i < EL; i++) key[i] = x[i] > -INFINITY ? key[i] * by + b[i] + 0.f : none;
        // A sigmoid: exp to 2 + 1.2 |x| units of its last place changes it by s (1 - s) times that, a unit at most; a
        // sum, a reciprocal and a sum: below 2^-21.  A softmax: exp to two units, a sum of up to 1024 scores in 32
        // chains, a reciprocal, a product and a sum: below 2^-18 of the largest score.
        tol = (p.sigmoid ? 0x1p-21f : 0x1p-18f * by) + 0x1p-22f * warp_max(most) + 1e-37f;
        // biases so large that sums of two overflow, or infinite: all in binary64
        if (!(tol < 0x1p100f)) c.close = groups = true;
    }
    if (p.groups > 1) {
        // lanes [g * part, (g + 1) * part) look through group g
        const int per = p.per, part = 32 >> (32 - __clz(p.groups - 1));
        const int g = lane / part;
#pragma unroll
        for (int i = 0; i < EL; i++)
            if (lane + 32 * i < p.E) keys[lane + 32 * i] = key[i];
        __syncwarp();
        float first = none, second = none;
        if (g < p.groups)
#pragma unroll 4
            for (int e = lane % part; e < per; e += part) {
                const float v = keys[g * per + e], low = first < v ? first : v;
                first = first < v ? v : first;
                second = second < low ? low : second;
            }
        __syncwarp();
        for (int o = 1; o < part; o <<= 1) {
            const float a = __shfl_xor_sync(0xffffffffu, first, o), d = __shfl_xor_sync(0xffffffffu, second, o);
            const float low = first < a ? first : a;
            first = first < a ? a : first;
            second = second < d ? d : second;
            second = second < low ? low : second;
        }
        const float value = p.best == 2 && second > none ? first + second + 0.f : first;
        uint32_t kept = 0;
        float last = 0.f;
        for (int j = 0; j <= p.keep; j++) {
            float v = g < p.groups && !(kept >> g & 1) ? value : none;
            int at = g;
            warp_best(v, at);
            if (v == none) break;
            if (j == p.keep) {
                if (!plain && last - v <= 4 * tol) c.close = groups = true;
                break;
            }
            kept |= 1u << at;
            last = v;
        }
        // (a lane's experts lie 32 apart)
        int at = lane;
#pragma unroll
        for (int i = 0; i < EL; i++, at += 32)
            if (!(kept >> p.group_of(at) & 1)) key[i] = none;
    }
    // the lane's best two of those not taken
    uint32_t taken = 0;
    float v1, v2;
    int i1, i2;
    auto look = [&]() {
        v1 = v2 = none, i1 = i2 = lane;
#pragma unroll
        for (int i = 0; i < EL; i++) {
            const float v = taken >> i & 1 ? none : key[i];
            if (v > v1) v2 = v1, i2 = i1, v1 = v, i1 = lane + 32 * i;
            else if (v > v2) v2 = v, i2 = lane + 32 * i;
        }
    };
    look();
    bool second = true;   // v2 is known
    float last = 0.f;
#pragma unroll 1
    for (int j = 0; j <= p.k; j++) {
        if (j == p.k && plain) break;
        float v = v1;
        int at = i1;
        warp_best(v, at);
        if (v == none) break;
        if (!plain && j && last - v <= 2 * tol) c.close = true;
        if (j == p.k) break;
        last = v;
        if (lane == j) c.id = at;
        bool again = false;
        if (at == i1 && v1 > none) {
            taken |= 1u << (at >> 5);
            again = !second;
            v1 = v2, i1 = i2, second = false;
        }
        if (__any_sync(0xffffffffu, again)) {
            if (again) look(), second = true;
            __syncwarp();
        }
    }
    if (c.close && !groups) {
        // Whatever lies below the last one's key by twice the error is not among the first k: only the others, mostly k
        // and one more, are looked at again.
        int *list = reinterpret_cast<int *>(keys), n = 0;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < EL; i++) {
            const bool in = key[i] > none && key[i] >= last - 2 * tol;
            const uint32_t all = __ballot_sync(0xffffffffu, in);
            if (in) list[n + __popc(all & ((1u << lane) - 1))] = lane + 32 * i;
            n += __popc(all);
        }
        __syncwarp();
        if (n <= 32) c.id = order_again(p, row, m, list, n, lane), c.close = false;
        __syncwarp();
    }
    return c;
}
// The same with binary64 keys, in shared memory: few tokens come here, but a kernel lasts as long as its last one, so four
// keys' chains of operations run side by side and are then compared as whole numbers (one at a time and as they
// are: 40 us for a token of 256).
template <typename T>
__device__ __noinline__ int choose_again(const RouteParams &p, const T *row, float m, uint64_t *keys, int lane) {
    double s = 0;
#pragma unroll 1
    for (int e0 = lane; e0 < p.E; e0 += 128) {
        float x[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int e = e0 + 32 * i;
            const float v = e < p.E ? route_load(row + e) : -INFINITY;
            x[i] = v > -INFINITY ? fminf(v, FLT_MAX) : -INFINITY;   // (NaN is not)
            b[i] = e < p.E && p.bias ? p.bias[e] : 0.f;
        }
        double v[4];
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = exp(p.sigmoid ? -(double)x[i] : (double)x[i] - m);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int e = e0 + 32 * i;
            const bool in = x[i] > -INFINITY && b[i] > -INFINITY;
            if (p.sigmoid) v[i] = 1 / (1 + v[i]) + b[i] + 0.0;
            else if (in) s += v[i];
            if (e < p.E) keys[e] = in ? order_of(v[i]) : 0;
        }
    }
    if (!p.sigmoid) {
        s = warp_add(s);
#pragma unroll 4
        for (int e = lane; e < p.E; e += 32)
            if (keys[e]) keys[e] = order_of(number_of(keys[e]) / s + (p.bias ? p.bias[e] : 0.f) + 0.0);
    }
    __syncwarp();
    if (p.groups > 1) {   // a lane per group
        uint64_t first = 0, second = 0;
#pragma unroll 4
        for (int e = 0; e < p.per; e++) {
            const uint64_t v = lane < p.groups ? keys[lane * p.per + e] : 0;
            const uint64_t low = v < first ? v : first;
            first = v < first ? first : v;
            second = low < second ? second : low;
        }
        uint64_t value = p.best == 2 && second ? order_of(number_of(first) + number_of(second) + 0.0) : first;
        uint32_t kept = 0;
#pragma unroll 1
        for (int j = 0; j < p.keep; j++) {
            uint64_t v = value;
            int at = lane;
            warp_best(v, at);
            if (!v) break;
            kept |= 1u << at;
            if (lane == at) value = 0;
        }
        for (int e = lane; e < p.E; e += 32)
            if (!(kept >> p.group_of(e) & 1)) keys[e] = 0;
        __syncwarp();
    }
    int id = -1;
#pragma unroll 1
    for (int j = 0; j < p.k; j++) {
        uint64_t v = 0;
        int at = lane;
#pragma unroll 4
        for (int e = lane; e < p.E; e += 32) {
            const uint64_t w = keys[e];
            if (w > v) v = w, at = e;
        }
        warp_best(v, at);
        if (!v) break;
        if (lane == j) id = at;
        if (lane == (at & 31)) keys[at] = 0;
        __syncwarp();
    }
    return id;
}

// Weight of the expert whose logit is x, one per lane (in: the lane has one).
__device__ __forceinline__ float weight_of(const RouteParams &p, float x, bool in, float m, float sum) {
    float s;
    if (!p.renormalize) {
        s = p.sigmoid ? 1.f / (1.f + expf(-x)) : exp_difference(x, m) / sum;
        return in ? s * p.scale : 0.f;
    }
    // the largest chosen logit's power of e goes out of all of them, so their sum is never 0 and only a weight that is itself
    // below binary32's normal numbers has fewer bits; sigmoids from a logit above 0 on are 1/2 at least as they are
    const float top = warp_max(in ? x : -INFINITY);
    if (p.sigmoid && top > 0.f) {
        const float e = expf(-fabsf(x));
        s = (x < 0.f ? e : 1.f) / (1.f + e);
    } else if (p.sigmoid) {
        s = exp_difference(x, top) / (1.f + expf(x));
    } else {
        s = exp_difference(x, top);
    }
    s = in ? s : 0.f;
    const float all = warp_add(s);
    return in ? s / all * p.scale : 0.f;
}

// Exclusive sums over the experts of `count` (shared, [E]) in place; all threads.  Returns the total.
template <int THREADS>
__device__ __forceinline__ int scan_experts(int32_t *count, int E, int32_t *part) {
    constexpr int kEach = LB_ROUTE_MAX_EXPERTS / THREADS > 1 ? LB_ROUTE_MAX_EXPERTS / THREADS : 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int v[kEach], sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; i++) {
        v[i] = tid * kEach + i < E ? count[tid * kEach + i] : 0;
        sum += v[i];
    }
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int w = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += w;
    }
    if (lane == 31) part[warp] = run;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; w++) {
        const int c = part[w];
        before += w < warp ? c : 0;
        total += c;
    }
    before += run - sum;
#pragma unroll
    for (int i = 0; i < kEach; i++) {
        if (tid * kEach + i < E) count[tid * kEach + i] = before;
        before += v[i];
    }
    __syncthreads();
    return total;
}

template <typename T, int EL, int THREADS, bool ALONE>
__global__ void __launch_bounds__(THREADS) route_kernel(const __grid_constant__ RouteParams p) {
    extern __shared__ uint64_t route_smem[];  // marks or counts [E], then with groups keys [warp][E]
    __shared__ int32_t start[ALONE ? LB_ROUTE_MAX_EXPERTS : 1], part[THREADS / 32];
    constexpr int kWarps = THREADS / 32, kHeld = kRouteTile / kWarps;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t *mark = route_smem;
    int32_t *count = reinterpret_cast<int32_t *>(route_smem);
    double *keys = reinterpret_cast<double *>(route_smem + p.E) + (p.bias || p.best == 2 || p.groups > 1 ? warp * p.E : 0);
    pdl_launch_dependents();
    for (int e = tid; e < p.E; e += THREADS) mark[e] = 0;
    __syncthreads();
    pdl_wait();
    const int live = p.live ? min(max(*p.live, 0), p.T) : p.T;
    const int t0 = blockIdx.x * p.tile, t1 = min(t0 + p.tile, p.T);
    int held[ALONE ? kHeld : 1];
    for (int n = 0; t0 + n * kWarps < t1; n++) {
        const int t = t0 + n * kWarps + warp;
        int id = -1;
        if (t < t1) {
            float w = 0.f;
            if (t < live) {
                const T *row = static_cast<const T *>(p.logits) + t * p.stride;
                float x[EL], b[EL], m = -INFINITY;
#pragma unroll
                for (int i = 0; i < EL; i++) {
                    const int e = lane + 32 * i;
                    x[i] = e < p.E ? route_load(row + e) : -INFINITY;
                    b[i] = p.bias && e < p.E ? p.bias[e] : 0.f;
                }
#pragma unroll
                for (int i = 0; i < EL; i++) {
                    x[i] = x[i] > -INFINITY && b[i] > -INFINITY ? fminf(x[i], FLT_MAX) : -INFINITY;   // (NaN is not)
                    m = fmaxf(m, x[i]);
                }
                if (!p.sigmoid) m = warp_max(m);
                Chosen c = choose<EL, T>(p, row, x, b, m, reinterpret_cast<float *>(keys), lane);
                if (c.close) c.id = choose_again(p, row, m, reinterpret_cast<uint64_t *>(keys), lane);
                id = c.id;
                const float xj = id >= 0 ? fminf(route_load(row + id), FLT_MAX) : 0.f;
                w = weight_of(p, xj, id >= 0, m, c.sum);
            }
            if (lane < p.k) {
                p.ids[(int64_t)t * p.k + lane] = id;
                p.weights[(int64_t)t * p.k + lane] = w;
            }
            if (id >= 0) {
                if (ALONE) atomicOr(reinterpret_cast<unsigned long long *>(mark + id), 1ull << (t - t0));
                else atomicAdd(count + id, 1);
            }
        }
        if (ALONE) {
#pragma unroll
            for (int i = 0; i < kHeld; i++)
                if (i == n) held[i] = id;
        }
    }
    __syncthreads();
    if constexpr (!ALONE) {
        for (int e = tid; e < p.pitch; e += THREADS)
            p.counts[(int64_t)blockIdx.x * p.pitch + e] = e < p.E ? (uint16_t)count[e] : 0;
    } else {
        for (int e = tid; e < p.E; e += THREADS) start[e] = __popcll(mark[e]);
        __syncthreads();
        const int total = scan_experts<THREADS>(start, p.E, part);
        for (int e = tid; e <= p.E; e += THREADS) p.start[e] = e < p.E ? start[e] : total;
#pragma unroll
        for (int n = 0; n < kHeld; n++) {
            const int at = n * kWarps + warp;
            if (t0 + at < t1 && held[n] >= 0)
                p.order[start[held[n]] + __popcll(mark[held[n]] & ((1ull << at) - 1))] = at * p.k + lane;
        }
        for (int i = total + tid; i < p.T * p.k; i += THREADS) p.order[i] = -1;
    }
}

// The second kernel: CTA b places the tokens of the first one's CTA b.
__global__ void __launch_bounds__(kPlaceThreads) place_kernel(const __grid_constant__ RouteParams p) {
    __shared__ int32_t before[LB_ROUTE_MAX_EXPERTS], start[LB_ROUTE_MAX_EXPERTS], part[kPlaceThreads / 32];
    __shared__ uint64_t mark[LB_ROUTE_MAX_EXPERTS];
    __shared__ __align__(16) uint32_t sums[2][kPlaceSums];   // of all CTAs, of those before this one: [threads' share][expert]
    const int tid = threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    // a thread adds up eight experts' counts over every `parts`-th CTA
    const int words = p.pitch / 8, parts = min(kPlaceThreads / words, kPlaceSums / p.pitch);
    const int w = tid % words, q = tid / words;
    if (q < parts) {
        uint32_t all[8] = {0, 0, 0, 0, 0, 0, 0, 0}, mine[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        const uint4 *counts = reinterpret_cast<const uint4 *>(p.counts) + w;
#pragma unroll 4
        for (int c = q; c < (int)gridDim.x; c += parts) {
            const uint4 v = counts[c * words];
            const uint32_t a[4] = {v.x, v.y, v.z, v.w};
            const bool early = c < (int)blockIdx.x;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                all[2 * i] += a[i] & 0xffff, all[2 * i + 1] += a[i] >> 16;
                if (early) mine[2 * i] += a[i] & 0xffff, mine[2 * i + 1] += a[i] >> 16;
            }
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint32_t *from = i ? mine : all;
            uint4 *to = reinterpret_cast<uint4 *>(&sums[i][q * p.pitch + 8 * w]);
            to[0] = make_uint4(from[0], from[1], from[2], from[3]);
            to[1] = make_uint4(from[4], from[5], from[6], from[7]);
        }
    }
    __syncthreads();
    for (int e = tid; e < p.E; e += kPlaceThreads) {
        uint32_t all = 0, mine = 0;
        for (int i = 0; i < parts; i++) all += sums[0][i * p.pitch + e], mine += sums[1][i * p.pitch + e];
        start[e] = (int)all, before[e] = (int)mine;
    }
    __syncthreads();
    const int total = scan_experts<kPlaceThreads>(start, p.E, part);
    if (blockIdx.x == 0)
        for (int e = tid; e <= p.E; e += kPlaceThreads) p.start[e] = e < p.E ? start[e] : total;
    for (int e = tid; e < p.E; e += kPlaceThreads) before[e] += start[e];
    const int t0 = blockIdx.x * p.tile, t1 = min(t0 + p.tile, p.T);
    for (int t = t0; t < t1; t += kRouteTile) {
        __syncthreads();
        for (int e = tid; e < p.E; e += kPlaceThreads) mark[e] = 0;
        __syncthreads();
        const int n = min(kRouteTile, t1 - t) * p.k;
        const int32_t *ids = p.ids + (int64_t)t * p.k;
        for (int i = tid; i < n; i += kPlaceThreads)
            if (ids[i] >= 0)
                atomicOr(reinterpret_cast<unsigned long long *>(mark + ids[i]), 1ull << (i / p.k));
        __syncthreads();
        for (int i = tid; i < n; i += kPlaceThreads) {
            const int e = ids[i];
            if (e >= 0) p.order[before[e] + __popcll(mark[e] & ((1ull << (i / p.k)) - 1))] = t * p.k + i;
        }
        __syncthreads();
        for (int e = tid; e < p.E; e += kPlaceThreads) before[e] += __popcll(mark[e]);
    }
    const int64_t pairs = (int64_t)p.T * p.k;
    for (int64_t i = total + blockIdx.x * (int64_t)kPlaceThreads + tid; i < pairs;
         i += (int64_t)gridDim.x * kPlaceThreads)
        p.order[i] = -1;
}

static int route_tile(int64_t T) {
    return (int)((T + kRouteTile * kRouteMaxCtas - 1) / (kRouteTile * kRouteMaxCtas)) * kRouteTile;
}

template <typename T, int EL, int THREADS>
static int launch_route(RouteParams p, cudaStream_t st) {
    const size_t smem = (size_t)p.E * 8 * (1 + (p.groups > 1 || p.best == 2 || p.bias ? THREADS / 32 : 0));
    int per_sm;
    if (THREADS > 256 && p.T <= 8) return launch_route<T, EL, 256>(p, st);   // (a warp per token does)
    if (p.T <= kRouteTile) {
        p.tile = kRouteTile;
        auto kernel = route_kernel<T, EL, THREADS, true>;
        if (int e = prepare_kernel((const void *)kernel, THREADS, smem, &per_sm)) return e;
        return launch_pdl(kernel, dim3(1), dim3(THREADS), smem, st, p);
    }
    p.tile = route_tile(p.T);
    const int ctas = (p.T + p.tile - 1) / p.tile;
    auto kernel = route_kernel<T, EL, THREADS, false>;
    if (int e = prepare_kernel((const void *)kernel, THREADS, smem, &per_sm)) return e;
    if (int e = launch_pdl(kernel, dim3(ctas), dim3(THREADS), smem, st, p)) return e;
    return launch_pdl(place_kernel, dim3(ctas), dim3(kPlaceThreads), 0, st, p);
}

template <typename T>
static int dispatch_route(const RouteParams &p, cudaStream_t st) {
    if (p.E <= 64) return launch_route<T, 2, 1024>(p, st);
    if (p.E <= 128) return launch_route<T, 4, 1024>(p, st);
    if (p.E <= 256) return launch_route<T, 8, 1024>(p, st);
    return launch_route<T, 32, 256>(p, st);
}

}  // namespace lb

LB_EXPORT size_t lb_route_workspace_bytes(int64_t T, int E) {
    using namespace lb;
    if (T < 0 || T > (1 << 20) || E < 1 || E > LB_ROUTE_MAX_EXPERTS) return 0;
    if (T <= kRouteTile) return 16;
    // (counts of as many CTAs as T, or any smaller number of tokens, can take: fewer where tiles have grown)
    const int64_t ctas = std::min<int64_t>((T + kRouteTile - 1) / kRouteTile, kRouteMaxCtas);
    return (size_t)ctas * ((E + 7) / 8 * 8) * 2;
}

LB_EXPORT int lb_route(const void *logits, int type, int64_t stride, int64_t T, int E, int k,
                       const lb_route_rules *rules, int32_t *ids, float *weights, int32_t *expert_start,
                       int32_t *order, void *workspace, size_t workspace_bytes, void *stream) {
    using namespace lb;
    if (!rules || !expert_start || !workspace || (T > 0 && (!logits || !ids || !weights || !order)))
        return LB_ERR_NULL;
    const lb_route_rules &r = *rules;
    if ((type != LB_OUT_F32 && type != LB_OUT_BF16) || T < 0 || T > (1 << 20) || E < 1 ||
        E > LB_ROUTE_MAX_EXPERTS || k < 1 || k > LB_ROUTE_MAX_CHOSEN || k > E || stride < E ||
        (r.scoring != LB_ROUTE_SOFTMAX && r.scoring != LB_ROUTE_SIGMOID) || r.groups < 1 ||
        r.groups > 32 || E % r.groups != 0 || r.keep_groups < 1 || r.keep_groups > r.groups ||
        (r.group_best != 1 && r.group_best != 2) || !(r.scale > -INFINITY && r.scale < INFINITY) ||
        workspace_bytes < lb_route_workspace_bytes(T, E))
        return LB_ERR_SHAPE;
    if (!aligned_to(logits, type == LB_OUT_F32 ? 4 : 2) || !aligned16(workspace)) return LB_ERR_ALIGN;
    for (const void *q : {(const void *)ids, (const void *)weights, (const void *)expert_start,
                          (const void *)order, (const void *)r.bias_opt, (const void *)r.live_opt})
        if (!aligned_to(q, 4)) return LB_ERR_ALIGN;
    DeviceInfo di;
    if (int e = current_device_info(&di)) return e;
    RouteParams p{};
    p.logits = logits, p.stride = stride, p.bias = r.bias_opt, p.live = r.live_opt;
    p.ids = ids, p.weights = weights, p.start = expert_start, p.order = order;
    p.counts = static_cast<uint16_t *>(workspace);
    p.T = (int)T, p.E = E, p.k = k, p.sigmoid = r.scoring == LB_ROUTE_SIGMOID;
    p.groups = r.groups, p.keep = r.keep_groups, p.best = r.group_best;
    p.per = E / r.groups, p.inverse = (1 << 20) / p.per + 1;
    p.renormalize = r.renormalize != 0, p.scale = r.scale, p.pitch = (E + 7) / 8 * 8;
    cudaStream_t st = as_stream(stream);
    return type == LB_OUT_F32 ? dispatch_route<float>(p, st) : dispatch_route<__nv_bfloat16>(p, st);
}
