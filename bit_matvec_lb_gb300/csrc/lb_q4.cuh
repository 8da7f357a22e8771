// lb_q4.cuh -- what the kernels over 4-bit weights with group scales share: the parameters of a
// product, of the experts' products, and the host checks.
#pragma once
#include "lb_kv4.cuh"

namespace lb {

// What a product is part of: y = W x itself, the experts' gate and up rows (h out), or their down
// rows (h in, one output row per pair).
enum Q4Use { kQ4Dense, kQ4Up, kQ4Down };

struct Q4Params {
    const uint16_t *scales;   // [rows][pitch]
    const uint8_t *zeros;     // [rows][pitch], or NULL
    const void *x;            // dense, up: the tokens; down: h [pair position][K] fp32
    void *y;                  // dense: [T][N]; up: h; down: [pair][N] fp32
    int64_t x_stride, y_stride;
    int64_t N;                // output rows of a matrix: dense, down; up: ffn
    int64_t T;                // tokens; experts: pairs
    int K, group, pitch;
    const int32_t *start, *order;  // experts
    int E, k;
    int *error;
};

inline int q4_pitch(int64_t K, int group) { return (int)((K / group + 7) / 8 * 8); }
inline bool q4_group_ok(int group) { return group == 32 || group == 64 || group == 128; }
inline bool q4_type_ok(int type) { return type == LB_OUT_F32 || type == LB_OUT_BF16; }

__device__ __forceinline__ uint32_t bits_of(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }
__device__ __forceinline__ __half2 half2_of(uint32_t v) { return *reinterpret_cast<const __half2 *>(&v); }

// Eight codes of a word less the zero, times the scale: pairs (0, 4), (1, 5), (2, 6), (3, 7) of fp16.  The codes
// go under the exponent of 1024, at the last place or (times 16) four above it.
// low: 1024 + z twice, high: -(64 + z) twice.
template <bool SCALED>
__device__ __forceinline__ void expand_f16(uint32_t w, __half2 low, __half2 high, __half2 d, uint32_t *r) {
    const __half2 sixteenth = half2_of(0x2C002C00u);
    const uint32_t s = w >> 8;
    uint32_t v[4];
    asm("lop3.b32 %0, %1, 0x000F000F, 0x64006400, 0xEA;" : "=r"(v[0]) : "r"(w));
    asm("lop3.b32 %0, %1, 0x00F000F0, 0x64006400, 0xEA;" : "=r"(v[1]) : "r"(w));
    asm("lop3.b32 %0, %1, 0x000F000F, 0x64006400, 0xEA;" : "=r"(v[2]) : "r"(s));
    asm("lop3.b32 %0, %1, 0x00F000F0, 0x64006400, 0xEA;" : "=r"(v[3]) : "r"(s));
#pragma unroll
    for (int i = 0; i < 4; i++) {
        __half2 h = i & 1 ? __hfma2(half2_of(v[i]), sixteenth, high) : __hsub2(half2_of(v[i]), low);
        if (SCALED) h = __hmul2(h, d);
        r[i] = bits_of(h);
    }
}

// Exponent field of the power of two that takes a number m >= 0 (its bits) to [2^14, 2^15), kept to powers whose
// inverse (254 less the field) is normal too.
__device__ __forceinline__ uint32_t q4_power(uint32_t m) { return (uint32_t)min(max(268 - (int)(m >> 23), 1), 253); }

// One to eight tokens (or an expert's tokens, eight at a time), on mma.sync: lb_q4_gemv.cu.
// codes: all matrices' rows, `rows` of them.
int q4_gemv(const Q4Params &p, Q4Use use, int type, const uint8_t *codes, int64_t rows, int sms,
            cudaStream_t st);

// More tokens, on tcgen05: lb_q4_gemm.cuh.  r is what q4_rows left: rows of K fp16 numbers (and with
// fp32 tensors, behind all of them, their second parts), each scaled by a power of two that row_scale
// takes back.
struct Q4Rows {
    const uint16_t *x;
    const float *row_scale;
    int64_t rows;        // of a part
};
int q4_gemm_dense(const Q4Params &p, const Q4Rows &r, int type, const uint8_t *codes, int64_t rows, int sms,
                  cudaStream_t st);
int q4_gemm_experts(const Q4Params &p, const Q4Rows &r, Q4Use use, int type, const uint8_t *codes, int64_t rows,
                    int sms, cudaStream_t st);
// rows [n][K] of x (fp32 if f32 else bf16), x_stride apart -> fp16 parts and row_scale.  n_opt: NULL, or where
// the number of rows that are there lies.  order: NULL, or the n pairs, whose rows of x are pair / k.
int q4_rows(const void *x, bool f32, int64_t x_stride, int64_t n, int K, const int32_t *n_opt,
            const int32_t *order, int k, int parts, uint16_t *to, float *row_scale, cudaStream_t st);

}  // namespace lb
