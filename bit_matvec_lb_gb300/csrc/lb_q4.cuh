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

// One to eight tokens (or an expert's tokens, eight at a time), on mma.sync: lb_q4_gemv.cu.
// codes: all matrices' rows, `rows` of them.
int q4_gemv(const Q4Params &p, Q4Use use, int type, const uint8_t *codes, int64_t rows, int sms,
            cudaStream_t st);

// More tokens, on tcgen05: lb_q4_gemm.cu.  r is what q4_rows left: rows of K fp16 numbers (and with
// fp32 tensors, behind all of them, their second parts), each scaled by a power of two that row_scale
// takes back.
struct Q4Rows {
    const uint16_t *x;
    const float *row_scale;
    int64_t rows;        // of a part
};
int q4_gemm(const Q4Params &p, const Q4Rows &r, Q4Use use, int type, const uint8_t *codes, int64_t rows,
            int sms, cudaStream_t st);
// rows [n][K] of x (fp32 if f32 else bf16), x_stride apart -> fp16 parts and row_scale.  n_opt: NULL, or where
// the number of rows that are there lies.  order: NULL, or the n pairs, whose rows of x are pair / k.
int q4_rows(const void *x, bool f32, int64_t x_stride, int64_t n, int K, const int32_t *n_opt,
            const int32_t *order, int k, int parts, uint16_t *to, float *row_scale, cudaStream_t st);

}  // namespace lb
