// lb_q4_gemm_experts.cu -- the experts' products for many tokens (lb_q4_gemm.cuh has the kernel).
#include "lb_q4_gemm.cuh"

namespace lb {

int q4_gemm_experts(const Q4Params &p, const Q4Rows &r, Q4Use use, int type, const uint8_t *codes, int64_t rows,
                    int sms, cudaStream_t st) {
    const bool f32 = type == LB_OUT_F32;
    // Pieces of 176 tokens expand weights less often, ones of 128 have more stages in flight: 32 experts of 2048 x 1024, 50,
    // 87, 137 and 375 tokens each: 76.0, 78, 93 and 194 us against 75.7, 84, 103 and 207 (256 and one accumulator: 76.0, 82,
    // 93 and 189).
    const bool wide = p.T > 64 * (int64_t)p.E;
    if (use == kQ4Up)
        return f32    ? dispatch_gemm<kQ4Up, float, 128>(p, r, codes, rows, sms, st)
               : wide ? dispatch_gemm<kQ4Up, __nv_bfloat16, 176>(p, r, codes, rows, sms, st)
                      : dispatch_gemm<kQ4Up, __nv_bfloat16, 128>(p, r, codes, rows, sms, st);
    return f32    ? dispatch_gemm<kQ4Down, float, 128>(p, r, codes, rows, sms, st)
           : wide ? dispatch_gemm<kQ4Down, __nv_bfloat16, 176>(p, r, codes, rows, sms, st)
                  : dispatch_gemm<kQ4Down, __nv_bfloat16, 128>(p, r, codes, rows, sms, st);
}

}  // namespace lb
