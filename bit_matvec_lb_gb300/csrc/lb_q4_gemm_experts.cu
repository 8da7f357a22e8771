// lb_q4_gemm_experts.cu -- the experts' products for many tokens (lb_q4_gemm.cuh has the kernel).
#include "lb_q4_gemm.cuh"

namespace lb {

int q4_gemm_experts(const Q4Params &p, const Q4Rows &r, Q4Use use, int type, const uint8_t *codes, int64_t rows,
                    int sms, cudaStream_t st) {
    const bool f32 = type == LB_OUT_F32;
    // Pieces of 256 tokens expand weights half as often, ones of 128 hide what happens behind an item's products: the
    // first are ahead from about 160 tokens per expert on (512: 551 against 576 us; 49: 201 against 188).
    const bool wide = p.T > 160 * (int64_t)p.E;
    if (use == kQ4Up)
        return f32    ? dispatch_gemm<kQ4Up, float, 128>(p, r, codes, rows, sms, st)
               : wide ? dispatch_gemm<kQ4Up, __nv_bfloat16, 256>(p, r, codes, rows, sms, st)
                      : dispatch_gemm<kQ4Up, __nv_bfloat16, 128>(p, r, codes, rows, sms, st);
    return f32    ? dispatch_gemm<kQ4Down, float, 128>(p, r, codes, rows, sms, st)
           : wide ? dispatch_gemm<kQ4Down, __nv_bfloat16, 256>(p, r, codes, rows, sms, st)
                  : dispatch_gemm<kQ4Down, __nv_bfloat16, 128>(p, r, codes, rows, sms, st);
}

}  // namespace lb
