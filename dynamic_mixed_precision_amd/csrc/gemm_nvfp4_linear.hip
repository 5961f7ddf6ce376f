// gemm_nvfp4_linear.hip -- the NVFP4 GEMM with a whole linear's epilogue.
#include "gemm_nvfp4.hpp"

namespace dmpq {

hipError_t launch_gemm_nvfp4_linear(hipStream_t s, const uint8_t *ca, const uint8_t *sa, const float *ga,
                                    const uint8_t *cw, const uint8_t *sw, const float *gw, int64_t M, int64_t N,
                                    int64_t K, int out_dtype, void *y, bool amax, float *partial,
                                    uint32_t *spart, const LinearEpi &lin) {
    if (M == 0 || N == 0) return hipSuccess;
#define DMPQ_LINEAR(OUT_, EPI_) \
    return launch_fp4_paths<OUT_, (EPI_)>(s, ca, sa, ga, cw, sw, gw, M, N, K, y, partial, spart, lin)
    const int epi = linear_epi(amax, lin, N);
    if ((epi & kEpiHeads) == 0 && (epi & kEpiLora) != 0)
        return launch_gemm_nvfp4_linear_lora(s, ca, sa, ga, cw, sw, gw, M, N, K, out_dtype, y, partial, spart, lin, epi);
    if (out_dtype == 0 && epi == kEpiLinear) DMPQ_LINEAR(0, kEpiLinear);
    if (out_dtype != 1) return hipErrorInvalidValue;
    if ((epi & kEpiHeads) != 0)
        return launch_gemm_nvfp4_linear_heads(s, ca, sa, ga, cw, sw, gw, M, N, K, y, partial, spart, lin, epi);
    switch (epi) {
        case kEpiLinear: DMPQ_LINEAR(1, kEpiLinear);
        case kEpiLinear | kEpiAmax: DMPQ_LINEAR(1, kEpiLinear | kEpiAmax);
    }
#undef DMPQ_LINEAR
    return hipErrorInvalidValue;
}

}  // namespace dmpq
