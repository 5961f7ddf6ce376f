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
    const int epi = kEpiLinear | (amax ? kEpiAmax : 0) | (lin.lora.t ? kEpiLora : 0) | (lin.qk.D ? kEpiHeads : 0);
    if (out_dtype == 0) {
        if (epi == kEpiLinear) DMPQ_LINEAR(0, kEpiLinear);
        if (epi == (kEpiLinear | kEpiLora)) DMPQ_LINEAR(0, kEpiLinear | kEpiLora);
    }
    if (out_dtype != 1) return hipErrorInvalidValue;
    switch (epi) {
        case kEpiLinear: DMPQ_LINEAR(1, kEpiLinear);
        case kEpiLinear | kEpiAmax: DMPQ_LINEAR(1, kEpiLinear | kEpiAmax);
        case kEpiLinear | kEpiLora: DMPQ_LINEAR(1, kEpiLinear | kEpiLora);
        case kEpiLinear | kEpiLora | kEpiAmax: DMPQ_LINEAR(1, kEpiLinear | kEpiLora | kEpiAmax);
        case kEpiLinear | kEpiHeads: DMPQ_LINEAR(1, kEpiLinear | kEpiHeads);
        case kEpiLinear | kEpiHeads | kEpiLora: DMPQ_LINEAR(1, kEpiLinear | kEpiHeads | kEpiLora);
    }
#undef DMPQ_LINEAR
    return hipErrorInvalidValue;
}

}  // namespace dmpq
