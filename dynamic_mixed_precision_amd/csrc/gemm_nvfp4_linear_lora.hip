// gemm_nvfp4_linear_lora.hip -- the NVFP4 GEMM with a whole linear's epilogue and
// adapters (a file of its own: the kernels of one GEMM take minutes to compile).
#include "gemm_nvfp4.hpp"

namespace dmpq {

hipError_t launch_gemm_nvfp4_linear_lora(hipStream_t s, const uint8_t *ca, const uint8_t *sa, const float *ga,
                                         const uint8_t *cw, const uint8_t *sw, const float *gw, int64_t M, int64_t N,
                                         int64_t K, int out_dtype, void *y, float *partial, uint32_t *spart,
                                         const LinearEpi &lin, int epi) {
#define DMPQ_LINEAR(OUT_, EPI_) \
    return launch_fp4_paths<OUT_, (EPI_)>(s, ca, sa, ga, cw, sw, gw, M, N, K, y, partial, spart, lin)
    if (out_dtype == 0 && epi == (kEpiLinear | kEpiLora)) DMPQ_LINEAR(0, kEpiLinear | kEpiLora);
    if (out_dtype == 1 && epi == (kEpiLinear | kEpiLora)) DMPQ_LINEAR(1, kEpiLinear | kEpiLora);
    if (out_dtype == 1 && epi == (kEpiLinear | kEpiLora | kEpiAmax)) DMPQ_LINEAR(1, kEpiLinear | kEpiLora | kEpiAmax);
#undef DMPQ_LINEAR
    return hipErrorInvalidValue;
}

}  // namespace dmpq
