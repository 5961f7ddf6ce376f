// gemm_nvfp4_linear_heads.hip -- the NVFP4 GEMM whose epilogue is the heads of q and k
// (a file of its own: the kernels of one GEMM take minutes to compile).
#include "gemm_nvfp4.hpp"

namespace dmpq {

hipError_t launch_gemm_nvfp4_linear_heads(hipStream_t s, const uint8_t *ca, const uint8_t *sa, const float *ga,
                                          const uint8_t *cw, const uint8_t *sw, const float *gw, int64_t M, int64_t
                                          N, int64_t K, void *y, float *partial, uint32_t *spart, const LinearEpi
                                          &lin, int epi) {
#define DMPQ_LINEAR(OUT_, EPI_) \
    return launch_fp4_paths<OUT_, (EPI_)>(s, ca, sa, ga, cw, sw, gw, M, N, K, y, partial, spart, lin)
    switch (epi) {
        case kEpiLinear | kEpiHeads: DMPQ_LINEAR(1, kEpiLinear | kEpiHeads);
        case kEpiLinear | kEpiHeads | kEpiBand: DMPQ_LINEAR(1, kEpiLinear | kEpiHeads | kEpiBand);
        case kEpiLinear | kEpiHeads | kEpiLora: DMPQ_LINEAR(1, kEpiLinear | kEpiHeads | kEpiLora);
    }
#undef DMPQ_LINEAR
    return hipErrorInvalidValue;
}

}  // namespace dmpq
