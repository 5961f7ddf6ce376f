// gemm_int8_linear.hip -- the INT8 GEMM with a whole linear's epilogue.
#include "gemm_int8.hpp"

namespace dmpq {

hipError_t launch_gemm_int8_linear(hipStream_t s, const int8_t *qa, const float *sa, const int8_t *qw,
                                   const float *sw, int64_t M, int64_t N, int64_t K, int out_dtype, void *y,
                                   bool amax, float *partial, uint32_t *spart, const LinearEpi &lin) {
    if (M == 0 || N == 0) return hipSuccess;
#define DMPQ_LINEAR(OUT_, EPI_) return launch_i8_paths<OUT_, (EPI_)>(s, qa, sa, qw, sw, M, N, K, y, partial, spart, lin)
    const int epi = linear_epi(amax, lin, N);
    if (out_dtype == 0) {
        if (epi == kEpiLinear) DMPQ_LINEAR(0, kEpiLinear);
        if (epi == (kEpiLinear | kEpiLora)) DMPQ_LINEAR(0, kEpiLinear | kEpiLora);
    }
    if (out_dtype != 1) return hipErrorInvalidValue;
    if ((epi & kEpiHeads) != 0)
        return launch_gemm_int8_linear_heads(s, qa, sa, qw, sw, M, N, K, y, partial, spart, lin, epi);
    switch (epi) {
        case kEpiLinear: DMPQ_LINEAR(1, kEpiLinear);
        case kEpiLinear | kEpiAmax: DMPQ_LINEAR(1, kEpiLinear | kEpiAmax);
        case kEpiLinear | kEpiLora: DMPQ_LINEAR(1, kEpiLinear | kEpiLora);
        case kEpiLinear | kEpiLora | kEpiAmax: DMPQ_LINEAR(1, kEpiLinear | kEpiLora | kEpiAmax);
    }
#undef DMPQ_LINEAR
    return hipErrorInvalidValue;
}

}  // namespace dmpq
