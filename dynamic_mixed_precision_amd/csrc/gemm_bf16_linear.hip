// gemm_bf16_linear.hip -- the BF16 GEMM with a whole linear's epilogue, and the
// fixup of split tiles that it shares with the NVFP4 GEMM.
#include "gemm_bf16.hpp"

namespace dmpq {

hipError_t launch_f32_fixup_linear(hipStream_t s, const float *ga, const float *gw, int64_t M, int64_t N,
                                   void *y, unsigned tiles_m, unsigned tiles_n, unsigned group_m,
                                   float *partial, const SplitPlan &sp, const uint32_t *spart,
                                   int out_dtype, int epi, const LinearEpi &lin) {
#define DMPQ_LINEAR(OUT_, EPI_) \
    return launch_fixup<OUT_, (EPI_)>(s, ga, gw, M, N, y, tiles_m, tiles_n, group_m, partial, sp, spart, lin)
    if (out_dtype == 0) {
        if (epi == kEpiLinear) DMPQ_LINEAR(0, kEpiLinear);
        if (epi == (kEpiLinear | kEpiLora)) DMPQ_LINEAR(0, kEpiLinear | kEpiLora);
    }
    if (out_dtype != 1) return hipErrorInvalidValue;
    if ((epi & kEpiHeads) != 0)
        return launch_f32_fixup_linear_heads(s, ga, gw, M, N, y, tiles_m, tiles_n, group_m, partial, sp, spart, epi, lin);
    switch (epi) {
        case kEpiLinear: DMPQ_LINEAR(1, kEpiLinear);
        case kEpiLinear | kEpiAmax: DMPQ_LINEAR(1, kEpiLinear | kEpiAmax);
        case kEpiLinear | kEpiLora: DMPQ_LINEAR(1, kEpiLinear | kEpiLora);
        case kEpiLinear | kEpiLora | kEpiAmax: DMPQ_LINEAR(1, kEpiLinear | kEpiLora | kEpiAmax);
    }
#undef DMPQ_LINEAR
    return hipErrorInvalidValue;
}

hipError_t launch_gemm_bf16_linear(hipStream_t s, const uint16_t *x, const uint16_t *w, int64_t M, int64_t N,
                                   int64_t K, int out_dtype, void *y, bool amax, float *partial, uint32_t *spart,
                                   const LinearEpi &lin) {
    if (M == 0 || N == 0) return hipSuccess;
#define DMPQ_LINEAR(OUT_, EPI_) return launch_bf16_paths<OUT_, (EPI_)>(s, x, w, M, N, K, y, partial, spart, lin)
    const int epi = linear_epi(amax, lin, N);
    if (out_dtype == 0) {
        if (epi == kEpiLinear) DMPQ_LINEAR(0, kEpiLinear);
        if (epi == (kEpiLinear | kEpiLora)) DMPQ_LINEAR(0, kEpiLinear | kEpiLora);
    }
    if (out_dtype != 1) return hipErrorInvalidValue;
    if ((epi & kEpiHeads) != 0)
        return launch_gemm_bf16_linear_heads(s, x, w, M, N, K, y, partial, spart, lin, epi);
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
