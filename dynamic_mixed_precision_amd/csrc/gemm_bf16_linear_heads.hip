// gemm_bf16_linear_heads.hip -- the BF16 GEMM whose epilogue is the heads of q and k
// (a file of its own: the kernels of one GEMM take minutes to compile).
#include "gemm_bf16.hpp"

namespace dmpq {

hipError_t launch_f32_fixup_linear_heads(hipStream_t s, const float *ga, const float *gw, int64_t M, int64_t N, void
                                         *y,
                                         unsigned tiles_m, unsigned tiles_n, unsigned group_m, float *partial,
                                         const SplitPlan &sp, const uint32_t *spart, int epi, const LinearEpi &lin) {
#define DMPQ_LINEAR(OUT_, EPI_) \
    return launch_fixup<OUT_, (EPI_)>(s, ga, gw, M, N, y, tiles_m, tiles_n, group_m, partial, sp, spart, lin)
    switch (epi) {
        case kEpiLinear | kEpiHeads: DMPQ_LINEAR(1, kEpiLinear | kEpiHeads);
        case kEpiLinear | kEpiHeads | kEpiBand: DMPQ_LINEAR(1, kEpiLinear | kEpiHeads | kEpiBand);
        case kEpiLinear | kEpiHeads | kEpiLora: DMPQ_LINEAR(1, kEpiLinear | kEpiHeads | kEpiLora);
    }
#undef DMPQ_LINEAR
    return hipErrorInvalidValue;
}

hipError_t launch_gemm_bf16_linear_heads(hipStream_t s, const uint16_t *x, const uint16_t *w, int64_t M, int64_t N,
                                         int64_t K, void *y, float *partial, uint32_t *spart, const LinearEpi &lin,
                                         int epi) {
#define DMPQ_LINEAR(OUT_, EPI_) return launch_bf16_paths<OUT_, (EPI_)>(s, x, w, M, N, K, y, partial, spart, lin)
    switch (epi) {
        case kEpiLinear | kEpiHeads: DMPQ_LINEAR(1, kEpiLinear | kEpiHeads);
        case kEpiLinear | kEpiHeads | kEpiBand: DMPQ_LINEAR(1, kEpiLinear | kEpiHeads | kEpiBand);
        case kEpiLinear | kEpiHeads | kEpiLora: DMPQ_LINEAR(1, kEpiLinear | kEpiHeads | kEpiLora);
    }
#undef DMPQ_LINEAR
    return hipErrorInvalidValue;
}

}  // namespace dmpq
