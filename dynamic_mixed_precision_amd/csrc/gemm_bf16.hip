// gemm_bf16.hip -- the BF16 GEMM's plain, GELU / amax and adapter forms.
#include "gemm_bf16.hpp"

namespace dmpq {

hipError_t launch_f32_fixup(hipStream_t s, const float *ga, const float *gw, int64_t M, int64_t N,
                            void *y, unsigned tiles_m, unsigned tiles_n, unsigned group_m,
                            float *partial, const SplitPlan &sp, const uint32_t *spart,
                            int out_dtype, int epi, const LoraEpi *lora) {
    const LoraEpi le = lora ? *lora : LoraEpi{};
#define DMPQ_F32_FIXUP(OUT_, EPI_) \
    return launch_fixup<OUT_, EPI_>(s, ga, gw, M, N, y, tiles_m, tiles_n, group_m, partial, sp, spart, le)
    if (out_dtype == 0 && epi == 0) DMPQ_F32_FIXUP(0, 0);
    if (out_dtype == 0 && epi == kEpiLora) DMPQ_F32_FIXUP(0, kEpiLora);
    if (out_dtype != 1) return hipErrorInvalidValue;
    switch (epi) {
        case 0: DMPQ_F32_FIXUP(1, 0);
        case 1: DMPQ_F32_FIXUP(1, 1);
        case 2: DMPQ_F32_FIXUP(1, 2);
        case 3: DMPQ_F32_FIXUP(1, 3);
        case 4: DMPQ_F32_FIXUP(1, 4);
        case 5: DMPQ_F32_FIXUP(1, 5);
        case 6: DMPQ_F32_FIXUP(1, 6);
        case 7: DMPQ_F32_FIXUP(1, 7);
    }
#undef DMPQ_F32_FIXUP
    return hipErrorInvalidValue;
}

hipError_t launch_gemm_bf16(hipStream_t s, const uint16_t *x, const uint16_t *w, int64_t M,
                            int64_t N, int64_t K, int out_dtype, void *y, int epi, float *partial,
                            uint32_t *spart, const LoraEpi *lora) {
    if (M == 0 || N == 0) return hipSuccess;
    const LoraEpi le = lora ? *lora : LoraEpi{};
    if (lora) epi |= kEpiLora;
#define DMPQ_BF16_PATHS(OUT_, EPI_) return launch_bf16_paths<OUT_, EPI_>(s, x, w, M, N, K, y, partial, spart, le)
    if (out_dtype == 0 && epi == 0) DMPQ_BF16_PATHS(0, 0);
    if (out_dtype == 0 && epi == kEpiLora) DMPQ_BF16_PATHS(0, kEpiLora);
    if (out_dtype != 1) return hipErrorInvalidValue;
    switch (epi) {
        case 0: DMPQ_BF16_PATHS(1, 0);
        case 1: DMPQ_BF16_PATHS(1, 1);
        case 2: DMPQ_BF16_PATHS(1, 2);
        case 3: DMPQ_BF16_PATHS(1, 3);
        case 4: DMPQ_BF16_PATHS(1, 4);
        case 5: DMPQ_BF16_PATHS(1, 5);
        case 6: DMPQ_BF16_PATHS(1, 6);
        case 7: DMPQ_BF16_PATHS(1, 7);
    }
#undef DMPQ_BF16_PATHS
    return hipErrorInvalidValue;
}

}  // namespace dmpq
