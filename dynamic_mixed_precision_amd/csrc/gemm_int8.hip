// gemm_int8.hip -- the INT8 GEMM's plain, GELU / amax and adapter forms, and
// the one that converts its NVFP4 weight.
#include "gemm_int8.hpp"

namespace dmpq {

hipError_t launch_gemm_int8_w4(hipStream_t s, const int8_t *qa, const float *sa, const uint8_t *cw,
                               const uint8_t *sw, const float *gw, const float *s_row,
                               const float *inv_row, int64_t M, int64_t N, int64_t K, int out_dtype,
                               void *y, int epi, float *partial) {
    if (M == 0 || N == 0) return hipSuccess;
    if (K % i8gemm::BK != 0) return hipErrorInvalidValue;
    if (epi == 0) {
        switch (out_dtype) {
            case 0: return launch_i8w4<0, 0>(s, qa, sa, cw, sw, gw, s_row, inv_row, M, N, K, y, partial);
            case 1: return launch_i8w4<1, 0>(s, qa, sa, cw, sw, gw, s_row, inv_row, M, N, K, y, partial);
            case 2: return launch_i8w4<2, 0>(s, qa, sa, cw, sw, gw, s_row, inv_row, M, N, K, y, partial);
        }
        return hipErrorInvalidValue;
    }
    if (out_dtype != 1) return hipErrorInvalidValue;
    switch (epi) {
        case 1: return launch_i8w4<1, 1>(s, qa, sa, cw, sw, gw, s_row, inv_row, M, N, K, y, partial);
        case 2: return launch_i8w4<1, 2>(s, qa, sa, cw, sw, gw, s_row, inv_row, M, N, K, y, partial);
        case 3: return launch_i8w4<1, 3>(s, qa, sa, cw, sw, gw, s_row, inv_row, M, N, K, y, partial);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_gemm_int8(hipStream_t s, const int8_t *qa, const float *sa, const int8_t *qw,
                            const float *sw, int64_t M, int64_t N, int64_t K, int out_dtype,
                            void *y, int epi, float *partial, uint32_t *spart, const LoraEpi *lora) {
    if (M == 0 || N == 0) return hipSuccess;
    const LoraEpi le = lora ? *lora : LoraEpi{};
    if (lora) epi |= kEpiLora;
#define DMPQ_I8_PATHS(OUT_, EPI_) \
    return launch_i8_paths<OUT_, EPI_>(s, qa, sa, qw, sw, M, N, K, y, partial, spart, le)
    if (epi == 0) {
        switch (out_dtype) {
            case 0: DMPQ_I8_PATHS(0, 0);
            case 1: DMPQ_I8_PATHS(1, 0);
            case 2: DMPQ_I8_PATHS(2, 0);
        }
        return hipErrorInvalidValue;
    }
    if (out_dtype == 0 && epi == kEpiLora) DMPQ_I8_PATHS(0, kEpiLora);
    if (out_dtype != 1) return hipErrorInvalidValue;
    switch (epi) {
        case 1: DMPQ_I8_PATHS(1, 1);
        case 2: DMPQ_I8_PATHS(1, 2);
        case 3: DMPQ_I8_PATHS(1, 3);
        case 4: DMPQ_I8_PATHS(1, 4);
        case 5: DMPQ_I8_PATHS(1, 5);
        case 6: DMPQ_I8_PATHS(1, 6);
        case 7: DMPQ_I8_PATHS(1, 7);
    }
#undef DMPQ_I8_PATHS
    return hipErrorInvalidValue;
}

}  // namespace dmpq
