// gemm_int8_linear_heads.hip -- the INT8 GEMM whose epilogue is the heads of q and k
// (a file of its own: the kernels of one GEMM take minutes to compile).
#include "gemm_int8.hpp"

namespace dmpq {

hipError_t launch_gemm_int8_linear_heads(hipStream_t s, const int8_t *qa, const float *sa, const int8_t *qw, const
                                         float *sw, int64_t M, int64_t N, int64_t K, void *y, float *partial,
                                         uint32_t *spart, const LinearEpi &lin, int epi) {
#define DMPQ_LINEAR(OUT_, EPI_) return launch_i8_paths<OUT_, (EPI_)>(s, qa, sa, qw, sw, M, N, K, y, partial, spart, lin)
    switch (epi) {
        case kEpiLinear | kEpiHeads: DMPQ_LINEAR(1, kEpiLinear | kEpiHeads);
        case kEpiLinear | kEpiHeads | kEpiBand: DMPQ_LINEAR(1, kEpiLinear | kEpiHeads | kEpiBand);
        case kEpiLinear | kEpiHeads | kEpiLora: DMPQ_LINEAR(1, kEpiLinear | kEpiHeads | kEpiLora);
    }
#undef DMPQ_LINEAR
    return hipErrorInvalidValue;
}

}  // namespace dmpq
