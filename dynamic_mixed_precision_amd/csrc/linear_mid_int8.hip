// linear_mid_int8.hip -- the whole linear in small tiles, INT8 operands.
#include "linear_mid.hpp"

namespace dmpq {

hipError_t launch_mid_int8(hipStream_t s, const int8_t *qa, const float *sa, const int8_t *qw, const float *sw,
                            int64_t M, int64_t N, int64_t K, int out_dtype, void *y, const LinearEpi &L, float *amax) {
    return launch_mid<MidI8>(s, {qa, qw, sa, sw}, M, N, K, out_dtype, y, L, amax);
}

}  // namespace dmpq
