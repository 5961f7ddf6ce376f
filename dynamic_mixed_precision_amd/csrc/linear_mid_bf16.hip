// linear_mid_bf16.hip -- the whole linear in small tiles, BF16 operands.
#include "linear_mid.hpp"

namespace dmpq {

hipError_t launch_mid_bf16(hipStream_t s, const uint16_t *x, const uint16_t *w,
                            int64_t M, int64_t N, int64_t K, int out_dtype, void *y, const LinearEpi &L, float *amax) {
    return launch_mid<MidBF16>(s, {x, w}, M, N, K, out_dtype, y, L, amax);
}

}  // namespace dmpq
