// linear_mid_nvfp4.hip -- the whole linear in small tiles, NVFP4 operands.
#include "linear_mid.hpp"

namespace dmpq {

hipError_t launch_mid_nvfp4(hipStream_t s, const uint8_t *ca, const uint8_t *sa, const float *ga, const uint8_t *cw, const uint8_t *sw,
                            const float *gw,
                            int64_t M, int64_t N, int64_t K, int out_dtype, void *y, const LinearEpi &L, float *amax) {
    return launch_mid<MidFP4>(s, {ca, sa, ga, cw, sw, gw}, M, N, K, out_dtype, y, L, amax);
}

}  // namespace dmpq
