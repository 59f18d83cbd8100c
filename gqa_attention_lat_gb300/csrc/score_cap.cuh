// score_cap.cuh — a capped score in the log2 domain, close in relative terms too.
#pragma once

#include "device_common.cuh"

namespace lat {

// cap * tanh(y), y the score over the cap.  1 - 2 / (1 + e^{2y}) loses bits of a small y (an
// error of a few 1e-7 of the cap, where most scores lie far below it), so below 0.3 it is tanh's
// Taylor series to y^9, whose next term is 5e-8 of y there.
__device__ __forceinline__ float capped_score_close(float y, float cap_log2) {
    const float far = cap_log2 - __fdividef(2.f * cap_log2, 1.f + fast_exp2(y * kTwoLog2e));
    const float z = y * y;
    const float t = fmaf(z, fmaf(z, fmaf(z, fmaf(z, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f), 1.f);
    return fabsf(y) < 0.3f ? cap_log2 * y * t : far;
}

}  // namespace lat
