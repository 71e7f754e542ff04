// What the host code of the log probabilities lends to the beams.
#pragma once

#include "host.h"
#include "logprobs.cuh"

namespace sgemm_host {

// Launches logprobs_kernel, and the checks of its matrix and mask.
__attribute__((visibility("hidden"))) int logprobs(const sgemm::LogprobArgs &a, int dtype, const Device &dev, cudaStream_t stream);
__attribute__((visibility("hidden"))) bool logprobs_shape_ok(int T, int V, int dtype, const void *z, int ldz, float scale,
                                                             const int32_t *mask, int ldm, int mask_rows);

}  // namespace sgemm_host
