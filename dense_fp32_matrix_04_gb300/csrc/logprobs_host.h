// The launch of logprobs_kernel, and checks, that the log probabilities and the beams
// share.
#pragma once

#include <algorithm>
#include <cstdint>

#include "host.h"
#include "logprobs.cuh"
#include "row_host.h"

namespace sgemm_host {

using sgemm::kLogprobRing;
using sgemm::LogprobArgs;
using sgemm::logprobs_kernel;

constexpr int kMostRows = 1 << 30;

template <int DT, int THREADS, bool TOP, bool MASK, bool BEAM>
int launch_logprobs(const LogprobArgs &a, unsigned parts, const Device &dev, cudaStream_t stream) {
    static std::atomic<int> regs[kMaxDevices];
    const auto kernel = logprobs_kernel<DT, THREADS, TOP, MASK, BEAM>;
    constexpr int smem = kLogprobRing<DT, THREADS, MASK>;
    if (!blocks_per_sm(regs, dev, kernel, THREADS, smem)) return SGEMM_ERR_LAUNCH;
    const dim3 grid(parts, (unsigned)std::min(a.T, 1024 / THREADS * dev.sms));
    return launch(kernel, grid, dim3(THREADS), smem, stream, parts, a);
}

template <int DT, bool MASK, bool BEAM>
int logprobs_by_length(const LogprobArgs &a, const Device &dev, cudaStream_t stream) {
    // few rows are shared by clusters of up to 8 blocks, until there are two blocks per SM; many
    // are walked by the blocks the SMs hold
    unsigned parts = 1;
    while (parts < 8 && (int64_t)a.T * parts * 2 <= 2 * dev.sms && a.V / (int)(parts * 2) >= 2048) parts *= 2;
    // two warps a row where a row is short, or nothing but its sums is wanted: what a row costs a
    // warp beside its columns weighs less (64000 x 1000 302 -> 81 us, 4096 x 50001 without
    // alternatives 91 -> 80 us; with five alternatives 104 -> 110 us)
    if constexpr (!BEAM) {  // (a step of beams has alternatives)
        if (!a.top)
            return parts == 1 ? launch_logprobs<DT, 64, false, MASK, false>(a, 1, dev, stream)
                              : launch_logprobs<DT, 256, false, MASK, false>(a, parts, dev, stream);
    }
    if (parts == 1 && a.V < 16384) return launch_logprobs<DT, 64, true, MASK, BEAM>(a, 1, dev, stream);
    // four warps for longer rows with alternatives, where there are two for each block that the SMs
    // hold (4096 x 50001 104 -> 89 us; 2000 x 32000 with 20 alternatives 44 -> 49 us), and while
    // the columns that may be alternatives are few, which grows with top and with what a thread
    // sees of a row (4096 x 100001 with 5 alternatives 173 -> 171 us, with 20 205 -> 256 us)
    if (parts == 1 && a.T >= 2 * 8 * dev.sms && (int64_t)a.top * a.V <= 1 << 20)
        return launch_logprobs<DT, 128, true, MASK, BEAM>(a, 1, dev, stream);
    return launch_logprobs<DT, 256, true, MASK, BEAM>(a, parts, dev, stream);
}

inline bool logprobs_shape_ok(int T, int V, int dtype, const Rows &z, float scale, const int32_t *mask, int ldm,
                       int mask_rows) {
    if (T < 0 || V < 0 || T > kMostRows || V > kMostRows || !dtype_ok(dtype)) return false;
    // (a larger scale's product with log2(e) would not be finite)
    if (!(scale > 0.f && scale <= 0x1p127f) || mask_rows < 0) return false;
    if (T == 0) return true;
    if (V > 0 && !z.ok(V, dtype_size(dtype))) return false;
    if ((mask != nullptr) != (mask_rows > 0)) return false;
    if (!mask) return true;
    return aligned(mask, 4) && (mask_rows == 1 || mask_rows == T) && (mask_rows == 1 || ldm >= (V + 31) / 32);
}

}  // namespace sgemm_host
