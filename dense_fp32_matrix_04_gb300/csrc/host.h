// Host-side facts and checks that the library's translation units share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>
#include <utility>

#include "../../include/sgemm_layers.h"

namespace sgemm_host {

constexpr int kMaxDevices = 64;

// The current device, its SM count and the address of its error word
// (SGEMM_OK or SGEMM_ERR_DEVICE); queried once per device (sgemm_api.cu).
struct Device {
    int dev = 0;
    int sms = 0;
    int *err_word = nullptr;
};
__attribute__((visibility("hidden"))) int device(Device &out);

// Tensor map of a row-major FP16 matrix (16-byte aligned base and rows), read in
// boxes of box_rows rows by 64 columns into 128-byte swizzled rows; zeros
// outside the matrix.
__attribute__((visibility("hidden"))) bool encode_f16(CUtensorMap *map, const void *ptr, int64_t rows, int64_t cols,
                                                      int64_t ld, int box_rows);

// The same of 8-bit integers, in boxes of 128 or 64 columns into swizzled rows of as many bytes.
__attribute__((visibility("hidden"))) bool encode_i8(CUtensorMap *map, const void *ptr, int64_t rows, int64_t cols,
                                                     int64_t ld, int box_rows, int box_cols);

// Nanoseconds a kernel may wait for its own copies before it gives up.
__attribute__((visibility("hidden"))) unsigned long long wait_limit_ns();

// The test-only switches (sgemm_testing.h); 0 unless a test turned some on.
__attribute__((visibility("hidden"))) int test_flags();

inline bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// A buffer's byte range; empty when it has no elements.
struct Range {
    uintptr_t lo = 0, hi = 0;
    Range() = default;
    Range(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t size)
        : lo(reinterpret_cast<uintptr_t>(p)),
          hi(p && rows > 0 && cols > 0 ? lo + (uintptr_t)(((rows - 1) * ld + cols) * size) : lo) {}
    bool overlaps(const Range &o) const { return lo < o.hi && o.lo < hi; }
};

// Launches a kernel, in clusters of `cluster` blocks along x where that is
// more than one, and with EARLY as soon as every block of the kernel before
// allows it (griddepcontrol); SGEMM_OK, or SGEMM_ERR_LAUNCH with the error
// cleared.
template <bool EARLY = false, class... Params, class... Args>
int launch(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, unsigned cluster,
           Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    if (EARLY) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    if (cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...) == cudaSuccess) return SGEMM_OK;
    (void)cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
}

// Blocks of a kernel that fit an SM, from the registers it was compiled to use;
// on a device's first use of it (`regs` is the caller's cache for the kernel)
// its shared-memory limit is raised.  0 if the device refuses.
template <class Kernel>
inline int blocks_per_sm(std::atomic<int> (&regs)[kMaxDevices], const Device &dev, Kernel kernel, int threads, int smem) {
    int r = regs[dev.dev].load(std::memory_order_acquire);
    if (r == 0) {
        cudaFuncAttributes at;
        if (cudaFuncGetAttributes(&at, kernel) != cudaSuccess ||
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 227 * 1024 - (int)at.sharedSizeBytes) != cudaSuccess) {
            (void)cudaGetLastError();
            return 0;
        }
        r = at.numRegs;
        regs[dev.dev].store(r, std::memory_order_release);
    }
    const int warps = (threads + 31) / 32;
    const int by_regs = 65536 / ((r + 7) / 8 * 8 * 32 * warps), by_smem = 227 * 1024 / (smem + 2048);
    return std::max(1, std::min({by_regs, by_smem, 64 / warps, 32}));
}

// Calls f(std::integral_constant<int, dtype>) for one of the three element types.
template <class F>
int by_dtype(int dtype, F &&f) {
    switch (dtype) {
        case SGEMM_F32: return f(std::integral_constant<int, SGEMM_F32>{});
        case SGEMM_BF16: return f(std::integral_constant<int, SGEMM_BF16>{});
        case SGEMM_F16: return f(std::integral_constant<int, SGEMM_F16>{});
        default: return SGEMM_ERR_INVALID_ARG;
    }
}

inline int dtype_size(int dtype) { return dtype == SGEMM_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == SGEMM_F32 || dtype == SGEMM_BF16 || dtype == SGEMM_F16; }

}  // namespace sgemm_host
