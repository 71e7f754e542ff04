// 8-bit integers as FP16 values.  Every 8-bit integer is an FP16 number and a
// product of two is an FP32 number, so the tensor cores' FP16 products with
// FP32 accumulators add up 8-bit products exactly until a partial sum passes
// 2^24.  (The integer tensor path of sm_103a reaches 273 products a cycle per
// SM, FP16 mma.sync 1045 and tcgen05 about 4096.)
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "rows.cuh"

namespace sgemm {

// Four 8-bit integers as four FP16 values: with the sign bit flipped a byte b
// is b + 128, which as the low byte of 0x64.. is the FP16 number 1024 + 128 + b.
__device__ __forceinline__ uint2 i8x4_to_f16(uint32_t w) {
    const uint32_t u = w ^ 0x80808080u;
    uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 offset = __half2half2(__ushort_as_half(0x6480));  // 1152
    const __half2 a = __hsub2(*reinterpret_cast<__half2 *>(&lo), offset);
    const __half2 b = __hsub2(*reinterpret_cast<__half2 *>(&hi), offset);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// 16 bytes from byte `shift` (0 .. 15) of the 32 in a and b: by two words, by
// one word, by bytes.
__device__ __forceinline__ uint4 shift_codes(const uint4 &a, const uint4 &b, unsigned shift) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = shift & 4 ? w[i + 1] : w[i];
    const unsigned bits = 8 * (shift & 3);
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// Bytes k .. k + 15 of a row of K 8-bit integers, of any alignment; bytes from K
// on are unspecified, and nothing beyond the 16-byte granule of the row's last
// byte is read.  ALIGNED: the row starts on 16 bytes; k is a multiple of 16.
template <bool ALIGNED>
__device__ __forceinline__ uint4 load_codes(const int8_t *row, int k, int K) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if constexpr (ALIGNED) {
        return k < K ? __ldg(reinterpret_cast<const uint4 *>(row + k)) : zero;
    } else {
        const uintptr_t lo = (reinterpret_cast<uintptr_t>(row) + k) & ~(uintptr_t)15;
        const uint4 a = k < K ? __ldg(reinterpret_cast<const uint4 *>(lo)) : zero;
        const uint4 b = k < K && lo + 16 < reinterpret_cast<uintptr_t>(row) + K
                            ? __ldg(reinterpret_cast<const uint4 *>(lo + 16)) : zero;
        return shift_codes(a, b, (unsigned)(reinterpret_cast<uintptr_t>(row) & 15));
    }
}

struct I8Args {
    int M, N, K;
    const int8_t *A, *B;
    int64_t lda, ldb;
    const float *a_scale, *b_scale, *bias;
    void *C;
    int64_t ldc;
    int ctype;
};

__device__ __forceinline__ void store_c(void *C, int64_t at, int ctype, float v) {
    if (ctype == SGEMM_F32) static_cast<float *>(C)[at] = v;
    else if (ctype == SGEMM_BF16) static_cast<__nv_bfloat16 *>(C)[at] = __float2bfloat16_rn(v);
    else static_cast<__half *>(C)[at] = __float2half_rn(v);
}

// Rows of 8-bit integers written out on padded, 16-byte aligned rows: as FP16
// (Code __half, ld a multiple of 8) or as they are (int8_t, ld a multiple of
// 16).  Elements between K and ld are not read by what follows.
template <bool ALIGNED, class Code>
__global__ void __launch_bounds__(256)
    i8_lay_out_kernel(int rows, int K, const int8_t *__restrict__ q, int64_t ldq, Code *__restrict__ out, int64_t ld) {
    griddep_launch_dependents();
    const int pieces = (K + 15) / 16;
    const int64_t total = (int64_t)rows * pieces;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = i / pieces;
        const int k = (int)(i - row * pieces) * 16;
        const uint4 c = load_codes<ALIGNED>(q + row * ldq, k, K);
        Code *to = out + row * ld + k;
        if constexpr (sizeof(Code) == 1) {
            *reinterpret_cast<uint4 *>(to) = c;
        } else {
            const uint2 a = i8x4_to_f16(c.x), b = i8x4_to_f16(c.y), d = i8x4_to_f16(c.z), e = i8x4_to_f16(c.w);
            *reinterpret_cast<uint4 *>(to) = make_uint4(a.x, a.y, b.x, b.y);
            if (k + 8 < ld) *reinterpret_cast<uint4 *>(to + 8) = make_uint4(d.x, d.y, e.x, e.y);
        }
    }
    // this kernel may run beside the one before, which the next one needs as well
    griddep_wait();
}

}  // namespace sgemm
