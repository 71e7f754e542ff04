// Rows quantised to 8-bit integers with one scale each: s = max|x| / 127,
// q = rint(x (127 / max|x|)).  The row is read once into registers (or, when
// it is too wide for them, a second time from L2) and written as bytes: the
// kernel is bound by memory.  Blocks walk several rows and read the next one
// before they reduce this one's maximum.  8192 x 8192 BF16 takes 40 us (5.1 TB/s).
// Rows of more than 16384 are read twice and by single elements: 2048 x 28672 BF16
// 148 us, 1.2 TB/s.
#pragma once

#include <cstdint>

#include "rows.cuh"

namespace sgemm {

// n 8-bit values to p, whole words at a time where `vec` says that they are aligned.
template <int N>
__device__ __forceinline__ void store_bytes(int8_t *p, const int8_t (&b)[N], bool vec) {
    if constexpr (N % 4 == 0) {
        if (vec) {
            uint32_t w[N / 4];
#pragma unroll
            for (int i = 0; i < N; i += 4)
                w[i / 4] = (uint32_t)(uint8_t)b[i] | (uint32_t)(uint8_t)b[i + 1] << 8 |
                           (uint32_t)(uint8_t)b[i + 2] << 16 | (uint32_t)(uint8_t)b[i + 3] << 24;
            if constexpr (N == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
            else *reinterpret_cast<uint32_t *>(p) = w[0];
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = b[i];
}

// The codes of a row as 8-bit integers or, for the tensor cores, as FP16 values.
__device__ __forceinline__ void put_code(int8_t *p, int8_t c) { *p = c; }
__device__ __forceinline__ void put_code(__half *p, int8_t c) { *p = __int2half_rn(c); }

template <int DT, int VW, int NV, class Code>
__global__ void __launch_bounds__(1024)
    quantize_i8_kernel(int M, int K, const typename Elem<DT>::type *__restrict__ x, int64_t ldx,
                       Code *__restrict__ q, int64_t ldq, float *__restrict__ scale, int q_vec) {
    using P = Piece<DT, VW>;
    __shared__ float slots[RowReducer::SLOTS];
    griddep_launch_dependents();
    RowReducer red{slots, (int)(blockDim.x >> 5)};
    const int threads = blockDim.x;
    const int step = gridDim.x * blockDim.y;
    // the next row is on its way while this one is reduced and written (rows of single elements,
    // and FP32 ones, have no registers for that)
    constexpr bool AHEAD = VW == 8;
    typename P::raw next[NV];
    auto load = [&](int64_t m) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * threads + (int)threadIdx.x) * VW;
            next[i] = m < M && c < K ? P::load(x + m * ldx + c) : P::zero();
        }
    };
    if (AHEAD) load((int64_t)blockIdx.x * blockDim.y + threadIdx.y);
    for (int64_t m = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; m < M; m += step) {
        float v[NV * VW];
        uint32_t top = 0;
        if (!AHEAD) load(m);
#pragma unroll
        for (int i = 0; i < NV; ++i) P::unpack(next[i], v + i * VW);
        if (AHEAD) load(m + step);
#pragma unroll
        for (int i = 0; i < NV * VW; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
        const I8Scale s(red.max(top));
        if (threadIdx.x == 0) scale[m] = s.scale;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * threads + (int)threadIdx.x) * VW;
            if (c >= K) continue;
            int8_t b[VW];
#pragma unroll
            for (int e = 0; e < VW; ++e) b[e] = s(v[i * VW + e]);
            if constexpr (sizeof(Code) == 1) {
                store_bytes(q + m * ldq + c, b, q_vec);
            } else if constexpr (VW > 1) {
                float f[VW];
#pragma unroll
                for (int e = 0; e < VW; ++e) f[e] = (float)b[e];
                if constexpr (VW == 8) {
                    *reinterpret_cast<uint4 *>(q + m * ldq + c) = pack16<SGEMM_F16>(f);
                } else {
                    const __half2 lo = __floats2half2_rn(f[0], f[1]), hi = __floats2half2_rn(f[2], f[3]);
                    *reinterpret_cast<uint2 *>(q + m * ldq + c) =
                        make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
                }
            } else {
                put_code(q + m * ldq + c, b[0]);
            }
        }
    }
}

template <int DT, class Code>
__global__ void __launch_bounds__(1024)
    quantize_i8_wide_kernel(int M, int K, const typename Elem<DT>::type *__restrict__ x, int64_t ldx,
                            Code *__restrict__ q, int64_t ldq, float *__restrict__ scale) {
    __shared__ float slots[RowReducer::SLOTS];
    griddep_launch_dependents();
    RowReducer red{slots, (int)(blockDim.x >> 5)};
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
        uint32_t top = 0;
        for (int c = threadIdx.x; c < K; c += blockDim.x)
            top = max(top, __float_as_uint(Elem<DT>::to_float(x[m * ldx + c])) & 0x7fffffffu);
        const I8Scale s(red.max(top));
        if (threadIdx.x == 0) scale[m] = s.scale;
        for (int c = threadIdx.x; c < K; c += blockDim.x)
            put_code(q + m * ldq + c, s(Elem<DT>::to_float(x[m * ldx + c])));
    }
}

}  // namespace sgemm
