// What the row-wise kernels share: element types, vector loads and stores that
// convert to and from FP32, and reductions over a warp or a block.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/sgemm_layers.h"
#include "ptx.cuh"

namespace sgemm {

// An element type and the number of its elements in 16 bytes.
template <int DT>
struct Elem;
template <>
struct Elem<SGEMM_F32> {
    using type = float;
    static constexpr int VEC = 4;
    __device__ static float to_float(float v) { return v; }
    __device__ static float from_float(float v) { return v; }
};
template <>
struct Elem<SGEMM_BF16> {
    using type = __nv_bfloat16;
    static constexpr int VEC = 8;
    __device__ static float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
    __device__ static __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<SGEMM_F16> {
    using type = __half;
    static constexpr int VEC = 8;
    __device__ static float to_float(__half v) { return __half2float(v); }
    __device__ static __half from_float(float v) { return __float2half_rn(v); }
};

// 16 bytes of elements as FP32 values.
template <int DT>
__device__ __forceinline__ void unpack16(const uint4 &raw, float *out) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == SGEMM_F32) {
            out[i] = __uint_as_float(w[i]);
        } else if constexpr (DT == SGEMM_BF16) {
            out[2 * i] = __uint_as_float(w[i] << 16);
            out[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            out[2 * i] = f.x;
            out[2 * i + 1] = f.y;
        }
    }
}

// The inverse, each value rounded once to nearest even.
template <int DT>
__device__ __forceinline__ uint4 pack16(const float *v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == SGEMM_F32) {
            w[i] = __float_as_uint(v[i]);
        } else if constexpr (DT == SGEMM_BF16) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&p);
        } else {
            const __half2 p = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&p);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A thread's part of a row: NV pieces of VW elements, piece v at column
// (v * threads + thread) * VW.  VW is 16 bytes' worth (rows that are 16-byte
// aligned and whole pieces long) or 1 (any other row).
template <int DT, int VW>
struct Piece {
    using type = typename Elem<DT>::type;
    using raw = uint4;
    __device__ static raw load(const type *p) { return *reinterpret_cast<const uint4 *>(p); }
    __device__ static raw zero() { return make_uint4(0, 0, 0, 0); }
    __device__ static void unpack(const raw &r, float *out) { unpack16<DT>(r, out); }
    __device__ static void store(type *p, const float *v) { *reinterpret_cast<uint4 *>(p) = pack16<DT>(v); }
};
template <int DT>
struct Piece<DT, 1> {
    using type = typename Elem<DT>::type;
    using raw = type;
    __device__ static raw load(const type *p) { return *p; }
    __device__ static raw zero() { return Elem<DT>::from_float(0.f); }
    __device__ static void unpack(const raw &r, float *out) { out[0] = Elem<DT>::to_float(r); }
    __device__ static void store(type *p, const float *v) { *p = Elem<DT>::from_float(v[0]); }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

// Sums and maxima over the threads that share a row: a warp (warps == 1), the
// block's warps through shared memory, or those of a cluster of `ranks` blocks
// of up to 16 warps through distributed shared memory; in an order that the
// numbers of warps and ranks fix, so every thread has the same bits.  Up to
// three sums are taken together.  Calls alternate between two sets of slots, so
// one barrier a call is enough.  (Blocks of a cluster meet once more before
// they leave.)
struct RowReducer {
    static constexpr int SLOTS = 2 * 3 * 32;
    float *slots;  // SLOTS floats of shared memory
    int warps, ranks = 1, turn = 0;
    template <int N, class Join>
    __device__ void all(uint32_t (&v)[N], uint32_t none, Join join) {
        float *s = slots + 96 * turn;
        turn ^= 1;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) s[32 * i + warp] = __uint_as_float(v[i]);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = none;
        if (ranks == 1) {
            __syncthreads();
            if (lane < warps)
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] = __float_as_uint(s[32 * i + lane]);
        } else {
            __syncwarp();
            cluster_sync();
            const int w = lane & 15;
            if (w < warps)
                for (int r = lane >> 4; r < ranks; r += 2)
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        v[i] = join(v[i], dsmem_ld_u32(dsmem_map(smem_addr(s + 32 * i + w), (uint32_t)r)));
        }
    }
    // Three sums within a block: a quarter of the lanes (the last two quarters the same) carries
    // one each, which halves the shuffles.
    __device__ void sum3(float (&v)[3]) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane >> 3;
        const bool hi = lane & 16, odd = lane & 8;
        float a = hi ? v[2] : v[0], b = v[1];
        a += __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 16);
        b += __shfl_xor_sync(0xffffffffu, v[1], 16);
        // lanes 0-15 hold the first two sums, 16-31 the third
        const float got = __shfl_xor_sync(0xffffffffu, hi || odd ? a : b, 8);
        a = (hi || !odd ? a : b) + got;
#pragma unroll
        for (int o = 4; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        if (warps > 1) {
            float *s = slots + 96 * turn;
            turn ^= 1;
            const int sum = min(q, 2), w = lane & 7;
            if (w == 0 && q < 3) s[32 * sum + warp] = a;
            __syncthreads();
            a = w < warps ? s[32 * sum + w] : 0.f;
            if (warps > 8 && w + 8 < warps) a += s[32 * sum + w + 8];
#pragma unroll
            for (int o = 4; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) v[i] = __shfl_sync(0xffffffffu, a, 8 * i);
    }
    template <int N>
    __device__ void sum(float (&v)[N]) {
        if constexpr (N == 3)
            if (ranks == 1) return sum3(v);  // of up to 16 warps
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
        if (warps == 1 && ranks == 1) return;
        uint32_t bits[N];
#pragma unroll
        for (int i = 0; i < N; ++i) bits[i] = __float_as_uint(v[i]);
        all(bits, 0u, [](uint32_t a, uint32_t b) {
            return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
        });
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = warp_sum(__uint_as_float(bits[i]));
    }
    __device__ float sum(float v) {
        float one[1] = {v};
        sum(one);
        return one[0];
    }
    __device__ uint32_t max(uint32_t v) {
        v = warp_max(v);
        if (warps == 1 && ranks == 1) return v;
        uint32_t one[1] = {v};
        all(one, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
        return warp_max(one[0]);
    }
};

// A row's scale and multiplier for 8 bits from the largest magnitude in it
// (as FP32 bits, so that a NaN counts as the largest): s = max / 127 and
// 127 / max.  Below 2^-100 the quotient could overflow: such rows are first
// multiplied by 2^64, exactly, in both factors.
struct I8Scale {
    float pre, inv, scale;
    __device__ explicit I8Scale(uint32_t max_bits) {
        const float m = __uint_as_float(max_bits);
        pre = 1.f;
        inv = 0.f;
        scale = m / 127.f;
        if (max_bits == 0) scale = 0.f;
        if (max_bits > 0 && max_bits < 0x7f800000u) {
            if (m < 0x1p-100f) pre = 0x1p64f;
            inv = 127.f / (m * pre);
        }
    }
    __device__ int8_t operator()(float x) const {
        // |x pre inv| <= 127 (1 + 2^-23); infinities and NaN have inv = 0 and become 0
        const int q = __float2int_rn(x * pre * inv);
        return (int8_t)(q > 127 ? 127 : q < -127 ? -127 : q);
    }
};

}  // namespace sgemm
