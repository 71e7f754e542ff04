// C = diag(sa) A B^T diag(sb) + bias with 8-bit A (M x K) and B (N x K).
#pragma once

#include <cstdint>

#include "rows.cuh"

namespace sgemm {

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

// 64 x 64 outputs a block from 64-byte deep tiles in shared memory, 4 x 4 a
// thread with four-way byte products into 32-bit integers (exact).
__global__ void __launch_bounds__(256) i8_tile_kernel(const I8Args p, int vec_a, int vec_b) {
    __shared__ int sa[64][17], sb[64][17];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
    int acc[4][4] = {};
    const int row = tid >> 2, seg = (tid & 3) * 16;
    auto fetch = [&](const int8_t *base, int64_t ld, int64_t r, int rows, int k, int vec) {
        int4 v = make_int4(0, 0, 0, 0);
        if (r >= rows || k >= p.K) return v;
        const int8_t *src = base + r * ld + k;
        if (vec && k + 16 <= p.K) return *reinterpret_cast<const int4 *>(src);
        uint32_t w[4] = {};
        for (int i = 0; i < 16; ++i)
            if (k + i < p.K) w[i >> 2] |= (uint32_t)(uint8_t)src[i] << (8 * (i & 3));
        return make_int4((int)w[0], (int)w[1], (int)w[2], (int)w[3]);
    };
    for (int k0 = 0; k0 < p.K; k0 += 64) {
        const int4 a = fetch(p.A, p.lda, m0 + row, p.M, k0 + seg, vec_a);
        const int4 b = fetch(p.B, p.ldb, n0 + row, p.N, k0 + seg, vec_b);
        __syncthreads();
        int *da = &sa[row][seg / 4], *db = &sb[row][seg / 4];
        da[0] = a.x, da[1] = a.y, da[2] = a.z, da[3] = a.w;
        db[0] = b.x, db[1] = b.y, db[2] = b.z, db[3] = b.w;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            int x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = sa[ty * 4 + i][k];
                y[i] = sb[tx + 16 * i][k];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(x[i], y[j], acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty * 4 + i, n = n0 + tx + 16 * j;
            if (m < p.M && n < p.N) {
                float v = (float)acc[i][j] * p.a_scale[m] * p.b_scale[n];
                if (p.bias) v += p.bias[n];
                store_c(p.C, m * p.ldc + n, p.ctype, v);
            }
        }
}

}  // namespace sgemm
