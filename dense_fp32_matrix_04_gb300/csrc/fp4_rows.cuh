// The product of 4-bit operands for up to four tokens: the time is that of reading
// B, its codes and scales, once.
//
// A warp takes a row of B at a time, 512 contiguous bytes of codes a load.  Codes
// become FP16 numbers, two an instruction, and are multiplied with the tokens' codes,
// which are FP16 in shared memory, in packed FMAs: eight products of at most 36, in
// quarters, in each half, are exact (288 is 1152 quarters, below the 2048 that FP16
// counts to).  The blocks' sums are then scaled and added in FP32.
//
// The scales of B lie in tiles of 128 rows by 4 blocks, where 32 bytes hold a word
// each of the rows 2 i, 2 i + 1 and those 32, 64 and 96 further on: the eight warps of a
// block take such rows, so that what one reads of them serves all.  Tokens that come
// unquantised are quantised by every block itself while its first row of B is on its way.
#pragma once

#include <cuda_fp8.h>

#include <cstdint>

#include "fp4_mma.cuh"
#include "fp4_quantize.cuh"
#include "rows.cuh"

namespace sgemm {

constexpr int kFp4RowsTokens = 4;
constexpr int kFp4RowsThreads = 256;
constexpr int kFp4RowsPieces = 4;    // loads of 16 bytes a lane has in flight
constexpr int kFp4RowsChunk = 1024;  // columns of a warp's load
constexpr int kFp4RowsSmem = 200 * 1024;

// Columns of a token in shared memory: whole loads.
__host__ __device__ constexpr int64_t fp4_rows_columns(int K) { return ((int64_t)K + kFp4RowsChunk - 1) / kFp4RowsChunk * kFp4RowsChunk; }
// Bytes of MT tokens: FP16 codes, an FP32 scale for every 16 columns (blocks of 32: twice the same).
__host__ __device__ constexpr int64_t fp4_rows_smem(int MT, int K) { return MT * fp4_rows_columns(K) / 16 * 36; }

// Place of columns c .. c + 7 (c a multiple of 8) among a token's codes: within a chunk, the four
// pieces of a lane's 32 columns are 32 pieces apart, so that lanes read beside each other.
__device__ __forceinline__ int fp4_rows_place(int c) {
    return (c & ~(kFp4RowsChunk - 1)) + ((c >> 3 & 3) * 32 + (c >> 5 & 31)) * 8;
}

// The eight codes of a word as FP16 numbers.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, __half2 *h) {
    uint32_t r[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = *reinterpret_cast<const __half2 *>(&r[i]);
}

// The value of an e8m0 scale.
__device__ __forceinline__ float e8m0_value(uint32_t s) {
    return __uint_as_float(s == 0 ? 0x400000u : s == 255 ? 0x7fc00000u : s << 23);
}
// Two block scales of 16 columns each from the 16 bits of two e4m3 scales, or the 8 bits of one e8m0.
template <int BLOCK>
__device__ __forceinline__ float2 fp4_scale_values(uint32_t s) {
    if constexpr (BLOCK == 16) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)s, __NV_E4M3);
        return __half22float2(__half2(h));
    } else {
        const float v = e8m0_value(s & 255u);
        return make_float2(v, v);
    }
}
// The bits of those scales for row r and columns 32 c .. 32 c + 31.
template <int BLOCK>
__device__ __forceinline__ uint32_t fp4_load_scales(const uint8_t *tiles, int64_t r, int c, int n_tiles) {
    if constexpr (BLOCK == 16)
        return __ldg(reinterpret_cast<const uint16_t *>(tiles + fp4_scale_word(r, c >> 1, n_tiles) + (c & 1) * 2));
    else
        return __ldg(tiles + fp4_scale_word(r, c >> 2, n_tiles) + (c & 3));
}

struct Fp4RowsArgs {
    Fp4Args p;
    const uint8_t *A, *B;
    int64_t lda, ldb;
    const void *X;  // tokens that are not quantised yet
    int64_t ldx;
};

// XT: the tokens are codes (-1) or values of that element type.
template <int MT, int XT, int BLOCK>
__global__ void __launch_bounds__(kFp4RowsThreads, MT == 1 ? 4 : MT == 2 ? 3 : 2) fp4_rows_kernel(const Fp4RowsArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float slots[kFp4RowsThreads / 32], row_scales[MT];
    constexpr int WARPS = kFp4RowsThreads / 32;
    static_assert(WARPS == 8);
    const Fp4Args &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, K = p.K;
    const int columns = (int)fp4_rows_columns(K), n_tiles = fp4_tiles(K, BLOCK), bytes = (K + 1) / 2;
    __half *codes = reinterpret_cast<__half *>(smem);                         // MT x columns
    float *scales = reinterpret_cast<float *>(codes + MT * columns);          // MT x columns / 16
    const int groups = (p.N + 127) / 128 * 16;
    int group = blockIdx.x;
    auto row_of = [&](int g) { return g / 16 * 128 + g % 16 * 2 + (warp & 1) + (warp >> 1) * 32; };

    uint4 w[kFp4RowsPieces];
    uint32_t ws[kFp4RowsPieces];
    auto load = [&](int row, int c0) {
#pragma unroll
        for (int j = 0; j < kFp4RowsPieces; ++j) {
            const int c = c0 + kFp4RowsChunk * j + 32 * lane;
            const bool in = row < p.N && c < K;
            // (rows are whole 16-byte pieces; what lies behind K meets tokens of 0)
            w[j] = in ? __ldg(reinterpret_cast<const uint4 *>(a.B + row * a.ldb + c / 2)) : make_uint4(0, 0, 0, 0);
            ws[j] = in ? fp4_load_scales<BLOCK>(p.b_tiles, row, c / 32, n_tiles) : 0u;
        }
    };
    int row = row_of(group);
    load(row, 0);

    auto put = [&](int m, int c, const __half2 (&h)[4]) {
        *reinterpret_cast<uint4 *>(codes + m * columns + fp4_rows_place(c)) = *reinterpret_cast<const uint4 *>(h);
    };
    if constexpr (XT < 0) {
        for (int m = 0; m < MT; ++m)
            for (int c = 32 * tid; c < columns; c += 32 * kFp4RowsThreads) {
                const bool in = m < p.M && c < K;
                const uint4 q = in ? __ldg(reinterpret_cast<const uint4 *>(a.A + m * a.lda + c / 2)) : make_uint4(0, 0, 0, 0);
                uint32_t word[4] = {q.x, q.y, q.z, q.w};
                const float2 s = fp4_scale_values<BLOCK>(in ? fp4_load_scales<BLOCK>(p.a_tiles, m, c / 32, n_tiles) : 0u);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // bytes behind the row's end may hold anything
                    const int left = bytes - c / 2 - 4 * i;
                    word[i] = left >= 4 ? word[i] : left > 0 ? word[i] & ((1u << 8 * left) - 1) : 0u;
                    __half2 h[4];
                    e2m1x8_to_f16(word[i], h);
                    put(m, c + 8 * i, h);
                }
                *reinterpret_cast<float2 *>(scales + (m * columns + c) / 16) = s;
            }
        if (tid < MT) row_scales[tid] = p.a_scale && tid < p.M ? p.a_scale[tid] : 1.f;
    } else {
        // the block's warps are shared out to the tokens, which are quantised side by side; a thread takes
        // 16 columns at a time
        using E = Elem<XT < 0 ? 0 : XT>;
        constexpr int SHARE = WARPS / MT, DT = XT < 0 ? 0 : XT;
        const int m = warp / SHARE, first = (warp % SHARE) * 32 + lane, step = SHARE * 32;
        const typename E::type *x = static_cast<const typename E::type *>(a.X) + min(m, p.M - 1) * a.ldx;
        const bool vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0;
        auto values = [&](int c, float (&v)[16]) {
            if (vec && c + 16 <= K) {
                Fp4Piece<DT, E::VEC> piece;
                piece.load(x, c, K);
                return piece.unpack(v);
            }
            Fp4Piece<DT, 1> piece;
            piece.load(x, c, K);
            return piece.unpack(v);
        };
        float v[16];
        uint32_t top = 0;
        if constexpr (BLOCK == 16) {
            for (int i = first; 16 * i < K; i += step) top = max(top, values(16 * i, v));
            top = warp_max(top);
            if (lane == 0) slots[warp] = __uint_as_float(top);
            __syncthreads();
            for (int i = 0; i < SHARE; ++i) top = max(top, __float_as_uint(slots[m * SHARE + i]));
        }
        const Fp4Row r(top);
        for (int i = first; 16 * i < columns; i += step) {
            const int c = 16 * i;
            const uint32_t most = values(c, v);
            uint2 q;
            const uint32_t s = fp4_encode<BLOCK>(v, most, r, q);
            __half2 h[4];
            e2m1x8_to_f16(q.x, h);
            put(m, c, h);
            e2m1x8_to_f16(q.y, h);
            put(m, c + 8, h);
            float scale;
            if constexpr (BLOCK == 16) scale = fp4_scale_values<16>(s).x;
            else scale = e8m0_value(s);
            scales[m * (columns / 16) + i] = scale;
        }
        if (warp % SHARE == 0 && lane == 0) row_scales[m] = BLOCK == 16 ? r.scale : 1.f;
    }
    __syncthreads();

    for (; group < groups; group += gridDim.x) {
        float acc[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m] = 0.f;
        for (int c0 = 0; c0 < columns; c0 += kFp4RowsChunk * kFp4RowsPieces) {
            if (c0 > 0) load(row, c0);
#pragma unroll
            for (int j = 0; j < kFp4RowsPieces; ++j) {
                const int c = c0 + kFp4RowsChunk * j;
                if (c >= columns) break;
                __half2 b[16];
                const uint32_t word[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) e2m1x8_to_f16(word[i], b + 4 * i);
                const float2 sb = fp4_scale_values<BLOCK>(ws[j]);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const __half *x = codes + m * columns + c + 8 * lane;
                    const float2 sx = *reinterpret_cast<const float2 *>(scales + (m * columns + c) / 16 + 2 * lane);
                    float sum[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        __half2 s = __float2half2_rn(0.f);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint4 q = *reinterpret_cast<const uint4 *>(x + (2 * h + i) * 256);
                            const __half2 *t = reinterpret_cast<const __half2 *>(&q);
#pragma unroll
                            for (int e = 0; e < 4; ++e) s = __hfma2(b[8 * h + 4 * i + e], t[e], s);
                        }
                        const float2 f = __half22float2(s);
                        sum[h] = f.x + f.y;
                    }
                    acc[m] = fmaf(sum[0], sb.x * sx.x, acc[m]);
                    acc[m] = fmaf(sum[1], sb.y * sx.y, acc[m]);
                }
            }
        }
        const int done = row;
        row = row_of(group + gridDim.x);
        if (group + (int)gridDim.x < groups) load(row, 0);
        float mine = 0.f;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const float s = warp_sum(acc[m]);
            if (lane == m) mine = s;
        }
        if (lane < MT && lane < p.M && done < p.N)
            store_c(p.C, lane * p.ldc + done, p.ctype,
                    fmaf(mine * row_scales[lane], p.b_scale ? p.b_scale[done] : 1.f, p.bias ? p.bias[done] : 0.f));
    }
}

}  // namespace sgemm
